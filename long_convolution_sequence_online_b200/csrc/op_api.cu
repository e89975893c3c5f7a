// C-ABI of the context-free operators (declared in include/fi.h): argument
// checks and launches.
#include <algorithm>
#include <cmath>
#include <string>

#include "op_internal.cuh"

using namespace fi;

namespace {

fi_status fail(fi_status s, const std::string& msg) {
  set_last_error(msg);
  return s;
}
fi_status invalid(const std::string& msg) { return fail(FI_E_INVALID, msg); }
fi_status cuda_fail(cudaError_t e, const char* what) {
  cudaGetLastError();
  return fail(FI_E_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

cudaError_t device_sms(int* sms) {
  static std::atomic<int> known[64];       // by device; 0: not asked yet
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
  return e;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Sequences x heads: with up to 4 blocks of dimensions and 64 segments each, tasks are
// counted below 2^31.
constexpr int64_t kMaxRows = 1 << 22;
constexpr int32_t kMaxPositions = 1 << 29;        // the three parts of fp32 rows are indexed below 2^31
constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxLd = (int64_t)1 << 38;      // below a tensor map's 2^40 bytes

// cfg -> s. `positions`: the number of positions the strides [0] step over (1:
// not used).
fi_status check_linattn(const fi_linattn_config* c, int64_t positions, LaShape* s) {
  if (!c) return invalid("cfg is NULL");
  if (c->heads < 1) return invalid("heads must be >= 1");
  if (c->batch < 1) return invalid("batch must be >= 1");
  if (c->key_dim < 1 || c->key_dim > 256) return invalid("key_dim must be in [1, 256]");
  if (c->value_dim < 1 || c->value_dim > 256) return invalid("value_dim must be in [1, 256]");
  if ((int64_t)c->heads * c->batch > kMaxRows) return invalid("batch x heads must be <= " + std::to_string(kMaxRows));
  if (c->dtype != FI_F32 && c->dtype != FI_BF16) return invalid("dtype must be FI_F32 or FI_BF16");
  if (!std::isfinite(c->scale)) return invalid("scale must be finite");
  for (int r : c->reserved)
    if (r != 0) return invalid("reserved fields must be 0");
  for (int i = 0; i < 3; ++i)
    for (int64_t v : {c->q_stride[i], c->k_stride[i], c->v_stride[i], c->o_stride[i]})
      if (v < 0 || v > kMaxStride) return invalid("strides must be in [0, 2^40]");
  // o's elements are distinct when, from the smallest stride up, each stride
  // passes over the whole extent below it
  struct Dim { int64_t stride, count; } d[3] = {{c->o_stride[0], positions}, {c->o_stride[1], c->batch}, {c->o_stride[2], c->heads}};
  std::sort(d, d + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  __int128 extent = c->value_dim;
  for (const Dim& x : d) {
    if (x.count <= 1) continue;
    if (x.stride < extent) return invalid("o_stride: rows of o overlap");
    extent += (__int128)x.stride * (x.count - 1);
  }
  *s = LaShape{};
  s->H = c->heads;
  s->dk = c->key_dim;
  s->dv = c->value_dim;
  s->B = c->batch;
  s->bf16 = c->dtype == FI_BF16;
  s->scale = c->scale;
  for (int i = 0; i < 3; ++i) {
    s->qs[i] = c->q_stride[i];
    s->ks[i] = c->k_stride[i];
    s->vs[i] = c->v_stride[i];
    s->os[i] = c->o_stride[i];
  }
  return FI_OK;
}

fi_status check_linear(const fi_linear_config* c, int32_t n, bool residual, LinShape* s) {
  if (!c) return invalid("cfg is NULL");
  if (n < 0 || n > kMaxPositions) return invalid("n must be in [0, 2^29]");
  if (c->in_features < 1 || c->in_features > (1 << 20)) return invalid("in_features must be in [1, 2^20]");
  if (c->out_features < 1 || c->out_features > (1 << 20)) return invalid("out_features must be in [1, 2^20]");
  if (c->dtype != FI_F32 && c->dtype != FI_BF16) return invalid("dtype must be FI_F32 or FI_BF16");
  if (c->act < FI_ACT_NONE || c->act > FI_ACT_TANH) return invalid("act must be an fi_act");
  for (int r : c->reserved)
    if (r != 0) return invalid("reserved fields must be 0");
  for (int64_t v : {c->ldx, c->ldw, c->ldr, c->ldy})
    if (v < 0 || v > kMaxLd) return invalid("leading dimensions must be in [0, 2^38]");
  if (c->ldx != 0 && c->ldx < c->in_features) return invalid("ldx must be >= in_features, or 0");
  if (c->ldw < c->in_features) return invalid("ldw must be >= in_features");
  if (c->ldy < c->out_features) return invalid("ldy must be >= out_features");
  if (residual && c->ldr != 0 && c->ldr < c->out_features) return invalid("ldr must be >= out_features, or 0");
  if ((int64_t)n * c->out_features > (int64_t)1 << 40) return invalid("n x out_features must be <= 2^40");
  *s = LinShape{n, c->in_features, c->out_features, c->dtype == FI_BF16, c->act, c->ldx, c->ldw, c->ldr, c->ldy};
  return FI_OK;
}

std::atomic<int> g_wait_limit{kDefaultWaitLimit};

}  // namespace

int fi::op_wait_limit() { return g_wait_limit.load(std::memory_order_relaxed); }

extern "C" {

fi_status fi_debug_set_op_wait_limit(int32_t limit) {
  g_wait_limit.store(limit < 0 ? kDefaultWaitLimit : limit, std::memory_order_relaxed);
  return FI_OK;
}

fi_status fi_linattn_workspace(const fi_linattn_config* cfg, int32_t n, const void* q, const void* k, const void* v,
                               uint64_t* bytes) {
  if (!bytes) return invalid("bytes is NULL");
  *bytes = 0;
  if (n < 0 || n > kMaxPositions) return invalid("n must be in [0, 2^29]");
  LaShape s;
  const fi_status r = check_linattn(cfg, n, &s);
  if (r != FI_OK) return r;
  if (n == 0) return FI_OK;
  s.n = n;
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  const LaPtrs a{q, k, v, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr};
  *bytes = linattn_prefill_workspace(s, a, sms);
  return FI_OK;
}

fi_status fi_linattn_prefill(const fi_linattn_config* cfg, int32_t n, const void* q, const void* k, const void* v,
                             const float* log_decay, const int32_t* lengths, const float* state_in, float* state_out,
                             void* o, void* workspace, uint64_t workspace_bytes, void* stream) {
  if (n < 0 || n > kMaxPositions) return invalid("n must be in [0, 2^29]");
  LaShape s;
  const fi_status r = check_linattn(cfg, n, &s);
  if (r != FI_OK) return r;
  if (!log_decay || (n > 0 && (!q || !k || !v || !o))) return invalid("NULL argument");
  const size_t esz = s.bf16 ? 2 : 4;
  if (!aligned(q, esz) || !aligned(k, esz) || !aligned(v, esz) || !aligned(o, esz) || !aligned(log_decay, 4) ||
      !aligned(lengths, 4) || !aligned(state_in, 4) || !aligned(state_out, 4))
    return invalid("a pointer is not aligned to its element size");
  if (n > 0 && (o == q || o == k || o == v)) return invalid("o must not be an input");
  if (state_in && state_out && state_in != state_out) {
    // one (sequence, head)'s state would be written before another's is read
    const uint64_t bytes = (uint64_t)s.B * s.H * s.dk * s.dv * 4, a = (uintptr_t)state_in, b = (uintptr_t)state_out;
    if ((a < b ? b - a : a - b) < bytes) return invalid("state_in and state_out overlap without being the same");
  }
  s.n = n;
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  const LaPtrs a{q, k, v, log_decay, lengths, state_in, state_out, o, nullptr};
  const size_t need = linattn_prefill_workspace(s, a, sms);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return invalid("workspace: " + std::to_string(need) + " bytes, 256-byte aligned, are needed");
  e = launch_linattn_prefill(s, a, need ? workspace : nullptr, sms, (cudaStream_t)stream);
  return e == cudaSuccess ? FI_OK : cuda_fail(e, "linear attention prefill launch");
}

fi_status fi_linattn_step(const fi_linattn_config* cfg, const void* q, const void* k, const void* v,
                          const float* log_decay, float* state, void* o, void* stream) {
  LaShape s;
  const fi_status r = check_linattn(cfg, 1, &s);
  if (r != FI_OK) return r;
  if (!q || !k || !v || !log_decay || !state || !o) return invalid("NULL argument");
  const size_t esz = s.bf16 ? 2 : 4;
  if (!aligned(q, esz) || !aligned(k, esz) || !aligned(v, esz) || !aligned(o, esz) || !aligned(log_decay, 4) ||
      !aligned(state, 4))
    return invalid("a pointer is not aligned to its element size");
  if (o == q || o == k || o == v) return invalid("o must not be an input");
  s.n = 1;
  const cudaError_t e = launch_linattn_step(s, q, k, v, log_decay, state, o, (cudaStream_t)stream);
  return e == cudaSuccess ? FI_OK : cuda_fail(e, "linear attention step launch");
}

fi_status fi_op_sync(void* stream) {
  int a = 0, b = 0, d = 0;
  cudaError_t e = linear_take_error((cudaStream_t)stream, &a);
  if (e == cudaSuccess) e = linear_few_take_error((cudaStream_t)stream, &d);
  if (e == cudaSuccess) e = linattn_take_error((cudaStream_t)stream, &b);
  if (e != cudaSuccess) return cuda_fail(e, "operator check");
  return a || b || d ? fail(FI_E_TIMEOUT, "a bounded wait in an operator's kernel gave up") : FI_OK;
}

fi_status fi_linear_workspace(const fi_linear_config* cfg, int32_t n, const void* x, const void* w, uint64_t* bytes) {
  if (!bytes) return invalid("bytes is NULL");
  *bytes = 0;
  LinShape s;
  const fi_status r = check_linear(cfg, n, false, &s);
  if (r != FI_OK || n == 0) return r;
  *bytes = linear_workspace(s, x, w);
  return FI_OK;
}

fi_status fi_linear(const fi_linear_config* cfg, int32_t n, const void* x, const void* w, const void* bias,
                    const void* residual, void* y, void* workspace, uint64_t workspace_bytes, void* stream) {
  LinShape s;
  const fi_status r = check_linear(cfg, n, residual != nullptr, &s);
  if (r != FI_OK || n == 0) return r;
  if (!x || !w || !y) return invalid("NULL argument");
  const size_t esz = s.bf16 ? 2 : 4;
  if (!aligned(x, esz) || !aligned(w, esz) || !aligned(y, esz) || !aligned(bias, esz) || !aligned(residual, esz))
    return invalid("a pointer is not aligned to its element size");
  if (y == x || y == w || y == bias) return invalid("y must not be an input");
  if (y == residual && s.ldr != s.ldy && n > 1) return invalid("residual may be y only with ldr == ldy");
  const size_t need = linear_workspace(s, x, w);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return invalid("workspace: " + std::to_string(need) + " bytes, 256-byte aligned, are needed");
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  e = launch_linear(s, x, w, bias, residual, y, workspace, sms, (cudaStream_t)stream);
  return e == cudaSuccess ? FI_OK : cuda_fail(e, "linear layer launch");
}

}  // extern "C"
