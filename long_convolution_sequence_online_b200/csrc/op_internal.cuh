// Declarations of the context-free operators (linear attention, linear layer):
// launchers in k_linattn*.cu and k_linear_*.cu, argument checks and entry points
// in op_api.cu.
#pragma once

#include <atomic>

#include "fi_internal.cuh"

namespace fi {

// The operators' launches allow programmatic stream serialization and wait for the
// launch before them ahead of their first read or write of global memory. Only
// those that another launch of the same call follows let that one start early: a
// later launch of the library's (the chunk kernel, say) reads what it takes for
// long finished before it waits, and that may be an operator's result.

// Checks of a barrier after which a wait in a kernel launched from now on gives up
// (fi_debug_set_op_wait_limit).
int op_wait_limit();

// Allows a kernel `bytes` of dynamic shared memory, once per device (a kernel's
// need is a constant of its instantiation).
template <auto Kern>
cudaError_t allow_smem(size_t bytes) {
  static std::atomic<uint64_t> done{0};     // bit per device; devices beyond 63 set it on every call
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// ---------------------------------------------------------------- linear attention
// Sizes and strides as in fi_linattn_config (strides in elements: position,
// sequence, head), widened for address arithmetic.
struct LaShape {
  int H, dk, dv, B, n;
  int bf16;
  float scale;
  int64_t qs[3], ks[3], vs[3], os[3];
  // Tensor-core form of a block of key dimensions: where the states' blocks lie (elements
  // between (sequence, head)s, between rows).
  int64_t state_slot;
  int state_ld;
};

// A prompt is cut into G segments of seg positions (a multiple of the chunk)
// that run at the same time: a first launch forms every segment's own
// contribution to the state, a second one adds up those before a segment and
// computes its outputs. G = 1: one launch, no scratch.
struct LaPlan {
  int G, seg;
};
// Scratch of a plan: slot 0 of (sequence, head) holds the state before the
// prompt, slot g the contribution of segment g - 1.
inline size_t la_workspace_bytes(const LaShape& s, const LaPlan& p) {
  return p.G > 1 ? ((size_t)s.B * s.H * p.G * s.dk * s.dv * sizeof(float) + 255) / 256 * 256 : 0;
}

struct LaPtrs {
  const void *q, *k, *v;
  const float* log_decay;
  const int32_t* lengths;   // NULL: all n
  const float* state_in;    // NULL: zeros
  float* state_out;         // NULL: not written
  void* o;
  float* ws;
};
// Scratch of a prompt: the segments' states, then inputs that are laid out first.
size_t linattn_prefill_workspace(const LaShape& s, const LaPtrs& a, int num_sms);
cudaError_t launch_linattn_prefill(const LaShape& s, const LaPtrs& a, void* workspace, int num_sms, cudaStream_t st);
// Tensor-core form (k_linattn_tc.cu): bf16 dimensions up to 128, fp32 in blocks of 64
// (linattn_tc_block: the heads and dimensions that a launch works on, for the plan and its
// scratch). `layout`: scratch for inputs that no tensor map describes, and all fp32 ones.
bool linattn_tc_fits(const LaShape& s);
LaShape linattn_tc_block(const LaShape& s);
size_t linattn_tc_layout_bytes(const LaShape& s, const LaPtrs& a);
LaPlan linattn_tc_plan(const LaShape& block, int num_sms);
cudaError_t launch_linattn_tc(const LaShape& s, const LaPlan& p, const LaPtrs& a, void* layout, int num_sms, cudaStream_t st);
// Whether a bounded wait gave up in these kernels since the last check
// (synchronises the stream; the flag is cleared).
cudaError_t linattn_take_error(cudaStream_t st, int* flag);
cudaError_t launch_linattn_step(const LaShape& s, const void* q, const void* k, const void* v, const float* log_decay,
                                float* state, void* o, cudaStream_t st);

// The decay's exponent base 2 per position; log_decay above 0 counts as 0, and
// -infinity becomes a finite value whose powers underflow to 0 (a lag of 0
// still gives 1). NaN stays NaN.
__device__ __forceinline__ float la_log2_decay(float log_decay) {
  const float l = log_decay < -1e30f ? -1e30f : (log_decay > 0.f ? 0.f : log_decay);
  return (float)((double)l * 1.4426950408889634);
}
// A decay of 0 (log_decay -infinity): the state before is dropped whatever it holds,
// where 0 times an infinity would be NaN. A power that merely underflows does not drop
// it: an infinity there stays one.
__device__ __forceinline__ bool la_drops(float log2_decay) { return log2_decay < -1e30f; }
// g^lag, lag >= 0.
__device__ __forceinline__ float la_pow(float log2_decay, int lag) { return exp2f(log2_decay * (float)lag); }

__device__ __forceinline__ int la_length(const int32_t* lengths, int b, int n) {
  if (!lengths) return n;
  const int l = __ldg(lengths + b);
  return l < 0 ? 0 : (l > n ? n : l);
}

// ---------------------------------------------------------------- linear layer
struct LinShape {
  int n, K, N;      // rows, in_features, out_features
  int bf16, act;
  int64_t ldx, ldw, ldr, ldy;
};
// Scratch for operands that have to be laid out first (256-byte aligned).
size_t linear_workspace(const LinShape& s, const void* x, const void* w);
cudaError_t launch_linear(const LinShape& s, const void* x, const void* w, const void* bias, const void* residual,
                          void* y, void* workspace, int num_sms, cudaStream_t st);
struct LinCall {
  const LinShape& s;
  const void *x, *w, *bias, *residual;
  void* y;
  int num_sms;
  cudaStream_t st;
};
// Few rows (k_linear_few.cu): tensor cores with W's rows as the wide side (operands
// by TMA), or a warp per row of W (any operands, n <= kWarpRows).
constexpr int kFewRows = 128, kWarpRows = 8;
bool linear_few_fits(const LinShape& s, int num_sms);
cudaError_t launch_linear_few(const LinCall& c);
cudaError_t launch_linear_rows(const LinCall& c);
// 16-byte aligned address and row stride.
inline bool linear_aligned16(const void* p, int64_t ld, int64_t rows, size_t esz) {
  return ((uintptr_t)p & 15) == 0 && (rows <= 1 || (ld * (int64_t)esz) % 16 == 0);
}
// Whether a bounded wait gave up in these kernels since the last check
// (synchronises the stream; the flag is cleared).
cudaError_t linear_take_error(cudaStream_t st, int* flag);
cudaError_t linear_few_take_error(cudaStream_t st, int* flag);

__device__ __forceinline__ float ex2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// GELU: u Phi(u) from the tail Phi(-z) = exp(-z^2/2) t Q(t), t = 1 / (1 + 0.21 z), z = |u|;
// Q is a least-maximum fit of degree 8 made for this form (relative error 1.9e-8 for z up
// to 14.5). By the error function, 1 + erf(u / sqrt 2) cancels for negative u (10 % off at
// -5, 0 below -5.6); by CUDA's complementary one it does not, but takes 7 us more of 59 in
// 8192 x 768 -> 768. The result is within (16 + 1.5 u^2) 2^-24 of itself (u^2: the
// exponent's roundings); below 2^-126 (u under -13.2) it may become 0.
template <int ACT>
__device__ __forceinline__ float linear_act(float u) {
  if constexpr (ACT == FI_ACT_GELU) {
    const float z = fminf(fabsf(u), 14.5f), d = fmaf(0.21f, z, 1.f);
    float t = rcp_fast(d);
    t = fmaf(t, fmaf(-d, t, 1.f), t);
    float p = fmaf(-0.07129445672035217f, t, 0.2818029224872589f);
    p = fmaf(p, t, -0.32648995518684387f);
    p = fmaf(p, t, 0.34498298168182373f);
    p = fmaf(p, t, -0.09077012538909912f);
    p = fmaf(p, t, 0.12347106635570526f);
    p = fmaf(p, t, 0.06957001239061356f);
    p = fmaf(p, t, 0.08501239866018295f);
    p = fmaf(p, t, 0.08371515572071075f);
    const float tail = z * (p * t) * ex2_fast(z * z * -0.72134752f);
    return u > 0.f ? u - tail : fmaf(u, 0.f, -tail);   // NaN stays, -infinity becomes it (u 0), as in u Phi(u)
  }
  if constexpr (ACT == FI_ACT_SILU) return u / (1.0f + expf(-u));
  if constexpr (ACT == FI_ACT_RELU) return u > 0.f || u != u ? u : 0.f;
  if constexpr (ACT == FI_ACT_TANH) return tanhf(u);
  return u;
}

// The same for results that are rounded to bf16 (2^-9 of the value on average), in
// fewer instructions (a tile's activations otherwise take as long as its
// products). GELU: as above with t = 1 / (1 + 0.265 z) and a fit of degree 6
// (relative error 6.3e-7 for z up to 14, where the tail is 8e-45).
// tanh: its series below 0.2, (1 - e) / (1 + e) with e = exp(-2 |u|) above.
// Relative errors: 1e-6, and for exponentials of large arguments the rounding of the
// argument besides: 2e-6 for GELU at -6, 7e-6 at -12, as much for SiLU at -80. Values
// below 2^-126 (GELU under -13.2, SiLU under -87) may become 0.
template <int ACT>
__device__ __forceinline__ float linear_act_bf16(float u) {
  if constexpr (ACT == FI_ACT_GELU) {
    const float z = fminf(fabsf(u), 14.f);
    const float t = rcp_fast(fmaf(0.265f, z, 1.f));
    float p = fmaf(-0.06778856f, t, 0.1952782f);
    p = fmaf(p, t, -0.06636963f);
    p = fmaf(p, t, 0.14249772f);
    p = fmaf(p, t, 0.08294514f);
    p = fmaf(p, t, 0.107837f);
    p = fmaf(p, t, 0.10559982f);
    const float tail = z * (p * t) * ex2_fast(z * z * -0.72134752f);
    return u > 0.f ? u - tail : fmaf(u, 0.f, -tail);   // NaN stays, -infinity becomes it (u 0), as in u Phi(u)
  }
  if constexpr (ACT == FI_ACT_SILU) return __fdividef(u, 1.0f + __expf(-u));
  if constexpr (ACT == FI_ACT_TANH) {
    const float z = fabsf(u), z2 = z * z;
    const float e = ex2_fast(z * -2.8853900817779268f);
    const float big = (1.f - e) * rcp_fast(1.f + e);
    const float small = z * fmaf(z2, fmaf(z2, fmaf(z2, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
    return copysignf(z < 0.2f ? small : big, u);
  }
  return linear_act<ACT>(u);
}

// One value of a bf16 or fp32 array, and one rounded into it.
template <typename T>
__device__ __forceinline__ float op_load(const T* p) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(*p);
  else return *p;
}
template <typename T>
__device__ __forceinline__ void op_store(T* p, float v) {
  if constexpr (sizeof(T) == 2) *p = __float2bfloat16_rn(v);
  else *p = v;
}

}  // namespace fi
