// Linear layer for few rows of x: every byte of W is read once and the rest is
// latency, so W's rows take the MMA's 128-row side, the rows of x the narrow
// one, and the contraction is split over a cluster of CTAs until the GPU is full.
#include "op_internal.cuh"
#include "tc.cuh"

namespace fi {

namespace {

using namespace tc;

constexpr int kBM = 128, kBK = 64;        // W rows per CTA, contraction per stage
constexpr int kFewThreads = 128;

__device__ int g_few_error;               // a bounded wait gave up since the last check

template <int NT>
constexpr int few_stage() { return (kBM + NT) * 128; }
template <int NT>
constexpr int few_stages() { return 98304 / few_stage<NT>(); }   // two CTAs per SM
template <int NT>
constexpr size_t few_smem() { return 1024 + (size_t)few_stages<NT>() * few_stage<NT>(); }

__device__ __forceinline__ float4 ld_cluster4(const float* p, uint32_t rank) {
  uint32_t at;
  float4 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(saddr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
  return v;
}

// Cluster of `split` CTAs: the same 128 rows of W, consecutive parts of the
// contraction. Each leaves its sums [NT][128] in shared memory; each then adds up
// 128 / split rows of all of them (in rank order) and finishes those outputs.
template <int NT, int ACT>
__global__ void __launch_bounds__(kFewThreads)
k_linear_few(LinShape s, const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
             const __nv_bfloat16* __restrict__ bias, const __nv_bfloat16* residual, __nv_bfloat16* y, int split,
             int vec, int wait_limit) {
  using T = __nv_bfloat16;
  constexpr int ST = few_stages<NT>(), SB = few_stage<NT>();
  constexpr uint32_t kCols = NT < 32 ? 32 : NT;
  extern __shared__ unsigned char raw_smem[];
  __shared__ uint64_t full[ST], empty[ST], done;
  __shared__ uint32_t tmem_s;
  __shared__ int abort_s;
  unsigned char* ring = raw_smem + ((1024 - (saddr(raw_smem) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  const int rank = split > 1 ? (int)cluster_rank() : 0;
  const int row0 = (int)(blockIdx.x / split) * kBM;
  const int blocks = (s.K + kBK - 1) / kBK;
  const int b0 = (int)((int64_t)blocks * rank / split), b1 = (int)((int64_t)blocks * (rank + 1) / split);
  if (warp == 0) tmem_alloc(&tmem_s, kCols);
  if (tid == 32) {
    for (int i = 0; i < ST; ++i) {
      bar_init(&full[i], 1);
      bar_init(&empty[i], 1);
    }
    bar_init(&done, 1);
    abort_s = 0;
    bar_init_fence();
    tma_prefetch(&xmap);
    tma_prefetch(&wmap);
  }
  fence_before();
  __syncthreads();
  fence_after();
  pdl_wait_primary();                     // from here on inputs are read and y is written
  const uint32_t tmem = tmem_s;
  volatile int* abort_flag = &abort_s;
  auto give_up = [&]() {
    *abort_flag = 1;
    atomicExch(&g_few_error, 1);
  };
  if (warp == 0) {
    const bool issuer = elect_one();
    bool alive = true;
    int i = 0;
    for (; i < b1 - b0; ++i) {
      const int st = i % ST;
      alive = __all_sync(0xffffffffu, i < ST || bar_wait(&empty[st], (i / ST - 1) & 1, wait_limit, abort_flag));
      if (!alive) break;
      if (issuer) {
        unsigned char* dst = ring + st * SB;
        bar_expect(&full[st], SB);
        tma_2d(dst, &wmap, &full[st], (b0 + i) * kBK, row0);
        tma_2d(dst + kBM * 128, &xmap, &full[st], (b0 + i) * kBK, 0);
      }
      __syncwarp();
    }
    if (!alive && lane == 0) give_up();
    // no copy of this CTA may still be in flight when its memory is reused
    for (int j = i > ST ? i - ST : 0; j < i; ++j) bar_wait(&full[j % ST], (j / ST) & 1, kDefaultWaitLimit);
  } else if (warp == 1) {
    const bool issuer = elect_one();
    constexpr uint32_t id = idesc(kBM, NT);
    bool alive = true;
    for (int i = 0; i < b1 - b0; ++i) {
      const int st = i % ST;
      alive = __all_sync(0xffffffffu, bar_wait(&full[st], (i / ST) & 1, wait_limit, abort_flag));
      if (!alive) break;
      fence_after();
      if (issuer) {
        const uint32_t wa = saddr(ring + st * SB), xa = wa + kBM * 128;
#pragma unroll
        for (int k = 0; k < kBK / 16; ++k) mma(tmem, desc_k(wa + 32 * k), desc_k(xa + 32 * k), id, i > 0 || k > 0);
        commit(&empty[st]);
      }
      __syncwarp();
    }
    if (!alive && lane == 0) give_up();
    if (issuer) commit(&done);
    __syncwarp();
  }
  // all MMAs (and with them all copies) are done: shared memory is free
  const bool arrived = bar_wait(&done, 0, kDefaultWaitLimit);
  if (!arrived) give_up();
  fence_after();
  __syncthreads();
  float* part = reinterpret_cast<float*>(ring);           // [NT][128]
  const uint32_t at = tmem + ((uint32_t)(32 * warp) << 16);
#pragma unroll
  for (int c = 0; c < NT; c += 16) {
    if (c >= s.n) break;
    uint32_t r[16];
    tmem_ld16(at + c, r);
    ld_wait();
#pragma unroll
    for (int e = 0; e < 16; ++e) part[(c + e) * kBM + tid] = b1 > b0 ? __uint_as_float(r[e]) : 0.f;
  }
  if (split > 1) cluster_sync();
  else __syncthreads();
  // Four rows of W and one row of x at a time; every CTA's sums are asked for
  // before the first is used (one at a time, 64 rows took 9.1 us instead of FEW_US).
  const int quads = kBM / 4 / split;                       // of this CTA to finish
  const int r = (rank * quads + tid % quads) * 4, c = row0 + r;
  if (c < s.N) {
    const int m = min(4, s.N - c);
    float bv[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) bv[e] = bias && e < m ? op_load(bias + c + e) : 0.f;
    for (int t = tid / quads; t < s.n; t += kFewThreads / quads) {
      float4 v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < split) v[q] = split == 1 ? *reinterpret_cast<const float4*>(part + t * kBM + r) : ld_cluster4(part + t * kBM + r, q);
      float u[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int q = 1; q < 8; ++q)
        if (q < split) {
          u[0] += v[q].x;
          u[1] += v[q].y;
          u[2] += v[q].z;
          u[3] += v[q].w;
        }
      const T* rp = residual + t * s.ldr + c;
      T* yp = y + t * s.ldy + c;
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = linear_act_bf16<ACT>(u[e] + bv[e]);
      if (vec) {                                           // N, the strides and the addresses allow it
        if (residual) {
          const uint2 x = *reinterpret_cast<const uint2*>(rp);
          u[0] += lo_f(x.x);
          u[1] += hi_f(x.x);
          u[2] += lo_f(x.y);
          u[3] += hi_f(x.y);
        }
        *reinterpret_cast<uint2*>(yp) = make_uint2(pack2(u[0], u[1]), pack2(u[2], u[3]));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < m) op_store(yp + e, u[e] + (residual ? op_load(rp + e) : 0.f));
      }
    }
  }
  fence_before();
  if (split > 1) cluster_sync_relaxed();                   // others may still read this CTA's sums
  else __syncthreads();
  fence_after();
  if (warp == 0) tmem_free(tmem, kCols);
}

// fp32, and bf16 rows at no 16-byte boundary: a warp per row of W, its lanes
// along the contraction, applied to kGroup rows of x at once.
constexpr int kGroup = 8;
template <typename T, int ACT, bool VEC>
__global__ void __launch_bounds__(256) k_linear_rows(LinShape s, const T* __restrict__ x, const T* __restrict__ w,
                                                    const T* __restrict__ bias, const T* residual, T* y) {
  pdl_launch_dependents();
  pdl_wait_primary();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 8 + warp;
  const int t0 = blockIdx.y * kGroup, nt = min(kGroup, s.n - t0);
  if (c >= s.N) return;
  const T* wr = w + (int64_t)c * s.ldw;
  const T* xr = x + (int64_t)t0 * s.ldx;
  float acc[kGroup] = {};
  constexpr int E = VEC ? 16 / (int)sizeof(T) : 1;          // elements per load
  constexpr int U = VEC ? 4 : 8;                            // loads of W in flight
  for (int k0 = lane * E; k0 < s.K; k0 += 32 * E * U) {
    float wv[U][E];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * 32 * E;
      if constexpr (VEC) {
        uint4 q = make_uint4(0, 0, 0, 0);
        if (k < s.K) q = __ldg(reinterpret_cast<const uint4*>(wr + k));
        const uint32_t v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (sizeof(T) == 2) {
            wv[u][2 * e] = lo_f(v[e]);
            wv[u][2 * e + 1] = hi_f(v[e]);
          } else {
            wv[u][e] = __uint_as_float(v[e]);
          }
        }
      } else {
        wv[u][0] = k < s.K ? op_load(wr + k) : 0.f;
      }
    }
#pragma unroll
    for (int t = 0; t < kGroup; ++t) {
      if (t >= nt) break;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * 32 * E;
        if (k >= s.K) break;
        const T* xp = xr + t * s.ldx + k;
        if constexpr (VEC) {
          const uint4 q = __ldg(reinterpret_cast<const uint4*>(xp));
          const uint32_t v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (sizeof(T) == 2) {
              acc[t] = fmaf(wv[u][2 * e], lo_f(v[e]), acc[t]);
              acc[t] = fmaf(wv[u][2 * e + 1], hi_f(v[e]), acc[t]);
            } else {
              acc[t] = fmaf(wv[u][e], __uint_as_float(v[e]), acc[t]);
            }
          }
        } else {
          acc[t] = fmaf(wv[u][0], op_load(xp), acc[t]);
        }
      }
    }
  }
  float out = 0.f;
#pragma unroll
  for (int t = 0; t < kGroup; ++t) {
    if (t >= nt) break;
    float v = acc[t];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == t) out = v;
  }
  if (lane < nt) {
    const int64_t t = t0 + lane;
    float u = linear_act<ACT>(out + (bias ? op_load(bias + c) : 0.f));
    if (residual) u += op_load(residual + t * s.ldr + c);
    op_store(y + t * s.ldy + c, u);
  }
}

template <int NT, int ACT>
cudaError_t run_few(const LinCall& c) {
  const LinShape& s = c.s;
  constexpr auto kern = k_linear_few<NT, ACT>;
  constexpr size_t smem = few_smem<NT>();
  cudaError_t e = allow_smem<kern>(smem);
  if (e != cudaSuccess) return e;
  CUtensorMap xmap, wmap;
  if (!linear_map(&xmap, c.x, s.n, s.K, s.ldx, NT) || !linear_map(&wmap, c.w, s.N, s.K, s.ldw, kBM)) return cudaErrorInvalidValue;
  const int tiles = (s.N + kBM - 1) / kBM, blocks = (s.K + kBK - 1) / kBK;
  int split = 1;
  while (split < 8 && 2 * split * tiles <= 2 * c.num_sms && 2 * split <= blocks) split *= 2;
  const int vec = s.N % 4 == 0 && (uintptr_t)c.y % 8 == 0 && s.ldy % 4 == 0 &&
                  (!c.residual || ((uintptr_t)c.residual % 8 == 0 && s.ldr % 4 == 0));
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * split));
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, s, xmap, wmap, (const __nv_bfloat16*)c.bias, (const __nv_bfloat16*)c.residual,
                            (__nv_bfloat16*)c.y, split, vec, (int)kDefaultWaitLimit);
}

template <int ACT>
cudaError_t run_few_nt(const LinCall& c) {
  if (c.s.n <= 16) return run_few<16, ACT>(c);
  if (c.s.n <= 32) return run_few<32, ACT>(c);
  if (c.s.n <= 64) return run_few<64, ACT>(c);
  return run_few<128, ACT>(c);
}

template <typename T, int ACT>
cudaError_t run_rows(const LinCall& c) {
  const LinShape& s = c.s;
  constexpr int E = 16 / (int)sizeof(T);
  const bool vec = s.K % E == 0 && linear_aligned16(c.x, s.ldx, s.n, sizeof(T)) && linear_aligned16(c.w, s.ldw, s.N, sizeof(T));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((s.N + 7) / 8), (unsigned)((s.n + kGroup - 1) / kGroup));
  cfg.blockDim = dim3(256);
  cfg.stream = c.st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kern = vec ? k_linear_rows<T, ACT, true> : k_linear_rows<T, ACT, false>;
  return cudaLaunchKernelEx(&cfg, kern, s, (const T*)c.x, (const T*)c.w, (const T*)c.bias, (const T*)c.residual, (T*)c.y);
}

}  // namespace

cudaError_t launch_linear_few(const LinCall& c) {
  switch (c.s.act) {
    case FI_ACT_NONE: return run_few_nt<FI_ACT_NONE>(c);
    case FI_ACT_GELU: return run_few_nt<FI_ACT_GELU>(c);
    case FI_ACT_SILU: return run_few_nt<FI_ACT_SILU>(c);
    case FI_ACT_RELU: return run_few_nt<FI_ACT_RELU>(c);
    case FI_ACT_TANH: return run_few_nt<FI_ACT_TANH>(c);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_linear_rows(const LinCall& c) {
#define FI_ROWS(A) case A: return c.s.bf16 ? run_rows<__nv_bfloat16, A>(c) : run_rows<float, A>(c)
  switch (c.s.act) {
    FI_ROWS(FI_ACT_NONE);
    FI_ROWS(FI_ACT_GELU);
    FI_ROWS(FI_ACT_SILU);
    FI_ROWS(FI_ACT_RELU);
    FI_ROWS(FI_ACT_TANH);
  }
#undef FI_ROWS
  return cudaErrorInvalidValue;
}

cudaError_t linear_few_take_error(cudaStream_t st, int* flag) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(flag, g_few_error, sizeof(int), 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && *flag) {
    const int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_few_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  return e;
}

}  // namespace fi
