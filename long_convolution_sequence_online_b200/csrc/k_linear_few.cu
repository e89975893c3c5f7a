// Linear layer for few rows of x: every byte of W is read once and the rest is
// latency, so W's rows take the MMA's 128-row side, the rows of x the narrow
// one, and the contraction is split over a cluster of CTAs until the GPU is full.
// 1 x 2048 -> 8192 bf16: 8.0 us (W's 34 MB from memory at 4.2 TB/s, launch and first loads
// included; 7.1 with W in L2), 64 x 2048 -> 2048 7.4 us, bound by latency.
#include "op_internal.cuh"
#include "tc.cuh"

namespace fi {

namespace {

using namespace tc;

constexpr int kBM = 128, kBK = 64;        // W rows per CTA, contraction per stage
constexpr int kFewThreads = 128;

__device__ int g_few_error;               // a bounded wait gave up since the last check

// A stage: a block of 64 of W's and x's rows, in 1 (bf16) or 3 (fp32) parts. bf16: two
// CTAs per SM.
template <int NT, int PARTS>
constexpr int few_stage() { return PARTS * (kBM + NT) * 128; }
template <int NT, int PARTS>
constexpr int few_stages() { return (PARTS == 1 ? 98304 : 221184) / few_stage<NT, PARTS>(); }
template <int NT, int PARTS>
constexpr size_t few_smem() { return 1024 + (size_t)few_stages<NT, PARTS>() * few_stage<NT, PARTS>(); }
// fp32: every block of the contraction has an accumulator of its own, since the tensor core's
// sums are not rounded to nearest: 1e-7 off in the 2-norm, with two blocks to an
// accumulator 6e-7. They are added up in registers: at the end, or in a second round where
// a CTA's blocks do not fit tensor memory (more rounds would leave the products waiting).
constexpr int kRounds = 2;
template <int NT, int PARTS>
constexpr int few_accs() { return PARTS == 3 ? 512 / NT : 1 << 30; }   // blocks of a round

// Cluster of `split` CTAs: the same 128 rows of W, consecutive parts of the
// contraction. Each leaves its sums [NT][128] in shared memory; each then adds up
// 128 / split rows of all of them (in rank order) and finishes those outputs.
template <int NT, int PARTS, typename T, int ACT>
__global__ void __launch_bounds__(kFewThreads)
k_linear_few(LinShape s, const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
             const T* __restrict__ bias, const T* residual, T* y, int split, int cols, int vec, int wait_limit) {
  constexpr int ST = few_stages<NT, PARTS>(), SB = few_stage<NT, PARTS>(), WB = kBM * 128, XB = NT * 128;
  extern __shared__ unsigned char raw_smem[];
  __shared__ uint64_t full[ST], empty[ST], done;
  __shared__ uint32_t tmem_s;
  __shared__ int abort_s;
  unsigned char* ring = raw_smem + ((1024 - (saddr(raw_smem) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = split > 1 ? (int)cluster_rank() : 0;
  const int row0 = (int)(blockIdx.x / split) * kBM;
  const int blocks = (s.K + kBK - 1) / kBK;
  const int b0 = (int)((int64_t)blocks * rank / split), b1 = (int)((int64_t)blocks * (rank + 1) / split);
  auto load = [&](int i) {                // stage of block b0 + i, by one thread
    unsigned char* dst = ring + i % ST * SB;
    bar_expect(&full[i % ST], SB);
    for (int part = 0; part < PARTS; ++part) {
      tma_2d(dst + part * WB, &wmap, &full[i % ST], (b0 + i) * kBK, part * s.N + row0);
      tma_2d(dst + PARTS * WB + part * XB, &xmap, &full[i % ST], (b0 + i) * kBK, part * s.n);
    }
  };
  const int ahead = min(ST, b1 - b0);     // the first copies go out before the other warps are ready
  if (warp == 0) {
    if (elect_one()) {
      tma_prefetch(&xmap);
      tma_prefetch(&wmap);
      for (int i = 0; i < ST; ++i) {
        bar_init(&full[i], 1);
        bar_init(&empty[i], 1);
      }
      bar_init(&done, 1);
      abort_s = 0;
      bar_init_fence();
      fence_async();                      // the copies signal these barriers without a sync in between
      pdl_wait_primary();
      for (int i = 0; i < ahead; ++i) load(i);
    }
    __syncwarp();
  } else if (warp == 1) {
    tmem_alloc(&tmem_s, cols);
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
  constexpr int CAP = few_accs<NT, PARTS>();
  const int total = b1 - b0, rounds = PARTS == 3 ? (total + CAP - 1) / CAP : 1;
  const uint32_t at = tmem + ((uint32_t)(32 * warp) << 16);
  [[maybe_unused]] float sums[PARTS == 3 ? NT : 1];        // of the rounds
#pragma unroll
  for (float& x : sums) x = 0.f;
  bool alive = true;
  int i = warp == 0 ? ahead : 0;
  for (int round = 0; round < rounds; ++round) {
    const int end = min(total, (PARTS == 3 ? round + 1 : 1) * CAP);
    if (warp == 0) {
      const bool issuer = elect_one();
      for (; alive && i < min(total, end + ST); ++i) {       // what a later round takes is on its way
        alive = warp_wait(&empty[i % ST], (i / ST - 1) & 1, wait_limit, abort_flag);
        if (!alive) break;
        if (issuer) load(i);
        __syncwarp();
      }
      if (!alive && lane == 0) give_up();
      // no copy of this CTA may still be in flight when its memory is reused
      if (round == rounds - 1)
        for (int j = i > ST ? i - ST : 0; j < i; ++j) bar_wait(&full[j % ST], (j / ST) & 1, kDrainLimit);
    } else if (warp == 1) {
      const bool issuer = elect_one();
      constexpr uint32_t id = idesc(kBM, NT);
      for (; alive && i < end; ++i) {
        const int st = i % ST;
        alive = warp_wait(&full[st], (i / ST) & 1, wait_limit, abort_flag);
        if (!alive) break;
        fence_after();
        if (issuer) {
          const uint32_t wa = saddr(ring + st * SB), xa = wa + PARTS * WB;
          if constexpr (PARTS == 1) {
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k) mma(tmem, desc_k(wa + 32 * k), desc_k(xa + 32 * k), id, i > 0 || k > 0);
          } else {
            constexpr int pw[6] = {2, 0, 1, 1, 0, 0}, px[6] = {0, 2, 1, 0, 1, 0};   // smallest first
            const uint32_t d = tmem + i % CAP * NT;
#pragma unroll
            for (int p = 0; p < 6; ++p)
#pragma unroll
              for (int k = 0; k < kBK / 16; ++k)
                mma(d, desc_k(wa + pw[p] * WB + 32 * k), desc_k(xa + px[p] * XB + 32 * k), id, p > 0 || k > 0);
          }
          commit(&empty[st]);
        }
        __syncwarp();
      }
      if (!alive && lane == 0) give_up();
      if (issuer) commit(&done);
      __syncwarp();
    }
    // all MMAs of the round (after the last: with them all copies) are done: shared memory is free
    const bool arrived = bar_wait(&done, round & 1, kDefaultWaitLimit);
    if (!arrived) give_up();
    __syncwarp();
    fence_after();
    __syncthreads();
    if constexpr (PARTS == 3) {
#pragma unroll
      for (int c = 0; c < NT; c += 16) {
        if (c >= s.n) break;
        for (int g = 0; g < end - round * CAP; ++g) {
          uint32_t r[16];
          tmem_ld16(at + g * NT + c, r);
          ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) sums[c + e] += __uint_as_float(r[e]);
        }
      }
      if (round < rounds - 1) {              // the next round's products take their place
        fence_before();
        __syncthreads();
        fence_after();
      }
    }
  }
  float* part = reinterpret_cast<float*>(ring);           // [NT][128]
#pragma unroll
  for (int c = 0; c < NT; c += 16) {
    if (c >= s.n) break;
    if constexpr (PARTS == 1) {
      uint32_t r[16];
      tmem_ld16(at + c, r);
      ld_wait();
#pragma unroll
      for (int e = 0; e < 16; ++e) part[(c + e) * kBM + tid] = __uint_as_float(r[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) part[(c + e) * kBM + tid] = sums[c + e];
    }
  }
  if (split > 1) cluster_sync();
  else __syncthreads();
  // Four rows of W and one row of x at a time; every CTA's sums are asked for
  // before the first is used (one at a time, 64 rows of 2048 -> 2048 took 9.1 us instead of 7.1).
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
        if (q < split) v[q] = split == 1 ? *reinterpret_cast<const float4*>(part + t * kBM + r) : ld_cluster4(cluster_addr(part + t * kBM + r, q));
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
      for (int e = 0; e < 4; ++e) u[e] = sizeof(T) == 2 ? linear_act_bf16<ACT>(u[e] + bv[e]) : linear_act<ACT>(u[e] + bv[e]);
      if (sizeof(T) == 2 && vec) {                         // N, the strides and the addresses allow it
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
  if (warp == 1) tmem_free(tmem, cols);
}

// At most kWarpRows rows of x, operands as they stand: a warp per RW rows of W, its
// lanes along the contraction, applied to all rows of x, which the CTA holds in
// shared memory in fp32, kRowsK columns at a time. RW = 2 halves the reads of x,
// which bound it from a few rows on (8 rows, 8192 -> 8192 fp32: 147 us with RW = 1).
constexpr int kRowsK = 1024;
template <typename T, int ACT, bool VEC, int RW>
__global__ void __launch_bounds__(256) k_linear_rows(LinShape s, const T* __restrict__ x, const T* __restrict__ w,
                                                    const T* __restrict__ bias, const T* residual, T* y) {
  __shared__ __align__(16) float xs[kWarpRows][kRowsK];
  pdl_wait_primary();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = (blockIdx.x * 8 + warp) * RW;
  const T* wr[RW];
#pragma unroll
  for (int r = 0; r < RW; ++r) wr[r] = w + (int64_t)min(c0 + r, s.N - 1) * s.ldw;
  float acc[RW][kWarpRows] = {};
  constexpr int E = VEC ? 16 / (int)sizeof(T) : 1;          // elements per load
  constexpr int U = VEC ? 4 / RW : 8 / RW;                  // loads of a row of W in flight
  for (int base = 0; base < s.K; base += kRowsK) {
    const int kn = min(kRowsK, s.K - base);
    __syncthreads();
    for (int t = 0; t < s.n; ++t)
      for (int k = threadIdx.x; k < kn; k += 256) xs[t][k] = op_load(x + t * s.ldx + base + k);
    __syncthreads();
    for (int k0 = lane * E; k0 < kn; k0 += 32 * E * U) {
      float wv[RW][U][E];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < RW; ++r) {
          const int k = k0 + u * 32 * E;
          if constexpr (VEC) {
            uint4 q = make_uint4(0, 0, 0, 0);
            if (k < kn) q = __ldcs(reinterpret_cast<const uint4*>(wr[r] + base + k));
            const uint32_t v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (sizeof(T) == 2) {
                wv[r][u][2 * e] = lo_f(v[e]);
                wv[r][u][2 * e + 1] = hi_f(v[e]);
              } else {
                wv[r][u][e] = __uint_as_float(v[e]);
              }
            }
          } else {
            wv[r][u][0] = k < kn ? op_load(wr[r] + base + k) : 0.f;
          }
        }
#pragma unroll
      for (int t = 0; t < kWarpRows; ++t) {
        if (t >= s.n) break;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = k0 + u * 32 * E;
          if (k >= kn) break;
          if constexpr (VEC) {
#pragma unroll
            for (int e = 0; e < E; e += 4) {
              const float4 f = *reinterpret_cast<const float4*>(&xs[t][k + e]);
#pragma unroll
              for (int r = 0; r < RW; ++r) {
                acc[r][t] = fmaf(wv[r][u][e], f.x, acc[r][t]);
                acc[r][t] = fmaf(wv[r][u][e + 1], f.y, acc[r][t]);
                acc[r][t] = fmaf(wv[r][u][e + 2], f.z, acc[r][t]);
                acc[r][t] = fmaf(wv[r][u][e + 3], f.w, acc[r][t]);
              }
            }
          } else {
            const float f = xs[t][k];
#pragma unroll
            for (int r = 0; r < RW; ++r) acc[r][t] = fmaf(wv[r][u][0], f, acc[r][t]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RW; ++r) {
    const int c = c0 + r;
    if (c >= s.N) return;
    float out = 0.f;
#pragma unroll
    for (int t = 0; t < kWarpRows; ++t) {
      if (t >= s.n) break;
      float v = acc[r][t];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == t) out = v;
    }
    if (lane < s.n) {
      const float in = out + (bias ? op_load(bias + c) : 0.f);
      float u = sizeof(T) == 2 ? linear_act_bf16<ACT>(in) : linear_act<ACT>(in);   // as the other forms have it
      if (residual) u += op_load(residual + lane * s.ldr + c);
      op_store(y + lane * s.ldy + c, u);
    }
  }
}

// CTAs that share the contraction of 128 rows of W: enough for two per SM.
int few_split(const LinShape& s, int num_sms) {
  const int tiles = (s.N + kBM - 1) / kBM, blocks = (s.K + kBK - 1) / kBK;
  int split = 1;
  while (split < 8 && 2 * split * tiles <= 2 * num_sms && 2 * split <= blocks) split *= 2;
  return split;
}

template <int NT, int PARTS, typename T, int ACT>
cudaError_t run_few(const LinCall& c) {
  const LinShape& s = c.s;
  constexpr auto kern = k_linear_few<NT, PARTS, T, ACT>;
  constexpr size_t smem = few_smem<NT, PARTS>();
  cudaError_t e = allow_smem<kern>(smem);
  if (e != cudaSuccess) return e;
  CUtensorMap xmap, wmap;
  if (!linear_map(&xmap, c.x, (int64_t)PARTS * s.n, s.K, s.ldx, NT) || !linear_map(&wmap, c.w, (int64_t)PARTS * s.N, s.K, s.ldw, kBM))
    return cudaErrorInvalidValue;
  const int split = few_split(s, c.num_sms), blocks = (s.K + kBK - 1) / kBK;
  const int own = (blocks + split - 1) / split;
  const int cols = PARTS == 3 ? NT * (own < few_accs<NT, PARTS>() ? own : few_accs<NT, PARTS>()) : NT;
  int alloc = 32;
  while (alloc < cols) alloc *= 2;
  const int vec = s.N % 4 == 0 && (uintptr_t)c.y % 8 == 0 && s.ldy % 4 == 0 &&
                  (!c.residual || ((uintptr_t)c.residual % 8 == 0 && s.ldr % 4 == 0));
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((s.N + kBM - 1) / kBM * split));
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, s, xmap, wmap, (const T*)c.bias, (const T*)c.residual, (T*)c.y, split, alloc, vec,
                            op_wait_limit());
}

template <int ACT>
cudaError_t run_few_nt(const LinCall& c) {
  using H = __nv_bfloat16;
  if (!c.s.bf16) {
    if (c.s.n <= 16) return run_few<16, 3, float, ACT>(c);
    if (c.s.n <= 32) return run_few<32, 3, float, ACT>(c);
    return run_few<64, 3, float, ACT>(c);
  }
  if (c.s.n <= 16) return run_few<16, 1, H, ACT>(c);
  if (c.s.n <= 32) return run_few<32, 1, H, ACT>(c);
  if (c.s.n <= 64) return run_few<64, 1, H, ACT>(c);
  return run_few<128, 1, H, ACT>(c);
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
  // two rows of W per warp where that still leaves every SM a few CTAs
  const int rw = s.n > 2 && s.N >= 16 * 2 * c.num_sms ? 2 : 1;
  cfg.gridDim = dim3((unsigned)((s.N + 8 * rw - 1) / (8 * rw)));
  cfg.blockDim = dim3(256);
  cfg.stream = c.st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kern = rw == 2 ? (vec ? k_linear_rows<T, ACT, true, 2> : k_linear_rows<T, ACT, false, 2>)
                      : (vec ? k_linear_rows<T, ACT, true, 1> : k_linear_rows<T, ACT, false, 1>);
  return cudaLaunchKernelEx(&cfg, kern, s, (const T*)c.x, (const T*)c.w, (const T*)c.bias, (const T*)c.residual, (T*)c.y);
}

}  // namespace

bool linear_few_fits(const LinShape& s, int num_sms) {
  if (s.bf16) return s.n <= kFewRows;
  if (s.n > 64) return false;
  const int blocks = (s.K + kBK - 1) / kBK, split = few_split(s, num_sms), nt = s.n <= 16 ? 16 : s.n <= 32 ? 32 : 64;
  return (blocks + split - 1) / split <= kRounds * (512 / nt);
}

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
