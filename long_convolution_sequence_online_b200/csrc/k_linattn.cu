// Linear attention with one decay per head, S_t = g S_{t-1} + k_t v_t^T,
// o_t = scale q_t^T S_t: the chunked form for prompts in fp32 arithmetic, and
// the recurrent form for one position.
//
// Chunked form, positions i, j of a chunk of C and S the state before it:
//   o_i = scale [ sum_{j <= i} g^{i-j} (q_i . k_j) v_j + g^{i+1} q_i^T S ]
//   S  <- g^C S + sum_j g^{C-1-j} k_j v_j^T.
// Every power of g has an exponent >= 0, so nothing overflows whatever the decay.
//
// The chunked form here takes the shapes whose tiles do not fit the tensor cores' kernel
// (k_linattn_tc.cu): bf16 above 128 dimensions. Bound by shared-memory reads of its 4 x 4
// outer products with one CTA per SM: 4 x 2048 positions, 8 heads of 256 1.5 ms (12 TFLOP/s).
#include "op_internal.cuh"

namespace fi {

namespace {

constexpr int kC = 64;           // positions per chunk
constexpr int kSlice = 64;       // value columns per CTA
constexpr int kLaThreads = 256;  // 16 x 16: 4 x 4 of every 64 x 64 product per thread

// DKP: key_dim padded to 64, 128 or 256 (zeros). Shared memory, fp32: Q [C][DKP],
// K [C][DKP + 4], V [C][kSlice], P [C][C + 4], S [DKP][kSlice], and the powers of g.
template <int DKP>
constexpr size_t la_smem() {
  return sizeof(float) * ((size_t)kC * (2 * DKP + 4) + kC * kSlice + kC * (kC + 4) + (size_t)DKP * kSlice + kC + 4);
}

__device__ __forceinline__ float dot4(const float4& a, const float4& b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}
__device__ __forceinline__ void axpy4(float a, const float4& x, float (&y)[4]) {
  y[0] = fmaf(a, x.x, y[0]);
  y[1] = fmaf(a, x.y, y[1]);
  y[2] = fmaf(a, x.z, y[2]);
  y[3] = fmaf(a, x.w, y[3]);
}

// Segment blockIdx.z of (sequence, head) blockIdx.x, value columns
// [kSlice blockIdx.y, + kSlice). OUT = false: the segment's own contribution
// to the state into slot segment + 1 (segment 0 also copies the state before
// the prompt into slot 0). OUT = true: the outputs, and the state after the
// last position.
template <int DKP, bool OUT>
__global__ void __launch_bounds__(kLaThreads) k_linattn(LaShape s, LaPlan p, LaPtrs a) {
  using T = __nv_bfloat16;
  extern __shared__ __align__(16) float sm[];
  float* Q = sm;                           // [C][DKP]
  float* K = Q + kC * DKP;                 // [C][DKP+4]
  float* V = K + kC * (DKP + 4);           // [C][kSlice]
  float* P = V + kC * kSlice;              // [C][C+4]
  float* S = P + kC * (kC + 4);            // [DKP][kSlice]
  float* G = S + DKP * kSlice;             // g^0 .. g^C
  constexpr int LD = DKP + 4, LP = kC + 4, R = DKP / 64;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int bh = blockIdx.x, b = bh / s.H, h = bh - b * s.H;
  const int c0 = blockIdx.y * kSlice, nc = min(kSlice, s.dv - c0);
  const int seg = blockIdx.z;
  const int len = la_length(a.lengths, b, s.n);
  const int64_t t0 = (int64_t)seg * p.seg;
  const size_t slot = (size_t)s.dk * s.dv;
  float* ws = a.ws ? a.ws + (size_t)bh * p.G * slot + c0 : nullptr;
  const float* s_in = a.state_in ? a.state_in + (size_t)bh * slot + c0 : nullptr;
  float* s_out = a.state_out ? a.state_out + (size_t)bh * slot + c0 : nullptr;
  if constexpr (!OUT) {
    if (seg == 0 && s_in)
      for (int e = tid; e < s.dk * nc; e += kLaThreads) {
        const int d = e / nc, c = e - d * nc;
        ws[(size_t)d * s.dv + c] = s_in[(size_t)d * s.dv + c];
      }
    if (t0 + p.seg >= len) return;         // no segment after this one
  } else {
    if (t0 >= len && seg > 0) return;
  }
  const int end = (int)min((int64_t)len, t0 + p.seg);
  const float ld2 = la_log2_decay(__ldg(a.log_decay + h));
  for (int e = tid; e <= kC; e += kLaThreads) G[e] = la_pow(ld2, e);
  // The state's rows 64 r + 4 ty + i, columns 4 tx + j, in registers.
  float st[R][4][4] = {};
  if constexpr (OUT) {
    const float* src = p.G > 1 ? ws : s_in;
    for (int g = 0; g <= seg && src; ++g) {
      // slot 0: the state before the prompt; slot g: segment g - 1's contribution
      if (g == 0 && (!s_in || (la_drops(ld2) && len > 0))) continue;
      const float f = la_pow(ld2, (g == 0 ? seg : seg - g) * p.seg);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int d = 64 * r + 4 * ty + i;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (d < s.dk && 4 * tx + j < nc)
              st[r][i][j] = fmaf(f, src[(size_t)g * slot + (size_t)d * s.dv + 4 * tx + j], st[r][i][j]);
        }
    }
  }
  const T* qp = (const T*)a.q + b * s.qs[1] + h * s.qs[2];
  const T* kp = (const T*)a.k + b * s.ks[1] + h * s.ks[2];
  const T* vp = (const T*)a.v + b * s.vs[1] + h * s.vs[2] + c0;
  T* op = (T*)a.o + b * s.os[1] + h * s.os[2] + c0;
  for (int64_t t = t0; t < end; t += kC) {
    const int m = (int)min((int64_t)kC, end - t);
    __syncthreads();
    for (int e = tid; e < kC * DKP; e += kLaThreads) {
      const int i = e / DKP, d = e & (DKP - 1);
      const bool in = i < m && d < s.dk;
      if constexpr (OUT) Q[i * DKP + d] = in ? op_load(qp + (t + i) * s.qs[0] + d) : 0.f;
      K[i * LD + d] = in ? op_load(kp + (t + i) * s.ks[0] + d) : 0.f;
    }
    for (int e = tid; e < kC * kSlice; e += kLaThreads) {
      const int i = e / kSlice, c = e & (kSlice - 1);
      V[e] = i < m && c < nc ? op_load(vp + (t + i) * s.vs[0] + c) : 0.f;
    }
    if constexpr (OUT) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(S + (64 * r + 4 * ty + i) * kSlice + 4 * tx) =
              make_float4(st[r][i][0], st[r][i][1], st[r][i][2], st[r][i][3]);
    }
    __syncthreads();
    if constexpr (OUT) {
      // scores: rows ty + 16 a, columns tx + 16 b
      float acc[4][4] = {};
      for (int d = 0; d < DKP; d += 4) {
        float4 qv[4], kv[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          qv[u] = *reinterpret_cast<const float4*>(Q + (ty + 16 * u) * DKP + d);
          kv[u] = *reinterpret_cast<const float4*>(K + (tx + 16 * u) * LD + d);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = dot4(qv[i], kv[j], acc[i][j]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int ri = ty + 16 * i, cj = tx + 16 * j;
          P[ri * LP + cj] = cj <= ri ? acc[i][j] * G[ri - cj] : 0.f;
        }
      __syncthreads();
      // rows 4 ty + i: g^{row+1} q^T S, then the scores' product
      float o[4][4] = {};
      for (int d = 0; d < DKP; d += 4) {
        float4 sv[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) sv[u] = *reinterpret_cast<const float4*>(S + (d + u) * kSlice + 4 * tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 qv = *reinterpret_cast<const float4*>(Q + (4 * ty + i) * DKP + d);
          axpy4(qv.x, sv[0], o[i]);
          axpy4(qv.y, sv[1], o[i]);
          axpy4(qv.z, sv[2], o[i]);
          axpy4(qv.w, sv[3], o[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] *= G[4 * ty + i + 1];
      for (int jj = 0; jj < kC; jj += 4) {
        float4 vv[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) vv[u] = *reinterpret_cast<const float4*>(V + (jj + u) * kSlice + 4 * tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 pv = *reinterpret_cast<const float4*>(P + (4 * ty + i) * LP + jj);
          axpy4(pv.x, vv[0], o[i]);
          axpy4(pv.y, vv[1], o[i]);
          axpy4(pv.z, vv[2], o[i]);
          axpy4(pv.w, vv[3], o[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ri = 4 * ty + i;
        if (ri >= m) break;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (4 * tx + j < nc) op_store(op + (t + ri) * s.os[0] + 4 * tx + j, s.scale * o[i][j]);
      }
    }
    // S <- g^m S + sum_j g^{m-1-j} k_j v_j^T
    const float gm = G[m];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) st[r][i][j] *= gm;
    for (int j = 0; j < m; ++j) {
      const float w = G[m - 1 - j];
      float4 v4 = *reinterpret_cast<const float4*>(V + j * kSlice + 4 * tx);
      v4.x *= w; v4.y *= w; v4.z *= w; v4.w *= w;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 k4 = *reinterpret_cast<const float4*>(K + j * LD + 64 * r + 4 * ty);
        axpy4(k4.x, v4, st[r][0]);
        axpy4(k4.y, v4, st[r][1]);
        axpy4(k4.z, v4, st[r][2]);
        axpy4(k4.w, v4, st[r][3]);
      }
    }
  }
  float* dst = nullptr;
  if constexpr (!OUT) dst = ws + (size_t)(seg + 1) * slot;
  else if (s_out && end == len) dst = s_out;   // this segment holds the last position
  if (!dst) return;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = 64 * r + 4 * ty + i;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (d < s.dk && 4 * tx + j < nc) dst[(size_t)d * s.dv + 4 * tx + j] = st[r][i][j];
    }
}

// One position. A CTA owns kStepCols columns of one (sequence, head)'s state;
// its eight warps take the rows in turn (a lane: V consecutive columns) and
// add up their parts of q^T S at the end.
// Bound by the state, read and written once: 64 sequences x 16 heads of 128, 134 MB in
// 23 us (5.9 TB/s, 0.90 of a copy); one sequence is a launch, 2.2 us. Three CTAs per SM, which
// 80 registers allow, are needed for it (37 x 9 heads of 56 x 104: 3.6 us, with two 4.5).
template <typename T, int V>
__global__ void __launch_bounds__(256, 3) k_linattn_step(LaShape s, const T* __restrict__ q, const T* __restrict__ k,
                                                     const T* __restrict__ v, const float* __restrict__ log_decay,
                                                     float* __restrict__ state, T* __restrict__ o) {
  using vec = typename std::conditional<V == 4, float4, typename std::conditional<V == 2, float2, float>::type>::type;
  __shared__ float qs[256], ks[256];
  __shared__ float part[8][32 * V];
  pdl_wait_primary();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = blockIdx.x, b = bh / s.H, h = bh - b * s.H;
  const int c = (blockIdx.y * 32 + lane) * V;
  const bool in = c < s.dv;
  const float ld2 = la_log2_decay(__ldg(log_decay + h)), g = la_pow(ld2, 1);
  const uint32_t keep = la_drops(ld2) ? 0u : ~0u;    // of the state before
  if (tid < s.dk) {
    qs[tid] = op_load(q + b * s.qs[1] + h * s.qs[2] + tid);
    ks[tid] = op_load(k + b * s.ks[1] + h * s.ks[2] + tid);
  }
  float vv[V], acc[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    vv[e] = in ? op_load(v + b * s.vs[1] + h * s.vs[2] + c + e) : 0.f;
    acc[e] = 0.f;
  }
  __syncthreads();
  float* sp = state + (size_t)bh * s.dk * s.dv + c;
  if (in) {
    // eight rows' loads before the first is used, past the caches' order: the state
    // is read and written once
    for (int d0 = warp; d0 < s.dk; d0 += 64) {
      vec x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (d0 + 8 * u < s.dk) x[u] = __ldcs(reinterpret_cast<const vec*>(sp + (size_t)(d0 + 8 * u) * s.dv));
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int d = d0 + 8 * u;
        if (d >= s.dk) break;
        float f[V];
        *reinterpret_cast<vec*>(f) = x[u];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          f[e] = fmaf(ks[d], vv[e], g * __uint_as_float(__float_as_uint(f[e]) & keep));
          acc[e] = fmaf(qs[d], f[e], acc[e]);
        }
        __stcs(reinterpret_cast<vec*>(sp + (size_t)d * s.dv), *reinterpret_cast<const vec*>(f));
      }
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) part[warp][lane * V + e] = acc[e];
  __syncthreads();
  const int cc = blockIdx.y * 32 * V + tid;
  if (tid < 32 * V && cc < s.dv) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) sum += part[w][tid];
    op_store(o + b * s.os[1] + h * s.os[2] + cc, s.scale * sum);
  }
}

template <int DKP>
cudaError_t prefill(const LaShape& s, const LaPlan& p, const LaPtrs& a, cudaStream_t st) {
  cudaError_t e;
  const dim3 grid((unsigned)(s.B * s.H), (unsigned)((s.dv + kSlice - 1) / kSlice), (unsigned)p.G);
  if (p.G > 1) {
    if ((e = allow_smem<k_linattn<DKP, false>>(la_smem<DKP>())) != cudaSuccess) return e;
    k_linattn<DKP, false><<<grid, kLaThreads, la_smem<DKP>(), st>>>(s, p, a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if ((e = allow_smem<k_linattn<DKP, true>>(la_smem<DKP>())) != cudaSuccess) return e;
  k_linattn<DKP, true><<<grid, kLaThreads, la_smem<DKP>(), st>>>(s, p, a);
  return cudaGetLastError();
}

cudaError_t prefill_dk(const LaShape& s, const LaPlan& p, const LaPtrs& a, cudaStream_t st) {
  if (s.dk <= 64) return prefill<64>(s, p, a, st);
  if (s.dk <= 128) return prefill<128>(s, p, a, st);
  return prefill<256>(s, p, a, st);
}

template <typename T, int V>
cudaError_t step(const LaShape& s, const void* q, const void* k, const void* v, const float* log_decay, float* state,
                 void* o, cudaStream_t st) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(s.B * s.H), (unsigned)((s.dv + 32 * V - 1) / (32 * V)));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_linattn_step<T, V>, s, (const T*)q, (const T*)k, (const T*)v, log_decay, state, (T*)o);
}

template <typename T>
cudaError_t step_vec(const LaShape& s, const void* q, const void* k, const void* v, const float* log_decay,
                     float* state, void* o, cudaStream_t st) {
  const uintptr_t at = (uintptr_t)state;
  if (s.dv % 4 == 0 && at % 16 == 0) return step<T, 4>(s, q, k, v, log_decay, state, o, st);
  if (s.dv % 2 == 0 && at % 8 == 0) return step<T, 2>(s, q, k, v, log_decay, state, o, st);
  return step<T, 1>(s, q, k, v, log_decay, state, o, st);
}

}  // namespace

// Enough segments that two CTAs per SM run, each of at least four chunks.
static LaPlan la_plan(const LaShape& s, int num_sms) {
  const int64_t per = (int64_t)s.B * s.H * ((s.dv + kSlice - 1) / kSlice);
  const int64_t chunks = ((int64_t)s.n + kC - 1) / kC;
  int64_t G = (2 * (int64_t)num_sms) / per;
  if (G > chunks / 4) G = chunks / 4;
  if (G > 64) G = 64;
  if (G < 2) return LaPlan{1, (int)(chunks > 0 ? chunks * kC : kC)};
  const int64_t c = (chunks + G - 1) / G;
  return LaPlan{(int)((chunks + c - 1) / c), (int)(c * kC)};
}

size_t linattn_prefill_workspace(const LaShape& s, const LaPtrs& a, int num_sms) {
  if (s.n == 0) return 0;
  if (!linattn_tc_fits(s)) return la_workspace_bytes(s, la_plan(s, num_sms));
  const LaShape b = linattn_tc_block(s);
  return la_workspace_bytes(b, linattn_tc_plan(b, num_sms)) + linattn_tc_layout_bytes(s, a);
}

cudaError_t launch_linattn_prefill(const LaShape& s, const LaPtrs& ptrs, void* workspace, int num_sms, cudaStream_t st) {
  LaPtrs a = ptrs;
  if (s.n == 0) {                          // the state before is the state after
    const size_t bytes = (size_t)s.B * s.H * s.dk * s.dv * sizeof(float);
    if (!a.state_out || a.state_out == a.state_in) return cudaSuccess;
    return a.state_in ? cudaMemcpyAsync(a.state_out, a.state_in, bytes, cudaMemcpyDeviceToDevice, st)
                      : cudaMemsetAsync(a.state_out, 0, bytes, st);
  }
  a.ws = (float*)workspace;
  if (linattn_tc_fits(s)) {
    const LaShape b = linattn_tc_block(s);
    const LaPlan p = linattn_tc_plan(b, num_sms);
    return launch_linattn_tc(s, p, a, (unsigned char*)workspace + la_workspace_bytes(b, p), num_sms, st);
  }
  return prefill_dk(s, la_plan(s, num_sms), a, st);
}

cudaError_t launch_linattn_step(const LaShape& s, const void* q, const void* k, const void* v, const float* log_decay,
                                float* state, void* o, cudaStream_t st) {
  return s.bf16 ? step_vec<__nv_bfloat16>(s, q, k, v, log_decay, state, o, st)
                : step_vec<float>(s, q, k, v, log_decay, state, o, st);
}

}  // namespace fi
