// Linear layer y = R(act(x W^T + bias) + residual).
#include "op_internal.cuh"

namespace fi {

namespace {

// 64 x 64 outputs per CTA, 4 x 4 per thread, fp32 products.
constexpr int kLinTile = 64, kLinK = 16;

template <typename T, int ACT>
__global__ void __launch_bounds__(256) k_linear(LinShape s, const T* __restrict__ x, const T* __restrict__ w,
                                               const T* __restrict__ bias, const T* residual, T* y) {
  __shared__ float xs[kLinK][kLinTile + 4], ws[kLinK][kLinTile + 4];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int64_t r0 = (int64_t)blockIdx.x * kLinTile, c0 = (int64_t)blockIdx.y * kLinTile;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < s.K; k0 += kLinK) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = tid + i * 256, k = e & (kLinK - 1), r = e >> 4;
      const bool in = k0 + k < s.K;
      xs[k][r] = in && r0 + r < s.n ? op_load(x + (r0 + r) * s.ldx + k0 + k) : 0.f;
      ws[k][r] = in && c0 + r < s.N ? op_load(w + (c0 + r) * s.ldw + k0 + k) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kLinK; ++k) {
      const float4 a = *reinterpret_cast<const float4*>(&xs[k][4 * ty]);
      const float4 b = *reinterpret_cast<const float4*>(&ws[k][4 * tx]);
      const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + 4 * ty + i;
    if (r >= s.n) break;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = c0 + 4 * tx + j;
      if (c >= s.N) break;
      float u = linear_act<ACT>(acc[i][j] + (bias ? op_load(bias + c) : 0.f));
      if (residual) u += op_load(residual + r * s.ldr + c);
      op_store(y + r * s.ldy + c, u);
    }
  }
}

template <typename T, int ACT>
cudaError_t run(const LinShape& s, const void* x, const void* w, const void* bias, const void* residual, void* y,
                cudaStream_t st) {
  const dim3 grid((unsigned)((s.n + (int64_t)kLinTile - 1) / kLinTile), (unsigned)((s.N + kLinTile - 1) / kLinTile));
  k_linear<T, ACT><<<grid, 256, 0, st>>>(s, (const T*)x, (const T*)w, (const T*)bias, (const T*)residual, (T*)y);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run_act(const LinShape& s, const void* x, const void* w, const void* bias, const void* residual, void* y,
                    cudaStream_t st) {
  switch (s.act) {
    case FI_ACT_NONE: return run<T, FI_ACT_NONE>(s, x, w, bias, residual, y, st);
    case FI_ACT_GELU: return run<T, FI_ACT_GELU>(s, x, w, bias, residual, y, st);
    case FI_ACT_SILU: return run<T, FI_ACT_SILU>(s, x, w, bias, residual, y, st);
    case FI_ACT_RELU: return run<T, FI_ACT_RELU>(s, x, w, bias, residual, y, st);
    case FI_ACT_TANH: return run<T, FI_ACT_TANH>(s, x, w, bias, residual, y, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_linear(const LinShape& s, const void* x, const void* w, const void* bias, const void* residual,
                          void* y, int num_sms, cudaStream_t st) {
  (void)num_sms;
  return s.bf16 ? run_act<__nv_bfloat16>(s, x, w, bias, residual, y, st) : run_act<float>(s, x, w, bias, residual, y, st);
}

}  // namespace fi
