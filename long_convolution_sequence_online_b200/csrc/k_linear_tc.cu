// Linear layer y = R(act(x W^T + bias) + residual) on the 5th-generation tensor
// cores (tcgen05, accumulators in tensor memory).
//
// A persistent pair of CTAs on neighbouring SMs walks over output tiles of 256
// rows x BN columns; each MMA works for both (cta_group::2): a CTA holds its 128
// rows of x and half of the W tile, which halves the W traffic from L2 and shared
// memory. The contraction runs in blocks of 64: x and W tiles as K-major operands
// of 128-byte rows in shared memory with the 128-byte swizzle, a ring of stages
// between the producers and the one thread that issues the MMAs. Accumulators
// are double buffered in tensor memory, so eight epilogue warps apply bias,
// activation and residual to one tile while the next is multiplied.
//
// Operands come by TMA, which wants bf16 rows that start at 16-byte boundaries.
// Others are laid out so first, by a launch of their own into scratch (on chip,
// loader warps that read and converted tiles for the MMAs took 3300 cycles per
// block of 64 where the MMAs take 264 and, fp32, 1584: two warps per scheduler do
// not hide their own instructions' latency).
//
// fp32 values are laid out as three bf16 parts each, v = v0 + v1 + v2 (8 + 8 + 8
// bits), and the products x0w0 + x0w1 + x1w0 + x1w1 + x0w2 + x2w0 are added up (the
// rest is below 2^-24). The tensor core does not round its sums to nearest: left
// in one accumulator, such products at a contraction of 2048 were 1.4e-5 off in
// the 2-norm; with two blocks of 64 to an accumulator (smallest products of a block
// first), added up in the epilogue warps' registers, they are 7e-7 off, cuBLAS's fp32
// product 8e-7.
#include "op_internal.cuh"
#include "tc.cuh"

namespace fi {

namespace {

using namespace tc;

constexpr int kBM = 128, kBK = 64;
constexpr int kEpiWarps = 8;
// Warps of a CTA: 0-7 epilogue, 8 the MMA issuer, 9 TMA.
constexpr int kLinThreads = 32 * (kEpiWarps + 2);

__device__ int g_linear_error;   // a bounded wait gave up since the last check

// fp32: blocks that share an accumulator before the epilogue warps add them up.
constexpr int kSumBlocks = 2;
// Stage of the ring: `units` x (x tile 128 x 128 bytes, half of a W tile BN / 2 x
// 128 bytes). The units are the parts of fp32 values, or two blocks of the
// contraction: a stage's waits and signals take 350 to 450 cycles whatever its
// size, more than the 264 that the MMAs of one block take at BN = 128.
template <int PARTS>
constexpr int kStageBlocks = PARTS == 3 ? 1 : 2;
template <int BN, int PARTS>
constexpr int stage_bytes() { return PARTS * kStageBlocks<PARTS> * (kBM + BN / 2) * 128; }
// VEC kernels need no staging and have room for more: fp32 3 stages instead of 2.
template <int BN, int PARTS, bool VEC>
constexpr int num_stages() { return (VEC ? 229376 : 196608) / stage_bytes<BN, PARTS>(); }
constexpr int kStagingCols = 16, kStagingLd = kStagingCols + 1;
constexpr int kStagingBytes = kEpiWarps * 32 * kStagingLd * 4;
template <int BN, int PARTS, bool VEC>
constexpr size_t smem_bytes() {
  return 1024 + (size_t)num_stages<BN, PARTS, VEC>() * stage_bytes<BN, PARTS>() + (VEC ? 0 : kStagingBytes);
}
template <int BN>
constexpr uint32_t acc_cols() { return BN <= 128 ? 256 : 512; }   // two accumulators

struct LinTiles {
  int mt, nt, group;   // row tiles, column tiles, row tiles per group
  int tiles;           // fewer than 2^31: y has at most 2^40 elements
};

// Tile order: groups of `group` row tiles, down the group's rows, then the next
// column, so that the tiles at work together share rows and columns in L2.
__device__ __forceinline__ void tile_at(const LinTiles& g, int t, int& m, int& n) {
  const int per = g.group * g.nt, gi = t / per, r = t - gi * per;
  const int rows = min(g.group, g.mt - gi * g.group);
  n = r / rows;
  m = gi * g.group + r - n * rows;
}

template <typename T, int ACT>
__device__ __forceinline__ float activate(float u) {
  if constexpr (sizeof(T) == 2) return linear_act_bf16<ACT>(u);
  else return linear_act<ACT>(u);
}

// act(acc + bias) + residual of 32 columns of a row per lane, to y: the lane
// finishes and stores its row's columns, 16 bytes at a time.
template <typename T, int ACT>
__device__ __forceinline__ void store_vec(const LinShape& s, float (&v)[32], const T* bias, const T* residual, T* y,
                                          int64_t row, int c0) {
  constexpr int E = 16 / sizeof(T);
  auto add = [&](const uint4& b, int u) {
    const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (sizeof(T) == 2) {
        v[u * 8 + 2 * e] += lo_f(w[e]);
        v[u * 8 + 2 * e + 1] += hi_f(w[e]);
      } else {
        v[u * 4 + e] += __uint_as_float(w[e]);
      }
    }
  };
  if (bias) {
#pragma unroll
    for (int u = 0; u < 32 / E; ++u) add(__ldg(reinterpret_cast<const uint4*>(bias + c0) + u), u);
  }
#pragma unroll
  for (int e = 0; e < 32; ++e) v[e] = activate<T, ACT>(v[e]);
  if (row >= s.n) return;
  if (residual) {
    const T* rp = residual + row * s.ldr + c0;
#pragma unroll
    for (int u = 0; u < 32 / E; ++u) add(*(reinterpret_cast<const uint4*>(rp) + u), u);
  }
  T* yp = y + row * s.ldy + c0;
#pragma unroll
  for (int u = 0; u < 32 / E; ++u) {
    uint4 o;
    if constexpr (sizeof(T) == 2)
      o = make_uint4(pack2(v[u * 8], v[u * 8 + 1]), pack2(v[u * 8 + 2], v[u * 8 + 3]),
                     pack2(v[u * 8 + 4], v[u * 8 + 5]), pack2(v[u * 8 + 6], v[u * 8 + 7]));
    else
      o = make_uint4(__float_as_uint(v[u * 4]), __float_as_uint(v[u * 4 + 1]), __float_as_uint(v[u * 4 + 2]),
                     __float_as_uint(v[u * 4 + 3]));
    *(reinterpret_cast<uint4*>(yp) + u) = o;
  }
}

// The same where columns end inside the chunk or rows start at no 16-byte boundary:
// the sums pass through shared memory and a lane finishes a column's rows (column
// c0 + lane % 16 or + 16, rows lane / 16, + 2, ...), so that loads and stores run
// along the columns.
template <typename T, int ACT>
__device__ __forceinline__ void store_apart(const LinShape& s, const float (&v)[32], const T* bias, const T* residual, T* y,
                                            int64_t row0, int c0, float* stg, int lane) {
  const int rows = (int)min((int64_t)32, s.n - row0), cl = lane & 15, r0 = lane >> 4;
  float res[2][16], bv[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {            // everything that comes from memory first
    const int c = c0 + 16 * h + cl;
    bv[h] = bias && c < s.N ? op_load(bias + c) : 0.f;
    const T* rp = residual + (row0 + r0) * s.ldr + c;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      res[h][r] = residual && c < s.N && r0 + 2 * r < rows ? op_load(rp) : 0.f;
      rp += 2 * s.ldr;
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int e = 0; e < kStagingCols; ++e) stg[lane * kStagingLd + e] = v[16 * h + e];
    const int c = c0 + 16 * h + cl;
    T* yp = y + (row0 + r0) * s.ldy + c;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      if (c < s.N && r0 + 2 * r < rows) op_store(yp, activate<T, ACT>(stg[(r0 + 2 * r) * kStagingLd + cl] + bv[h]) + res[h][r]);
      yp += 2 * s.ldy;
    }
    __syncwarp();
  }
}

// BN: columns of a tile. PARTS: 1 (bf16) or 3 (fp32; part p of a matrix is its rows
// p n .. (p + 1) n). VEC: rows of y, bias and residual at 16-byte boundaries and
// whole chunks of 32 columns only. An epilogue warp drains tensor-memory lanes 32 (w % 4) .. + 31,
// column half w / 4.
template <int BN, int PARTS, bool VEC, typename T, int ACT>
__global__ void __launch_bounds__(kLinThreads, 1)
k_linear_tc(LinShape s, LinTiles g, const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
            const T* __restrict__ bias, const T* residual, T* y,
            int wait_limit) {
  constexpr int BW = BN / 2;                       // W rows in this CTA's stages
  constexpr int KS = kStageBlocks<PARTS>, UNITS = PARTS * KS;
  constexpr int ST = num_stages<BN, PARTS, VEC>(), SB = stage_bytes<BN, PARTS>();
  constexpr int XB = kBM * 128, WB = BW * 128;
  constexpr int TM = 2 * kBM;                      // rows of a tile
  extern __shared__ unsigned char raw_smem[];
  __shared__ uint64_t full_bar[ST], empty_bar[ST], acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_s;
  __shared__ int abort_s;
  unsigned char* ring = raw_smem + ((1024 - (saddr(raw_smem) & 1023)) & 1023);
  float* staging = reinterpret_cast<float*>(ring + (size_t)ST * SB);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &abort_s;
  const int rank = (int)cluster_rank();
  const int first = blockIdx.x >> 1, stride = gridDim.x >> 1;
  if (warp == 0) tmem_alloc2(&tmem_s, acc_cols<BN>());
  if (tid == 32) {
    for (int i = 0; i < ST; ++i) {
      bar_init(&full_bar[i], 1);
      bar_init(&empty_bar[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&acc_full[i], 1);
      bar_init(&acc_empty[i], 2 * kEpiWarps);
    }
    abort_s = 0;
    bar_init_fence();
  }
  fence_before();
  cluster_sync();
  fence_after();
  pdl_wait_primary();                              // from here on inputs are read and y is written
  const uint32_t tmem = tmem_s;
  const int nk = (s.K + KS * kBK - 1) / (KS * kBK);   // stages per tile
  auto give_up = [&]() {
    *abort_flag = 1;
    atomicExch(&g_linear_error, 1);
  };

  if (warp < kEpiWarps) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, half = warp >> 2;
    constexpr int CW = BN / 2;                     // columns of this warp
    float* stg = staging + warp * 32 * kStagingLd;
    uint32_t unit = 0;                             // accumulators drained
    bool alive = true;
    for (int t = first; t < g.tiles && alive; t += stride) {
      int m, n;
      tile_at(g, t, m, n);
      const int64_t row0 = (int64_t)m * TM + rank * kBM + 32 * q;
      const int col0 = n * BN + half * CW;
      const uint32_t at = tmem + ((uint32_t)(32 * q) << 16) + half * CW;
      // the tile's residual on its way into L2 while the tile is multiplied: a lane per row
      if (residual && row0 + lane < s.n) {
        const char* rp = reinterpret_cast<const char*>(residual + (row0 + lane) * s.ldr + col0);
        const int bytes = min(CW, s.N - col0) * (int)sizeof(T);
        for (int o = 0; o < bytes; o += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(rp + o));
      }
      auto store = [&](float (&v)[32], int c) {
        if (row0 >= s.n || col0 + c >= s.N) return;
        if constexpr (VEC) store_vec<T, ACT>(s, v, bias, residual, y, row0 + lane, col0 + c);
        else store_apart<T, ACT>(s, v, bias, residual, y, row0, col0 + c, stg, lane);
      };
      if constexpr (PARTS == 1) {
        alive = warp_wait(&acc_full[unit & 1], (unit >> 1) & 1, wait_limit, abort_flag);
        if (!alive) break;
        fence_after();
        auto load = [&](int c, float (&v)[32]) {
          uint32_t r[32];
          tmem_ld32(at + (unit & 1) * BN + c, r);
          ld_wait();
          if (c + 32 >= CW) {                      // all columns read: the MMA may overwrite them
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive_leader(&acc_empty[unit & 1]);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
        };
#pragma unroll 1                                   // straight-line code would be fetched once per launch
        for (int c = 0; c < CW; c += 32) {
          float v[32];
          load(c, v);
          store(v, c);
        }
        ++unit;
      } else {
        float acc[CW];
#pragma unroll
        for (int e = 0; e < CW; ++e) acc[e] = 0.f;
        for (int kb = 0; kb < nk; kb += kSumBlocks, ++unit) {
          alive = warp_wait(&acc_full[unit & 1], (unit >> 1) & 1, wait_limit, abort_flag);
          if (!alive) break;
          fence_after();
#pragma unroll
          for (int c = 0; c < CW; c += 16) {
            uint32_t r[16];
            tmem_ld16(at + (unit & 1) * BN + c, r);
            ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[c + e] += __uint_as_float(r[e]);
          }
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive_leader(&acc_empty[unit & 1]);
        }
        if (!alive) break;
#pragma unroll
        for (int c = 0; c < CW; c += 32) {
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = acc[c + e];
          store(v, c);
        }
      }
    }
    if (!alive && lane == 0) give_up();
  } else if (warp == kEpiWarps) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0) {
      constexpr uint32_t id = idesc(TM, BN);
      const bool issuer = elect_one();
      uint32_t kbs = 0, unit = 0;
      bool alive = true;
      for (int t = first; t < g.tiles && alive; t += stride) {
        for (int kb = 0; kb < nk; ++kb, ++kbs) {
          const int st = kbs % ST;
          if (PARTS > 1 ? kb % kSumBlocks == 0 : kb == 0)
            alive = unit < 2 || warp_wait(&acc_empty[unit & 1], ((unit >> 1) - 1) & 1, wait_limit, abort_flag);
          alive = alive && warp_wait(&full_bar[st], (kbs / ST) & 1, wait_limit, abort_flag);
          if (!alive) break;
          fence_after();
          const uint32_t xa = saddr(ring + (size_t)st * SB), wa = xa + UNITS * XB;
          const uint32_t d = tmem + (unit & 1) * BN;
          const bool last = kb == nk - 1 || (PARTS > 1 && kb % kSumBlocks == kSumBlocks - 1);
          if (issuer) {
            if constexpr (PARTS == 1) {
              const int steps = min(KS * kBK / 16, (s.K - kb * KS * kBK + 15) / 16);   // of 16
#pragma unroll
              for (int k = 0; k < KS * kBK / 16; ++k) {
                if (k >= steps) break;
                const uint32_t xo = (k / 4) * XB + (k % 4) * 32, wo = (k / 4) * WB + (k % 4) * 32;
                mma2(d, desc_k(xa + xo), desc_k(wa + wo), id, kb > 0 || k > 0);
              }
            } else {
              constexpr int px[6] = {2, 0, 1, 1, 0, 0}, pw[6] = {0, 2, 1, 0, 1, 0};   // smallest first
#pragma unroll
              for (int p = 0; p < 6; ++p)
#pragma unroll
                for (int k = 0; k < kBK / 16; ++k)
                  mma2(d, desc_k(xa + px[p] * XB + 32 * k), desc_k(wa + pw[p] * WB + 32 * k), id,
                       kb % kSumBlocks > 0 || p > 0 || k > 0);
            }
            commit2(&empty_bar[st]);
            if (last) commit2(&acc_full[unit & 1]);
          }
          __syncwarp();
          if (last) ++unit;
        }
      }
      if (!alive && lane == 0) give_up();
      // shared and tensor memory are released only once the last MMAs are done
      if (kbs > 0) bar_wait(&empty_bar[(kbs - 1) % ST], ((kbs - 1) / ST) & 1, kDrainLimit);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ TMA producer
    const bool issuer = elect_one();
    uint32_t kbs = 0;
    bool alive = true;
    for (int t = first; t < g.tiles && alive; t += stride) {
      int m, n;
      tile_at(g, t, m, n);
      for (int kb = 0; kb < nk; ++kb, ++kbs) {
        const int st = kbs % ST, k = kb * KS * kBK;
        alive = kbs < ST || warp_wait(&empty_bar[st], (kbs / ST - 1) & 1, wait_limit, abort_flag);
        if (!alive) break;
        if (issuer) {
          unsigned char* dst = ring + (size_t)st * SB;
          const int units = PARTS == 1 ? min(KS, (s.K - k + kBK - 1) / kBK) : PARTS;
          if (rank == 0) bar_expect(&full_bar[st], 2 * units * (XB + WB));   // both CTAs' tiles
#pragma unroll
          for (int u = 0; u < UNITS; ++u)
            if (u < units) {
              const int ku = PARTS == 1 ? k + u * kBK : k;
              tma_2d_pair(dst + u * XB, &xmap, &full_bar[st], ku, (PARTS == 1 ? 0 : u * s.n) + m * TM + rank * kBM);
              tma_2d_pair(dst + UNITS * XB + u * WB, &wmap, &full_bar[st], ku, (PARTS == 1 ? 0 : u * s.N) + n * BN + rank * BW);
            }
        }
        __syncwarp();
      }
    }
    if (!alive && lane == 0) give_up();
    // no copy of this CTA may still be in flight when it ends: each stage's last use is done
    for (uint32_t i = kbs > ST ? kbs - ST : 0; i < kbs; ++i) bar_wait(&empty_bar[i % ST], (i / ST) & 1, kDrainLimit);
  }
  fence_before();
  cluster_sync_relaxed();                          // neither CTA ends while the other may still signal it
  fence_after();
  if (warp == 0) tmem_free2(tmem, acc_cols<BN>());
}

// An operand that TMA cannot take (fp32, or rows at no 16-byte boundary) as
// `parts` bf16 matrices of rows of Kp = K rounded up to 8 elements, the rest zero:
// 8 elements per thread, read once, written once.
struct LinOperand {
  const void* src;
  __nv_bfloat16* dst;
  int64_t rows, ld;
  int vec;               // rows start at 16-byte boundaries
};
template <typename T>
__global__ void __launch_bounds__(256) k_linear_layout(LinOperand a, LinOperand b, int K, int Kp, int64_t units_a, int64_t units) {
  pdl_launch_dependents();                 // the product, which waits for this launch's end
  pdl_wait_primary();
  const int per = Kp / 8;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += (int64_t)gridDim.x * 256) {
    const bool first = u < units_a;
    const LinOperand& o = first ? a : b;
    const int64_t v = first ? u : u - units_a, row = v / per;
    const int k = (int)(v - row * per) * 8;
    const T* p = (const T*)o.src + row * o.ld + k;
    __nv_bfloat16* d = o.dst + row * Kp + k;
    if constexpr (sizeof(T) == 2) {
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k + e < K) w[e / 2] |= (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p) + e) << (16 * (e & 1));
      *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      float f[8];
      if (o.vec && k + 8 <= K) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(p)), y = __ldg(reinterpret_cast<const float4*>(p) + 1);
        f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
        f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = k + e < K ? __ldg(p + e) : 0.f;
      }
      uint32_t q[3][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split3(f[2 * e], f[2 * e + 1], q[0][e], q[1][e], q[2][e]);
#pragma unroll
      for (int i = 0; i < 3; ++i)
        *reinterpret_cast<uint4*>(d + i * o.rows * Kp) = make_uint4(q[i][0], q[i][1], q[i][2], q[i][3]);
    }
  }
}

template <int BN, int PARTS, bool VEC, typename T, int ACT>
cudaError_t run_vec(const LinCall& c) {
  const LinShape& s = c.s;
  constexpr auto kern = k_linear_tc<BN, PARTS, VEC, T, ACT>;
  constexpr int TM = 2 * kBM;
  constexpr size_t smem = smem_bytes<BN, PARTS, VEC>();
  cudaError_t e = allow_smem<kern>(smem);
  if (e != cudaSuccess) return e;
  CUtensorMap xmap, wmap;
  if (!linear_map(&xmap, c.x, (int64_t)PARTS * s.n, s.K, s.ldx, kBM) ||
      !linear_map(&wmap, c.w, (int64_t)PARTS * s.N, s.K, s.ldw, BN / 2))
    return cudaErrorInvalidValue;
  LinTiles g{};
  g.mt = (int)(((int64_t)s.n + TM - 1) / TM);
  g.nt = (s.N + BN - 1) / BN;
  g.group = g.mt < 8 ? g.mt : 8;
  g.tiles = g.mt * g.nt;
  const int pairs = g.tiles < c.num_sms / 2 ? g.tiles : c.num_sms / 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, s, g, xmap, wmap, (const T*)c.bias, (const T*)c.residual, (T*)c.y, (int)kDefaultWaitLimit);
}

template <int BN, int PARTS, typename T, int ACT>
cudaError_t run(const LinCall& c) {
  const LinShape& s = c.s;
  const bool vec = s.N % 32 == 0 && linear_aligned16(c.y, s.ldy, s.n, sizeof(T)) && ((uintptr_t)c.bias & 15) == 0 &&
                   (!c.residual || linear_aligned16(c.residual, s.ldr, s.n, sizeof(T)));
  return vec ? run_vec<BN, PARTS, true, T, ACT>(c) : run_vec<BN, PARTS, false, T, ACT>(c);
}

template <int BN, int PARTS, typename T>
cudaError_t run_act(const LinCall& c) {
  switch (c.s.act) {
    case FI_ACT_NONE: return run<BN, PARTS, T, FI_ACT_NONE>(c);
    case FI_ACT_GELU: return run<BN, PARTS, T, FI_ACT_GELU>(c);
    case FI_ACT_SILU: return run<BN, PARTS, T, FI_ACT_SILU>(c);
    case FI_ACT_RELU: return run<BN, PARTS, T, FI_ACT_RELU>(c);
    case FI_ACT_TANH: return run<BN, PARTS, T, FI_ACT_TANH>(c);
  }
  return cudaErrorInvalidValue;
}

// Which operands TMA takes as they are. A row stride of 0 (one row of x for all)
// is no tensor-map stride.
bool direct_x(const LinShape& s, const void* x) {
  return s.bf16 && linear_aligned16(x, s.ldx, s.n, 2) && (s.ldx != 0 || s.n == 1);
}
bool direct_w(const LinShape& s, const void* w) { return s.bf16 && linear_aligned16(w, s.ldw, s.N, 2); }
int padded(int K) { return (K + 7) / 8 * 8; }
// Rows of x up to which operands that would have to be laid out are read as they
// stand: laying out W alone moves its bytes three times (fp32: four and a half).
int warp_rows(const LinShape& s) { return s.bf16 ? 2 : kWarpRows; }
size_t operand_bytes(const LinShape& s, int64_t rows) {
  return ((size_t)(s.bf16 ? 1 : 3) * rows * padded(s.K) * 2 + 255) / 256 * 256;
}

}  // namespace

size_t linear_workspace(const LinShape& s, const void* x, const void* w) {
  const bool dx = direct_x(s, x), dw = direct_w(s, w);
  if ((dx && dw) || s.n <= warp_rows(s)) return 0;
  return (dx ? 0 : operand_bytes(s, s.n)) + (dw ? 0 : operand_bytes(s, s.N));
}

bool encode_map(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                const uint32_t* box) {
  using Fn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                          const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                          CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Fn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return (Fn)p;
  }();
  if (!fn) return false;
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool linear_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint64_t strides[1] = {rows > 1 ? (uint64_t)ld * 2 : (uint64_t)((cols + 7) / 8 * 16)};
  const uint32_t box[2] = {(uint32_t)kBK, (uint32_t)box_rows};
  return encode_map(map, p, 2, dims, strides, box);
}

cudaError_t launch_linear(const LinShape& shape, const void* x, const void* w, const void* bias, const void* residual,
                          void* y, void* workspace, int num_sms, cudaStream_t st) {
  LinShape s = shape;
  LinCall c{s, x, w, bias, residual, y, num_sms, st};
  const bool dx = direct_x(s, x), dw = direct_w(s, w);
  if (!dx || !dw) {
    if (s.n <= warp_rows(s)) return launch_linear_rows(c);
    const int Kp = padded(s.K);
    LinOperand a{}, b{};
    unsigned char* at = (unsigned char*)workspace;
    if (!dx) {
      a = LinOperand{x, (__nv_bfloat16*)at, s.n, s.ldx, linear_aligned16(x, s.ldx, s.n, s.bf16 ? 2 : 4)};
      at += operand_bytes(s, s.n);
      c.x = a.dst;
      s.ldx = Kp;
    }
    if (!dw) {
      b = LinOperand{w, (__nv_bfloat16*)at, s.N, s.ldw, linear_aligned16(w, s.ldw, s.N, s.bf16 ? 2 : 4)};
      c.w = b.dst;
      s.ldw = Kp;
    }
    const int64_t ua = a.rows * (Kp / 8), units = ua + b.rows * (Kp / 8);
    const int64_t blocks = (units + 255) / 256, most = (int64_t)num_sms * 16;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks < most ? blocks : most));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = s.bf16 ? cudaLaunchKernelEx(&cfg, k_linear_layout<__nv_bfloat16>, a, b, s.K, Kp, ua, units)
                                 : cudaLaunchKernelEx(&cfg, k_linear_layout<float>, a, b, s.K, Kp, ua, units);
    if (e != cudaSuccess) return e;
  }
  if (linear_few_fits(s, num_sms)) return launch_linear_few(c);
  if (!s.bf16) return run_act<128, 3, float>(c);
  // Columns of a tile: the rounds of tiles over the CTA pairs times a tile's time,
  // which goes with its columns and about 48 more (wider tiles read W less often, but
  // leave a last round emptier).
  const int64_t mt = ((int64_t)s.n + 2 * kBM - 1) / (2 * kBM), pairs = num_sms / 2;
  auto cost = [&](int bn) { return (mt * ((s.N + bn - 1) / bn) + pairs - 1) / pairs * (bn + 48); };
  if (cost(256) <= cost(192) && cost(256) <= cost(128)) return run_act<256, 1, __nv_bfloat16>(c);
  if (cost(192) <= cost(128)) return run_act<192, 1, __nv_bfloat16>(c);
  return run_act<128, 1, __nv_bfloat16>(c);
}

cudaError_t linear_take_error(cudaStream_t st, int* flag) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(flag, g_linear_error, sizeof(int), 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && *flag) {
    const int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_linear_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  return e;
}

}  // namespace fi
