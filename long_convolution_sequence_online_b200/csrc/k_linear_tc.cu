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
// activation and residual to one tile while the next is multiplied. Where tiles
// leave most SMs idle, 2 or 4 pairs share a tile's contraction in a cluster and add
// up their sums through distributed shared memory.
//
// Bound: the tensor pipe. 16384 x 2048 -> 8192 bf16 + GELU 439 to 460 us (1.2 PFLOP/s
// under the power cap, where the library's product alone takes 400 to 415), 8192 x 2048 ->
// 2048 49 us (46); fp32 8192 x 768 -> 768 + GELU 57 us, 10 of them laying out (192 tiles
// are 2.6 rounds of the pairs), 4096 x 2048 -> 2048 170 to 175 us. Small products are bound by
// latency, 6 to 7 us up to a contraction of 1000.
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
// the 2-norm, with two blocks of 64 to an accumulator 6e-7; with one, smallest products
// first, added up in the epilogue warps' registers, they are 1e-7 off, the library's
// fp32 product 8e-7.
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

// Stage of the ring: an x tile 128 x 128 bytes and half of a W tile, BN / 2 x 128 bytes. bf16:
// of two blocks of the contraction (a stage's waits and signals take 350 to 450 cycles
// whatever its size, more than the 264 that the MMAs of one block take at BN = 128). fp32: of
// one part of a block's values, the smallest part first, as the products let go of them:
// with whole blocks only two fit, and the copies of one had to be there within the MMAs of the
// other.
template <int PARTS>
constexpr int kStageBlocks = PARTS == 3 ? 1 : 2;
template <int BN, int PARTS>
constexpr int stage_bytes() { return kStageBlocks<PARTS> * (kBM + BN / 2) * 128; }
// bytes of an epilogue warp's stage (Staged below): 32 rows of 64 bytes and 16 more, 32 biases
constexpr int kStagingBytes = 32 * (64 + 16) + 128;
template <int BN, int PARTS>
constexpr int num_stages() { return (232448 - 1024 - kEpiWarps * kStagingBytes) / stage_bytes<BN, PARTS>(); }
template <int BN, int PARTS>
constexpr size_t smem_bytes() {
  return 1024 + (size_t)num_stages<BN, PARTS>() * stage_bytes<BN, PARTS>() + kEpiWarps * kStagingBytes;
}
// Accumulators: two; fp32, which changes them at every block, four, so that an epilogue
// has four blocks' time.
template <int PARTS>
constexpr int kAccs = PARTS == 3 ? 4 : 2;
template <int BN, int PARTS>
constexpr uint32_t acc_cols() { return kAccs<PARTS> * BN <= 256 ? 256 : 512; }

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

// act(acc + bias) + residual of 64 bytes of columns, a row per lane, go to y by way of shared
// memory, so that a warp's accesses to memory run along the rows (a row per lane costs a lookup per lane and access: 8192 x 768 -> 2048 bf16 25.4
// us, along the rows 21.4). Rows may start anywhere (not ALIGNED) and end inside the
// chunk: each is moved up in shared memory by the elements `a` that its address in
// memory is past a 16-byte boundary, so that memory is still read and written in whole
// units of 16 bytes; its elements then start with E - a single ones, end with a, and
// have units between (a = 0: units alone). A lane's rows lie 8 apart and so share
// their a, which keeps addresses out of the loops: with two warps per scheduler it is
// instructions that bound this. (8192 x 768 -> 767 bf16 + GELU + residual: 23.6 us, 36.0
// with addresses formed per access; 1777 x 865 -> 1727 + tanh + residual: 20.7, 27.3 an
// element at a time.)
template <typename T, bool ALIGNED>
struct StagedSide {                                        // y or the residual: the warp's 32 rows
  static constexpr int C = 64 / sizeof(T);                 // columns of a chunk
  static constexpr int E = 16 / sizeof(T), U = C / E;      // elements of a unit, units of a chunk
  static constexpr int H = E / 4;                          // single elements of a lane and row
  static constexpr int kWords = 16, kRow = 64 + 16;
  T* p;
  int64_t ld;
  T *unit_p, *single_p[H];
  int unit_s, single_s[H], row_a;                          // places in the stage; a of the lane's own row
  int units, singles;                                      // the lane's first row, or 32: it has no such

  static __device__ __forceinline__ int past(const T* q) { return ALIGNED ? 0 : (int)((uintptr_t)q / sizeof(T)) & (E - 1); }
  __device__ __forceinline__ void init(T* first, int64_t stride, int lane) {
    p = first;
    ld = stride;
    row_a = past(p + lane * ld);
    int r = lane / U, a = past(p + r * ld), c = (E - a) % E + E * (lane % U);
    unit_p = p + r * ld + c;
    unit_s = r * kRow + (c + a) * (int)sizeof(T);
    units = lane % U < U - 1 || a == 0 ? r : 32;
    r = lane % 8;
    a = past(p + r * ld);
    singles = a != 0 ? r : 32;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int e = lane / 8 + 4 * h;
      c = e < E - a ? e : C - E + e;
      single_p[h] = p + r * ld + c;
      single_s[h] = r * kRow + (c + a) * (int)sizeof(T);
    }
  }
  __device__ __forceinline__ unsigned char* at(unsigned char* stg, int r, int c) const {
    return stg + r * kRow + (c + past(p + r * ld)) * (int)sizeof(T);
  }
};

template <typename T, bool ALIGNED>
struct Staged {
  using S = StagedSide<T, ALIGNED>;
  static constexpr int C = S::C, E = S::E, U = S::U, H = S::H, kWords = S::kWords, kRow = S::kRow;
  S y, res;
  uint4 unit[U];                                           // a lane's share of a residual on its way
  T single[4 * H];

  __device__ __forceinline__ void fetch(int c, int rows) {   // the columns c .. c + C - 1 are there
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (res.units + 8 * i < rows) unit[i] = *reinterpret_cast<const uint4*>(res.unit_p + c + i * (8 * res.ld));
#pragma unroll
    for (int i = 0; i < 4 && !ALIGNED; ++i)
#pragma unroll
      for (int h = 0; h < H; ++h)
        if (res.singles + 8 * i < rows) single[i * H + h] = res.single_p[h][c + i * (8 * res.ld)];
  }

  // v = act(v + bias) + residual of a row per lane, to y's columns c on. rows, cols:
  // how many there are. With all C the residual has been fetched, and next()
  // fetches the next chunk's.
  template <int ACT, typename Next>
  __device__ __forceinline__ void store(float (&v)[C], int c, int rows, int cols, const T* bias, bool residual, Next next,
                                        unsigned char* stg, int lane) {
    const bool whole = cols >= C;
    float* bs = reinterpret_cast<float*>(stg + 32 * kRow);
    bs[lane] = bias && lane < C && lane < cols ? op_load(bias + lane) : 0.f;
    if (residual) {
      if (whole) {
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (res.units + 8 * i < rows) *reinterpret_cast<uint4*>(stg + res.unit_s + i * (8 * kRow)) = unit[i];
#pragma unroll
        for (int i = 0; i < 4 && !ALIGNED; ++i)
#pragma unroll
          for (int h = 0; h < H; ++h)
            if (res.singles + 8 * i < rows) *reinterpret_cast<T*>(stg + res.single_s[h] + i * (8 * kRow)) = single[i * H + h];
        next();
      } else if (lane < cols) {                            // fewer than C
#pragma unroll 16
        for (int r = 0; r < rows; ++r) *reinterpret_cast<T*>(res.at(stg, r, lane)) = res.p[r * res.ld + c + lane];
      }
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < C; e += 4) {
      const float4 b = *reinterpret_cast<const float4*>(bs + e);
      v[e] = activate<T, ACT>(v[e] + b.x);
      v[e + 1] = activate<T, ACT>(v[e + 1] + b.y);
      v[e + 2] = activate<T, ACT>(v[e + 2] + b.z);
      v[e + 3] = activate<T, ACT>(v[e + 3] + b.w);
    }
    // a row is moved by the bits of its a, words of 4 bytes first
    uint32_t w[kWords + 4];
    unsigned char* mine = stg + lane * kRow;
    if (residual) {
#pragma unroll
      for (int k = 0; k < kWords + 4; k += 4) {
        const uint4 q = *reinterpret_cast<const uint4*>(mine + 4 * k);
        w[k] = q.x; w[k + 1] = q.y; w[k + 2] = q.z; w[k + 3] = q.w;
      }
      const int by = res.row_a * (int)sizeof(T) / 4;
#pragma unroll
      for (int k = 0; k < kWords + 2; ++k) w[k] = by & 2 ? w[k + 2] : w[k];
#pragma unroll
      for (int k = 0; k < kWords + 1; ++k) w[k] = by & 1 ? w[k + 1] : w[k];
      if constexpr (sizeof(T) == 2) {
        const uint32_t sel = res.row_a & 1 ? 0x5432 : 0x3210;
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
          const uint32_t x = __byte_perm(w[k], w[k + 1], sel);
          v[2 * k] += lo_f(x);
          v[2 * k + 1] += hi_f(x);
        }
      } else {
#pragma unroll
        for (int k = 0; k < kWords; ++k) v[k] += __uint_as_float(w[k]);
      }
      __syncwarp();
    }
    const int by = y.row_a * (int)sizeof(T) / 4;
#pragma unroll
    for (int k = 0; k < kWords + 4; ++k) w[k] = 0;
    if constexpr (sizeof(T) == 2) {
      const uint32_t sel = y.row_a & 1 ? 0x5432 : 0x7654;
      uint32_t before = 0;
#pragma unroll
      for (int k = 0; k < kWords; ++k) {
        const uint32_t x = pack2(v[2 * k], v[2 * k + 1]);
        w[k] = __byte_perm(before, x, sel);
        before = x;
      }
      w[kWords] = before >> 16;
    } else {
#pragma unroll
      for (int k = 0; k < kWords; ++k) w[k] = __float_as_uint(v[k]);
    }
#pragma unroll
    for (int k = kWords + 1; k > 0; --k) w[k] = by & 1 ? w[k - 1] : w[k];
#pragma unroll
    for (int k = kWords + 3; k > 1; --k) w[k] = by & 2 ? w[k - 2] : w[k];
#pragma unroll
    for (int k = 0; k < kWords + 4; k += 4)
      *reinterpret_cast<uint4*>(mine + 4 * k) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
    __syncwarp();
    if (whole) {
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (y.units + 8 * i < rows)
          *reinterpret_cast<uint4*>(y.unit_p + c + i * (8 * y.ld)) =
              *reinterpret_cast<const uint4*>(stg + y.unit_s + i * (8 * kRow));
#pragma unroll
      for (int i = 0; i < 4 && !ALIGNED; ++i)
#pragma unroll
        for (int h = 0; h < H; ++h)
          if (y.singles + 8 * i < rows) y.single_p[h][c + i * (8 * y.ld)] = *reinterpret_cast<const T*>(stg + y.single_s[h] + i * (8 * kRow));
    } else if (lane < cols) {
#pragma unroll 4
      for (int r = 0; r < rows; ++r) y.p[r * y.ld + c + lane] = *reinterpret_cast<const T*>(y.at(stg, r, lane));
    }
    __syncwarp();
  }
};

// BN: columns of a tile. PARTS: 1 (bf16) or 3 (fp32; part p of a matrix is its rows
// p n .. (p + 1) n). ALIGNED: rows of y and residual at 16-byte boundaries. An epilogue
// warp drains tensor-memory lanes 32 (w % 4) .. + 31, column half w / 4.
template <int BN, int PARTS, bool ALIGNED, bool SPLIT, typename T, int ACT>
__global__ void __launch_bounds__(kLinThreads, 1)
k_linear_tc(LinShape s, LinTiles g, const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
            const T* __restrict__ bias, const T* residual, T* y, int log_split, int wait_limit) {
  constexpr int BW = BN / 2;                       // W rows in this CTA's stages
  constexpr int KS = kStageBlocks<PARTS>, NA = kAccs<PARTS>;
  constexpr int ST = num_stages<BN, PARTS>(), SB = stage_bytes<BN, PARTS>();
  constexpr int XB = kBM * 128, WB = BW * 128;
  constexpr int TM = 2 * kBM;                      // rows of a tile
  extern __shared__ unsigned char raw_smem[];
  __shared__ uint64_t full_bar[ST], empty_bar[ST], acc_full[NA], acc_empty[NA];
  __shared__ uint32_t tmem_s;
  __shared__ int abort_s;
  unsigned char* ring = raw_smem + ((1024 - (saddr(raw_smem) & 1023)) & 1023);
  unsigned char* staging = ring + (size_t)ST * SB;
  float* sums = reinterpret_cast<float*>(ring);    // [BN][kBM], once no stage is used any more
  static_assert(!SPLIT || BN * kBM * 4 <= ST * SB, "the ring holds the sums");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &abort_s;
  // a cluster is `split` pairs, which share a tile's contraction
  const int crank = (int)cluster_rank(), rank = crank & 1, part = crank >> 1;
  const uint16_t pair = (uint16_t)(3 << (crank & ~1));
  if constexpr (!SPLIT) log_split = 0;
  const int split = 1 << log_split, first = blockIdx.x >> (log_split + 1), stride = gridDim.x >> (log_split + 1);
  if (warp == 0) tmem_alloc2(&tmem_s, acc_cols<BN, PARTS>());
  if (tid == 32) {
    for (int i = 0; i < ST; ++i) {
      bar_init(&full_bar[i], 1);
      bar_init(&empty_bar[i], 1);
    }
    for (int i = 0; i < NA; ++i) {
      bar_init(&acc_full[i], 1);
      bar_init(&acc_empty[i], 2 * kEpiWarps);
    }
    abort_s = 0;
    bar_init_fence();
    tma_prefetch(&xmap);
    tma_prefetch(&wmap);
  }
  fence_before();
  cluster_sync();
  fence_after();
  pdl_wait_primary();                              // from here on inputs are read and y is written
  const uint32_t tmem = tmem_s;
  const int stages = (s.K + KS * kBK - 1) / (KS * kBK);   // of a tile; this pair's: k0 .. k1
  const int k0 = (int)((uint32_t)(stages * part) >> log_split), k1 = (int)((uint32_t)(stages * (part + 1)) >> log_split);
  auto give_up = [&]() {
    *abort_flag = 1;
    atomicExch(&g_linear_error, 1);
  };

  if (warp < kEpiWarps) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, half = warp >> 2;
    constexpr int CW = BN / 2, SC = Staged<T, ALIGNED>::C;   // columns of this warp, of a chunk
    unsigned char* stg = staging + warp * kStagingBytes;
    uint32_t unit = 0;                             // accumulators drained
    bool alive = true;
    for (int t = first; t < g.tiles && alive; t += stride) {
      int m, n;
      tile_at(g, t, m, n);
      const int64_t row0 = (int64_t)m * TM + rank * kBM + 32 * q;
      const int col0 = n * BN + half * CW;
      const uint32_t at = tmem + ((uint32_t)(32 * q) << 16) + half * CW;
      // the tile's residual on its way into L2 while the tile is multiplied: a lane per row
      if (!SPLIT && residual && row0 + lane < s.n) {
        const char* rp = reinterpret_cast<const char*>(residual + (row0 + lane) * s.ldr + col0);
        const int bytes = min(CW, s.N - col0) * (int)sizeof(T);
        for (int o = 0; o < bytes; o += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(rp + o));
      }
      const int rows = (int)min((int64_t)32, s.n - row0);   // may be negative
      Staged<T, ALIGNED> staged;
      staged.y.init(y + row0 * s.ldy + col0, s.ldy, lane);
      if (residual) staged.res.init(const_cast<T*>(residual) + row0 * s.ldr + col0, s.ldr, lane);
      auto fetch = [&](int c) {
        if (residual && c < CW && rows > 0 && col0 + c + SC <= s.N) staged.fetch(c, rows);
      };
      auto store = [&](float (&v)[SC], int c) {
        if constexpr (SPLIT) {
#pragma unroll
          for (int e = 0; e < SC; ++e) sums[(half * CW + c + e) * kBM + 32 * q + lane] = v[e];
        } else {
          if (rows <= 0 || col0 + c >= s.N) return;
          staged.template store<ACT>(v, c, rows, s.N - col0 - c, bias ? bias + col0 + c : nullptr, residual != nullptr,
                                     [&] { fetch(c + SC); }, stg, lane);
        }
      };
      if constexpr (!SPLIT) fetch(0);
      if constexpr (PARTS == 1) {
        alive = warp_wait(&acc_full[unit % NA], (unit / NA) & 1, wait_limit, abort_flag);
        if (!alive) break;
        fence_after();
        auto load = [&](int c, float (&v)[32]) {
          uint32_t r[32];
          tmem_ld32(at + (unit % NA) * BN + c, r);
          ld_wait();
          if (c + 32 >= CW) {                      // all columns read: the MMA may overwrite them
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive_leader(&acc_empty[unit % NA]);
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
        for (int kb = k0; kb < k1; ++kb, ++unit) {
          alive = warp_wait(&acc_full[unit % NA], (unit / NA) & 1, wait_limit, abort_flag);
          if (!alive) break;
          fence_after();
#pragma unroll
          for (int c = 0; c < CW; c += 16) {
            uint32_t r[16];
            tmem_ld16(at + (unit % NA) * BN + c, r);
            ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[c + e] += __uint_as_float(r[e]);
          }
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive_leader(&acc_empty[unit % NA]);
        }
        if (!alive) break;
#pragma unroll
        for (int c = 0; c < CW; c += SC) {
          float v[SC];
#pragma unroll
          for (int e = 0; e < SC; ++e) v[e] = acc[c + e];
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
        for (int kb = k0; kb < k1; ++kb) {
          const bool start = PARTS > 1 || kb == k0;              // of an accumulator
          if (start)
            alive = unit < NA || warp_wait(&acc_empty[unit % NA], (unit / NA - 1) & 1, wait_limit, abort_flag);
#pragma unroll
          for (int p = 0; p < PARTS; ++p)
            alive = alive && warp_wait(&full_bar[(kbs + p) % ST], ((kbs + p) / ST) & 1, wait_limit, abort_flag);
          if (!alive) break;
          fence_after();
          const uint32_t d = tmem + (unit % NA) * BN;
          const bool last = PARTS > 1 || kb == k1 - 1;
          if (issuer) {
            if constexpr (PARTS == 1) {
              const uint32_t xa = saddr(ring + (size_t)(kbs % ST) * SB), wa = xa + KS * XB;
              const int steps = min(KS * kBK / 16, (s.K - kb * KS * kBK + 15) / 16);   // of 16
#pragma unroll
              for (int k = 0; k < KS * kBK / 16; ++k) {
                if (k >= steps) break;
                const uint32_t xo = (k / 4) * XB + (k % 4) * 32, wo = (k / 4) * WB + (k % 4) * 32;
                mma2(d, desc_k(xa + xo), desc_k(wa + wo), id, !start || k > 0);
              }
              commit2(&empty_bar[kbs % ST], pair);
            } else {
              constexpr int px[6] = {2, 0, 1, 1, 0, 0}, pw[6] = {0, 2, 1, 0, 1, 0};   // smallest first
              uint32_t at[3];                                    // the stage of part 2 - j follows that of 3 - j
#pragma unroll
              for (int j = 0; j < 3; ++j) at[2 - j] = saddr(ring + (size_t)((kbs + j) % ST) * SB);
#pragma unroll
              for (int p = 0; p < 6; ++p) {
#pragma unroll
                for (int k = 0; k < kBK / 16; ++k)
                  mma2(d, desc_k(at[px[p]] + 32 * k), desc_k(at[pw[p]] + XB + 32 * k), id, p > 0 || k > 0);
                if (p == 1) commit2(&empty_bar[kbs % ST], pair);         // part 2 is done with
                if (p == 4) commit2(&empty_bar[(kbs + 1) % ST], pair);
                if (p == 5) commit2(&empty_bar[(kbs + 2) % ST], pair);
              }
            }
            if (last) commit2(&acc_full[unit % NA], pair);
          }
          __syncwarp();
          kbs += PARTS;
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
      for (int kb = k0; kb < k1 && alive; ++kb)
#pragma unroll
        for (int p = PARTS - 1; p >= 0; --p, ++kbs) {
          const int st = kbs % ST, k = kb * KS * kBK;
          alive = kbs < ST || warp_wait(&empty_bar[st], (kbs / ST - 1) & 1, wait_limit, abort_flag);
          if (!alive) break;
          if (issuer) {
            unsigned char* dst = ring + (size_t)st * SB;
            const int units = min(KS, (s.K - k + kBK - 1) / kBK);
            if (rank == 0) bar_expect(&full_bar[st], 2 * units * (XB + WB));   // both CTAs' tiles
#pragma unroll
            for (int u = 0; u < KS; ++u)
              if (u < units) {
                tma_2d_pair(dst + u * XB, &xmap, &full_bar[st], k + u * kBK, p * s.n + m * TM + rank * kBM);
                tma_2d_pair(dst + KS * XB + u * WB, &wmap, &full_bar[st], k + u * kBK, p * s.N + n * BN + rank * BW);
              }
          }
          __syncwarp();
        }
    }
    if (!alive && lane == 0) give_up();
    // no copy of this CTA may still be in flight when it ends: each stage's last use is done
    const uint32_t oldest = kbs > ST ? kbs - ST : 0;
    bool used = true;
    for (uint32_t i = oldest; i < kbs && used; ++i) used = bar_wait(&empty_bar[i % ST], (i / ST) & 1, kDrainLimit, abort_flag);
    if (!used) {
      // The products gave up. Both CTAs' copies count on the leader's barriers, and the pair
      // ends together: the leader waits for the stages that it asked for, the other CTA for
      // as long as the limit allows (it may have asked for one more).
      if (rank == 0) {
        for (uint32_t i = oldest; i < kbs; ++i) bar_wait(&full_bar[i % ST], (i / ST) & 1, kDrainLimit);
      } else {
        bar_wait(&empty_bar[(kbs - 1) % ST], ((kbs - 1) / ST) & 1, kDrainLimit);
      }
    }
  }
  if constexpr (SPLIT) {
    // every pair left its sums in shared memory, where no stage is used any more; each
    // finishes BN / split columns, in the order of the pairs
    const int q = warp & 3, half = warp >> 2, width = BN >> log_split, c0 = part * width + 32 * half;
    int m, n;
    tile_at(g, first, m, n);
    const int64_t row0 = (int64_t)m * TM + rank * kBM + 32 * q;
    const int col0 = n * BN + c0, rows = (int)min((int64_t)32, s.n - row0);
    const bool work = warp < kEpiWarps && 32 * half < width && rows > 0 && col0 < s.N;
    constexpr int SC = Staged<T, ALIGNED>::C;
    Staged<T, ALIGNED> staged;
    if (work) {
      staged.y.init(y + row0 * s.ldy + col0, s.ldy, lane);
      if (residual) staged.res.init(const_cast<T*>(residual) + row0 * s.ldr + col0, s.ldr, lane);
      if (residual && col0 + SC <= s.N) staged.fetch(0, rows);
    }
    fence_before();
    cluster_sync();
    fence_after();
    if (work) {
      float v[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = 0.f;
      for (int i = 0; i < split; ++i) {
        const uint32_t from = cluster_addr(sums + c0 * kBM + 32 * q + lane, 2 * i + rank);
        float u[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) u[e] = ld_cluster(from + e * (kBM * 4));
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] += u[e];
      }
#pragma unroll
      for (int c = 0; c < 32; c += SC) {
        if (col0 + c >= s.N) break;
        float u[SC];
#pragma unroll
        for (int e = 0; e < SC; ++e) u[e] = v[c + e];
        auto next = [&] {
          if (residual && c + SC < 32 && col0 + c + 2 * SC <= s.N) staged.fetch(c + SC, rows);
        };
        staged.template store<ACT>(u, c, rows, s.N - col0 - c, bias ? bias + col0 + c : nullptr, residual != nullptr, next,
                                   staging + warp * kStagingBytes, lane);
      }
    }
  }
  fence_before();
  cluster_sync_relaxed();                          // no CTA ends while another may still signal it or read its sums
  fence_after();
  if (warp == 0) tmem_free2(tmem, acc_cols<BN, PARTS>());
}

// An operand that TMA cannot take (fp32, or rows at no 16-byte boundary) as
// `parts` bf16 matrices of rows of Kp = K rounded up to 8 elements, the rest zero:
// 8 elements per thread, read once, written once. I: what counts them.
struct LinOperand {
  const void* src;
  __nv_bfloat16* dst;
  int64_t rows, ld;
  int vec;               // rows start at 16-byte boundaries
};
template <typename T, typename I>
__global__ void __launch_bounds__(256) k_linear_layout(LinOperand a, LinOperand b, int K, int Kp, int64_t units_a, int64_t units) {
  pdl_launch_dependents();                 // the product, which waits for this launch's end
  pdl_wait_primary();
  const I per = (I)(Kp / 8);
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += (int64_t)gridDim.x * 256) {
    const bool first = u < units_a;
    const LinOperand& o = first ? a : b;
    const I v = (I)(first ? u : u - units_a), r = v / per;
    const int k = (int)(v - r * per) * 8;
    const int64_t row = (int64_t)r;
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

// Pairs that share a tile's contraction, log2, where tiles leave most SMs idle: worth
// its 1 us of exchange from a contraction of about 1500 in bf16 and 256 in fp32 (300 x
// 512 -> 512 bf16: 6.3 us, split by two 7.2; 600 x 4096 -> 256: 16.6, by four 10.5, fp32
// 69.7 and 27.0). Clusters of 8 CTAs do not fill every group of SMs: 16 tiles by four
// need two rounds (160 x 2048 -> 2048 fp32: 36.6 us, by two 27.3).
int linear_log_split(const LinShape& s, int tiles, int num_sms) {
  const int stages = (s.K + kBK - 1) / kBK / (s.bf16 ? kStageBlocks<1> : kStageBlocks<3>);
  if (8 * tiles <= num_sms * 3 / 4 && stages >= (s.bf16 ? 16 : 8)) return 2;
  return 4 * tiles <= num_sms * 9 / 10 && stages >= (s.bf16 ? 12 : 4);
}

LinTiles tiles_of(const LinShape& s, int bn) {
  LinTiles g{};
  g.mt = (int)(((int64_t)s.n + 2 * kBM - 1) / (2 * kBM));
  g.nt = (s.N + bn - 1) / bn;
  g.group = g.mt < 8 ? g.mt : 8;
  g.tiles = g.mt * g.nt;
  return g;
}

template <int BN, int PARTS, bool ALIGNED, bool SPLIT, typename T, int ACT>
cudaError_t run_rows(const LinCall& c, int log_split) {
  const LinShape& s = c.s;
  constexpr auto kern = k_linear_tc<BN, PARTS, ALIGNED, SPLIT, T, ACT>;
  constexpr size_t smem = smem_bytes<BN, PARTS>();
  cudaError_t e = allow_smem<kern>(smem);
  if (e != cudaSuccess) return e;
  CUtensorMap xmap, wmap;
  if (!linear_map(&xmap, c.x, (int64_t)PARTS * s.n, s.K, s.ldx, kBM) ||
      !linear_map(&wmap, c.w, (int64_t)PARTS * s.N, s.K, s.ldw, BN / 2))
    return cudaErrorInvalidValue;
  const LinTiles g = tiles_of(s, BN);
  const int split = 1 << log_split, pairs = SPLIT ? g.tiles * split : g.tiles < c.num_sms / 2 ? g.tiles : c.num_sms / 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2 * split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, s, g, xmap, wmap, (const T*)c.bias, (const T*)c.residual, (T*)c.y, log_split,
                            op_wait_limit());
}

template <int BN, int PARTS, typename T, int ACT>
cudaError_t run(const LinCall& c) {
  const LinShape& s = c.s;
  if constexpr (BN == 128) {
    // a warp stores 32 columns once: no kernels of their own for aligned rows
    if (const int log_split = linear_log_split(s, tiles_of(s, BN).tiles, c.num_sms))
      return run_rows<BN, PARTS, false, true, T, ACT>(c, log_split);
  }
  const bool aligned = linear_aligned16(c.y, s.ldy, s.n, sizeof(T)) &&
                       (!c.residual || linear_aligned16(c.residual, s.ldr, s.n, sizeof(T)));
  return aligned ? run_rows<BN, PARTS, true, false, T, ACT>(c, 0)
                 : run_rows<BN, PARTS, false, false, T, ACT>(c, 0);
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
    const bool narrow = units <= UINT32_MAX;
    const cudaError_t e =
        s.bf16 ? cudaLaunchKernelEx(&cfg, narrow ? k_linear_layout<__nv_bfloat16, uint32_t> : k_linear_layout<__nv_bfloat16, uint64_t>,
                                    a, b, s.K, Kp, ua, units)
               : cudaLaunchKernelEx(&cfg, narrow ? k_linear_layout<float, uint32_t> : k_linear_layout<float, uint64_t>, a, b, s.K, Kp,
                                    ua, units);
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
