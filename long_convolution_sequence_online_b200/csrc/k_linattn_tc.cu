// Linear attention over prompts on the 5th-generation tensor cores: the chunked
// form (k_linattn.cu) with chunks of 128 positions, bf16 inputs by TMA,
// accumulators in tensor memory.
//
// One CTA runs the chunks of a segment of one (sequence, head) in order. Per
// chunk, with Q, K, V the 128-row tiles and S the state before it:
//     scores = Q K^T            -> P = scale scores * g^{i-j} for j <= i (over them)
//     inter  = Q S              (S as two bf16 parts)
//     intra  = P V              (P as two bf16 parts, read from tensor memory)
//     KV     = K^T (w V)        w_j = g^{m-1-j}, w V as three bf16 parts
//     S     <- g^m S + KV       (fp32, in registers)
//     o      = scale g^{i+1} inter + intra
// Roundings below fp32: the result, and P and S where they enter their products, to two
// bf16 parts, 16 bits each: 2^-16 of every term at most, where the result's own rounding
// is 2^-8 of itself. (With one part each, 32 x 2K positions of 16 heads of 128 took 300
// us instead of 357 and 16K of one sequence 113 instead of 125, with an error of the size
// of the result's own rounding, 0.00235 in the 2-norm instead of 0.00166, and a multiple
// of it where the two terms cancel.) S's parts take the same place one after the other;
// shared memory has none for both. The state itself must stay an fp32 sum, so w V
// is not rounded: three parts hold all 24 bits of it, the products with the
// bf16 K are exact, and every chunk's KV is accumulated on its own (the tensor
// core's sums are not rounded to nearest) and added to S in registers.
//
// Sixteen worker warps do all arithmetic, each on a 32 x 32 (state, outputs: 32 x
// DV / 4) block of every matrix, one phase after another; one warp issues the
// MMAs, one the TMA copies. Per chunk c the workers form the first half of w V,
// the outputs of chunk c - 1, the second half of w V, P, and the state; the MMAs
// run in the order KV (first half), Q K^T, Q S, KV (second half), Q S (second part), P V. Each phase
// of the workers then overlaps MMAs that do not need it, and an arrival on
// w_ready tells the issuer that everything before it in the workers' order is done
// as well. CTAs are persistent: the copies run ahead into the next task. (Warps
// with a role each - P and outputs 4, state 8, w V 4 - took 10400 cycles a chunk at
// 128 x 128, two groups of eight, w V and state beside P and outputs, 9000: a few
// warps do not hide their own latency, and more code at a time misses the
// instruction cache.)
//
// Bound: the workers' instruction latency, at 51 % of the issue slots and 42 % of the
// tensor pipe: 5.8 us a chunk at 128 x 128 with all SMs at work (16 chunks with the CTA's
// start). 16 heads of 128, bf16: one sequence of 16K 125 us (states 40, outputs 85; 2.2
// TB/s), 32 of 2K 353 to 362 us (3.1 TB/s). fp32, 12 heads of 64, 8K: 108 us (layout 27,
// states 26, outputs 56), waiting on products and single-buffered tiles.
//
// fp32 inputs come as three bf16 parts each and every product as six products of parts;
// their tiles fit up to 64 dimensions. Above, blocks of 64 value dimensions are tasks of
// their own, and blocks of key dimensions launches of their own, of which the later
// ones add to the outputs (q . k is the sum over them). Scores are formed once per
// block: 4 x 2048 positions, 16 heads of 128, 0.51 ms; in fp32 arithmetic (k_linattn.cu) 0.97.
#include <type_traits>

#include "op_internal.cuh"
#include "tc.cuh"

namespace fi {

namespace {

using namespace tc;

constexpr int kCh = 128;                 // positions per chunk
constexpr int kWHalf = 64;               // positions of w V in shared memory at a time
constexpr int kWorkers = 16;
constexpr int kMmaWarp = kWorkers, kTmaWarp = kMmaWarp + 1;
constexpr int kLaTcThreads = 32 * (kTmaWarp + 1);

__device__ int g_linattn_error;          // a bounded wait gave up since the last check

// DK, DV: key and value dimensions padded to 64 or 128. V is double
// buffered (the next chunk's w V starts first), K and Q where there is room.
// The launch that forms states only has room for two halves of w V.
// PARTS: bf16 parts of an input, 1 or 3 (fp32).
template <int DK, int DV, bool OUT, int PARTS>
struct LaSmem {
  static constexpr int kSlotsKQ = PARTS == 3 || (DK == 128 && DV == 128) ? 1 : 2, kSlotsV = PARTS == 3 && OUT ? 1 : 2;
  static constexpr int kHalves = OUT ? 1 : 2;
  static constexpr int kPlaneK = kCh * 2 * DK, kPlaneV = kCh * 2 * DV;   // a part of a tile
  static constexpr int kTileK = PARTS * kPlaneK, kTileV = PARTS * kPlaneV;
  static constexpr int kPart = kWHalf * 2 * DV;
  // the state passes through in fp32 rows of 64 columns and 16 bytes on its way in and out
  static constexpr int kLd = 64 + 4, kStage = 128 * kLd * 4;
  static constexpr int kHalf = 3 * kPart;
  static constexpr int kW = kHalves * kHalf > kStage ? kHalves * kHalf : kStage;
  static constexpr int kStatePart = DK * 2 * DV, kState = OUT ? PARTS * kStatePart : 0;
  static constexpr size_t bytes = 1024 + (size_t)(OUT ? 2 : 1) * kSlotsKQ * kTileK + kSlotsV * kTileV + kW + kState;
};

// Coordinates of a tensor map [dim][position][sequence][head]; a stride of 0
// becomes a dimension of 1 and a coordinate of 0.
struct LaMul {
  int qb, qh, kb, kh, vb, vh;
};

// TMEM columns: scores, with two parts of P over them, fp32's third beside them, Q S, P V
// and K^T (w V), the last twice in the launch that forms states only. fp32: P V and K^T (w V)
// have an accumulator for each half of the chunk, 64 columns apart. The tensor core cuts
// its sums off, so what counts is how many products add to a sum of full size: of the six
// of parts only the last, four steps of 16 (with one accumulator, 28 of K^T (w V) and 8 of
// P V: outputs 6.7e-7 off in the 2-norm, now 3e-7, where a plain fp32 form has 2.2e-7).
template <int PARTS>
struct LaCols {
  static constexpr uint32_t scores = 0, p = 0, p2 = 128, inter = PARTS == 3 ? 192 : 128, intra = 256, kv = 384,
                            half = PARTS == 3 ? 64 : 0, next_kv = PARTS == 3 ? 256 : 128;
};
// Which parts a product takes, smallest products first: two bits per product.
// Three parts on both sides: (2,0) (0,2) (1,1) (1,0) (0,1) (0,0); one against three:
// (0,2) (0,1) (0,0).
constexpr uint32_t kPairA = 0x052, kPairB = 0x118, kSingleB = 0x006;

// What a CTA does for one (sequence, head), segment and, fp32, block of 64 value
// dimensions (v0 ..); `slot` counts the former without the segments.
struct LaTask {
  int slot, bh, b, h, v0, dv, seg, len, end, nch;
  int64_t t0;
  bool ragged;    // the last chunk ends inside a longer batch: what stands behind is cleared in the tiles
};
template <bool OUT, int PARTS>
__device__ __forceinline__ LaTask la_task(const LaShape& s, const LaPlan& p, const LaPtrs& a, int i) {
  LaTask t;
  const int blocks = PARTS == 3 ? (s.dv + 63) / 64 : 1, slots = s.B * s.H * blocks;
  t.slot = i % slots;                    // segments of a head far apart: the early ones end first
  t.bh = PARTS == 3 ? t.slot / blocks : t.slot;
  t.v0 = PARTS == 3 ? (t.slot - t.bh * blocks) * 64 : 0;
  t.dv = PARTS == 3 ? min(64, s.dv - t.v0) : s.dv;
  t.seg = i / slots;
  t.b = t.bh / s.H;
  t.h = t.bh - t.b * s.H;
  t.len = la_length(a.lengths, t.b, s.n);
  t.t0 = (int64_t)t.seg * p.seg;
  t.end = (int)min((int64_t)t.len, t.t0 + p.seg);
  // the state's launch skips a segment that none follows
  const bool work = OUT ? t.t0 < t.len : t.t0 + p.seg < t.len;
  t.nch = work ? (int)((t.end - t.t0 + kCh - 1) / kCh) : 0;
  // behind the longest sequence stand zeros, or (parts one after the other) the next part's start
  t.ragged = t.end == t.len && (t.len < s.n || PARTS == 3) && (t.end - t.t0) % kCh != 0;
  return t;
}

// ADD: outputs are added to o (a further block of key dimensions).
template <int DK, int DV, bool OUT, int PARTS, bool ADD>
__global__ void __launch_bounds__(kLaTcThreads, 1)
k_linattn_tc(LaShape s, LaPlan p, LaPtrs a, const __grid_constant__ CUtensorMap qmap,
             const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
             const __grid_constant__ CUtensorMap omap, LaMul mul, int vec_out, int tile_out, int vec_state, int wait_limit) {
  using L = LaSmem<DK, DV, OUT, PARTS>;
  using C = LaCols<PARTS>;
  using T = typename std::conditional<PARTS == 3, float, __nv_bfloat16>::type;
  constexpr bool STAGED = OUT && PARTS == 1;   // outputs leave by way of V's tile
  constexpr int NKQ = L::kSlotsKQ, NV = L::kSlotsV;
  constexpr int CW = DV / 4;             // a warp's columns of the state and of the outputs
  extern __shared__ unsigned char raw_smem[];
  __shared__ uint64_t k_full[2], k_empty[2], q_full[2], q_empty[2], v_full[2], v_empty[2];   // v_empty: unless outputs pass through V's tile
  __shared__ uint64_t w_ready[2], w_free[2], qk_done, kv_done[2], qs0_done, qs_done, p_ready, o_done, o_read, o_staged, drained;
  __shared__ float G[kCh + 1];           // g^0 .. g^128
  __shared__ __align__(16) float GR[32]; // g^31 .. g^0
  __shared__ float GD[63];               // GD[31 + i] = scale g^i, i = 0 .. 31 (masked below)
  __shared__ uint32_t tmem_s;
  __shared__ int abort_s;
  unsigned char* ks = raw_smem + ((1024 - (saddr(raw_smem) & 1023)) & 1023);
  unsigned char* qs = ks + NKQ * L::kTileK;
  unsigned char* vs = qs + (OUT ? NKQ * L::kTileK : 0);
  unsigned char* sop = vs + NV * L::kTileV;
  unsigned char* wv = sop + L::kState;
  if constexpr (!OUT) pdl_launch_dependents();   // the launch of the outputs, which waits for this one's end
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tasks = s.B * s.H * (PARTS == 3 ? (s.dv + 63) / 64 : 1) * p.G;
  const int ws_ld = PARTS == 3 ? min(64, s.dv) : s.dv;     // the scratch's states: dk x ws_ld
  const size_t slot = (size_t)s.dk * ws_ld;
  if (warp == 0) tmem_alloc(&tmem_s, 512);
  if (tid == 32) {
    for (int i = 0; i < 2; ++i) {
      bar_init(&k_full[i], 1);
      bar_init(&k_empty[i], 1);
      bar_init(&q_full[i], 1);
      bar_init(&q_empty[i], 1);
      bar_init(&v_full[i], 1);
      bar_init(&v_empty[i], 1);
      bar_init(&w_ready[i], kWorkers);             // by half of the chunk
      bar_init(&w_free[i], 1);
      bar_init(&kv_done[i], 1);                    // by the CTA's chunk, odd and even
    }
    bar_init(&qk_done, 1);
    bar_init(&qs0_done, 1);
    bar_init(&qs_done, 1);
    bar_init(&p_ready, kWorkers);
    bar_init(&o_done, 1);
    bar_init(&o_read, kWorkers);
    bar_init(&o_staged, kWorkers);
    bar_init(&drained, 1);
    abort_s = 0;
    bar_init_fence();
  }
  fence_before();
  __syncthreads();
  fence_after();
  pdl_wait_primary();
  const uint32_t tmem = tmem_s;
  volatile int* abort_flag = &abort_s;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return warp_wait(bar, parity, wait_limit, abort_flag); };
  auto give_up = [&]() {
    if (lane == 0) {
      *abort_flag = 1;
      atomicExch(&g_linattn_error, 1);
    }
    __syncwarp();
  };
  // The arithmetic warps meet at barriers of their own, so after a wait that gave up
  // they run on to the end (no wait lasts any more, the results are not valid).
  auto need = [&](uint64_t* bar, uint32_t parity) {
    if (!wait(bar, parity)) give_up();
  };
  // `it` counts a CTA's chunks over all its tasks; barrier phases go by it.
  bool alive = true;
  int it = 0;

  if (warp < kWorkers) {
    // ------------------------------------------------------------ workers
    const int quarter = warp & 3, grp = warp >> 2;
    const int row = 32 * quarter + lane;           // of the chunk (P, outputs) and of the state (key dimension)
    const int col0 = grp * CW;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
    float* stage = reinterpret_cast<float*>(wv);   // [128][kLd], when w V is not in use
    auto sync = [] {
      __syncwarp();                                // the barrier takes whole warps; lanes may have parted before it
      asm volatile("bar.sync 5, %0;" ::"n"(32 * kWorkers) : "memory");
    };
    float st[CW];                                  // S, row `row`, columns col0 ..
    // S as the B operand of Q S: rows of 64 bf16 columns, 128-byte swizzle. bf16: one of
    // its two parts, which take the same place one after the other.
    auto publish = [&](int part) {
      if (OUT && row < DK) {
#pragma unroll
        for (int e = 0; e < CW; e += 8) {
          const int col = col0 + e, unit = (col & 63) >> 3;
          unsigned char* dst = sop + (col >> 6) * (DK * 128) + row * 128 + ((unit ^ (row & 7)) << 4);
          if constexpr (PARTS == 1) {
            uint32_t q[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              q[x] = pack2_finite(st[e + 2 * x], st[e + 2 * x + 1]);
              if (part == 1) q[x] = pack2(st[e + 2 * x] - lo_f(q[x]), st[e + 2 * x + 1] - hi_f(q[x]));
            }
            *reinterpret_cast<uint4*>(dst) = make_uint4(q[0], q[1], q[2], q[3]);
          } else {
            uint32_t q[3][4];
#pragma unroll
            for (int x = 0; x < 4; ++x) split3(st[e + 2 * x], st[e + 2 * x + 1], q[0][x], q[1][x], q[2][x]);
#pragma unroll
            for (int x = 0; x < 3; ++x)
              *reinterpret_cast<uint4*>(dst + x * L::kStatePart) = make_uint4(q[x][0], q[x][1], q[x][2], q[x][3]);
          }
        }
      }
    };
    // Half of w V as three parts, m positions of the chunk in use, then what `also` does.
    // The arrival also hands over S (published before) and releases the tensor memory read before.
    auto scale = [&](const unsigned char* v, int half, int m, auto also) {
      constexpr int UNITS = kWHalf * DV / 8 / (32 * kWorkers);   // 16-byte units per thread
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int e = tid + u * (32 * kWorkers);   // 64-column block, row, unit
        const int blk = e / (kWHalf * 8), rem = e & (kWHalf * 8 - 1), r = half * kWHalf + (rem >> 3);
        const unsigned char* src = v + blk * (kCh * 128) + half * (kWHalf * 128) + rem * 16;
        const float w = r < m ? G[m - 1 - r] : 0.f;
        float f[8];
#pragma unroll
        for (int part = PARTS - 1; part >= 0; --part) {   // their sum is exact
          uint4 x = *reinterpret_cast<const uint4*>(src + part * L::kPlaneV);
          if (r >= m) x = make_uint4(0, 0, 0, 0);
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[2 * i] = part == PARTS - 1 ? lo_f(xs[i]) : f[2 * i] + lo_f(xs[i]);
            f[2 * i + 1] = part == PARTS - 1 ? hi_f(xs[i]) : f[2 * i + 1] + hi_f(xs[i]);
          }
        }
        uint32_t q0[4], q1[4], q2[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split3(w * f[2 * i], w * f[2 * i + 1], q0[i], q1[i], q2[i]);
        unsigned char* dst = wv + (L::kHalves > 1 ? half * L::kHalf : 0) + blk * (kWHalf * 128) + rem * 16;
        *reinterpret_cast<uint4*>(dst) = make_uint4(q0[0], q0[1], q0[2], q0[3]);
        *reinterpret_cast<uint4*>(dst + L::kPart) = make_uint4(q1[0], q1[1], q1[2], q1[3]);
        *reinterpret_cast<uint4*>(dst + 2 * L::kPart) = make_uint4(q2[0], q2[1], q2[2], q2[3]);
      }
      also();
      fence_async();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&w_ready[half]);
    };
    // Outputs of a task's chunk c (the CTA's chunk j): rows `row`, columns col0 .., 16 at
    // a time (more would not fit the registers beside the state, and a spill goes to
    // L2: shared memory leaves little L1). They go to V's tile, which is not read any
    // more, and from there by TMA (a lane per row, stores from registers touch 32
    // lines each and took 2500 cycles a chunk). Directly go rows behind the end of a
    // sequence, which a tile would overwrite, an o that no tensor map describes, and one
    // whose rows are no multiple of 16 bytes: a TMA store writes whole units of 16
    // bytes, also over what stands behind the end of a row.
    auto outputs = [&](const LaTask& k, int c, int j) {
      need(&o_done, j & 1);
      fence_after();
      const int64_t t = k.t0 + (int64_t)c * kCh + row;
      const float f_inter = s.scale * G[row + 1];   // P carries the scale
      const bool tile = STAGED && tile_out && !(k.ragged && c == k.nch - 1);
      unsigned char* dst = vs + (j % NV) * L::kTileV + row * 128;
      T* op = (T*)a.o + k.b * s.os[1] + k.h * s.os[2] + t * s.os[0] + k.v0 + col0;
#pragma unroll
      for (int d = 0; d < CW; d += 16) {
        uint32_t r[16], q[16];
        __syncwarp();                              // lanes part below, at rows behind the end; these loads take whole warps
        tmem_ld16(lanes + C::inter + col0 + d, r);
        tmem_ld16(lanes + C::intra + col0 + d, q);
        ld_wait();
        if constexpr (PARTS == 3) {
          uint32_t q1[16];
          tmem_ld16(lanes + C::intra + C::half + col0 + d, q1);
          ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) q[e] = __float_as_uint(__uint_as_float(q[e]) + __uint_as_float(q1[e]));
        }
        if (d + 16 >= CW) {                        // all read: the next products may take their place
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&o_read);
        }
        if constexpr (PARTS == 3) {
          if (t >= k.end) continue;
          float w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = fmaf(f_inter, __uint_as_float(r[e]), __uint_as_float(q[e]));
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            if (vec_out && col0 + d + e + 4 <= k.dv) {
              float4 v = make_float4(w[e], w[e + 1], w[e + 2], w[e + 3]);
              if constexpr (ADD) {
                const float4 u = *reinterpret_cast<const float4*>(op + d + e);
                v = make_float4(u.x + v.x, u.y + v.y, u.z + v.z, u.w + v.w);
              }
              *reinterpret_cast<float4*>(op + d + e) = v;
            } else {
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (col0 + d + e + x < k.dv) op_store(op + d + e + x, ADD ? op_load(op + d + e + x) + w[e + x] : w[e + x]);
            }
          }
          continue;
        }
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[e] = pack2(fmaf(f_inter, __uint_as_float(r[2 * e]), __uint_as_float(q[2 * e])),
                       fmaf(f_inter, __uint_as_float(r[2 * e + 1]), __uint_as_float(q[2 * e + 1])));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int col = col0 + d + 8 * u;
          const uint4 v = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
          if (tile) {
            *reinterpret_cast<uint4*>(dst + (col >> 6) * (kCh * 128) + ((((col & 63) >> 3) ^ (row & 7)) << 4)) = v;
          } else if (t < k.end) {
            if (vec_out && col + 8 <= k.dv) {
              *reinterpret_cast<uint4*>(op + d + 8 * u) = v;
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (col + e < k.dv)
                  reinterpret_cast<unsigned short*>(op)[d + 8 * u + e] = (unsigned short)(w[4 * u + e / 2] >> (16 * (e & 1)));
            }
          }
        }
      }
      if constexpr (STAGED) {
        fence_async();
        __syncwarp();
        if (lane == 0) bar_arrive(&o_staged);
      }
    };
    for (int i = blockIdx.x; i < tasks; i += gridDim.x) {
      const LaTask k = la_task<OUT, PARTS>(s, p, a, i);
      float* ws = a.ws ? a.ws + (size_t)k.slot * p.G * slot : nullptr;
      const float ld2 = la_log2_decay(__ldg(a.log_decay + k.h));
      // an empty sequence passes its state on whatever the decay
      const bool from_state = a.state_in && (k.len == 0 || !la_drops(ld2));
      const float* s_in = from_state ? a.state_in + k.bh * s.state_slot + k.v0 : nullptr;
      if (!OUT && k.seg == 0 && s_in)
        for (int r = warp; r < s.dk; r += kWorkers)
          for (int c = lane; c < k.dv; c += 32) ws[r * ws_ld + c] = s_in[(size_t)r * s.state_ld + c];
      if (k.nch == 0 && !(OUT && k.seg == 0 && k.len == 0)) continue;
      sync();                                      // the task before is done with the tables and the stage
      if (tid <= kCh) G[tid] = la_pow(ld2, tid);
      if (tid >= 160 && tid < 192) GR[tid - 160] = la_pow(ld2, 191 - tid);
      if (tid >= 192 && tid < 192 + 63) GD[tid - 192] = s.scale * la_pow(ld2, max(0, tid - 192 - 31));
#pragma unroll
      for (int e = 0; e < CW; ++e) st[e] = 0.f;
      const float* src = !OUT ? nullptr : p.G > 1 ? ws : s_in;
      const int src_ld = p.G > 1 ? ws_ld : s.state_ld;
      const int g0 = s_in ? 0 : 1;
      constexpr int PER = DV / 8;                  // float4s of half a row of the state
      if (src && g0 <= k.seg) {
        // slot 0: the state before the prompt; slot g: segment g - 1's contribution
        if (vec_state) {
          // half of the columns at a time: along the rows into the stage, then a row per lane
          for (int hc = 0; hc < 2; ++hc) {
#pragma unroll
            for (int u = 0; u < 128 * PER / (32 * kWorkers); ++u) {
              const int e = tid + u * (32 * kWorkers), r = e / PER, c = hc * (DV / 2) + 4 * (e % PER);
              float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
              if (r < s.dk && c < k.dv)
                for (int g = g0; g <= k.seg; ++g) {
                  const float f = la_pow(ld2, (g == 0 ? k.seg : k.seg - g) * p.seg);
                  const float4 v = *reinterpret_cast<const float4*>(src + (size_t)g * slot + (size_t)r * src_ld + c);
                  x.x = fmaf(f, v.x, x.x);
                  x.y = fmaf(f, v.y, x.y);
                  x.z = fmaf(f, v.z, x.z);
                  x.w = fmaf(f, v.w, x.w);
                }
              *reinterpret_cast<float4*>(stage + r * L::kLd + 4 * (e % PER)) = x;
            }
            sync();
            if (grp / 2 == hc) {
#pragma unroll
              for (int e = 0; e < CW; e += 4) {
                const float4 v = *reinterpret_cast<const float4*>(stage + row * L::kLd + (grp & 1) * CW + e);
                st[e] = v.x; st[e + 1] = v.y; st[e + 2] = v.z; st[e + 3] = v.w;
              }
            }
            sync();
          }
        } else if (row < s.dk) {
          for (int g = g0; g <= k.seg; ++g) {
            const float f = la_pow(ld2, (g == 0 ? k.seg : k.seg - g) * p.seg);
            const float* sp = src + (size_t)g * slot + (size_t)row * src_ld + col0;
#pragma unroll
            for (int e = 0; e < CW; ++e)
              if (col0 + e < k.dv) st[e] = fmaf(f, sp[e], st[e]);
          }
        }
      }
      sync();                                      // the tables are there, the stage is free
      publish(0);                                  // no Q S of the task before is left: its qs_done was waited for
      // S <- g^m S + KV of the task's chunk c, the CTA's chunk j
      auto update = [&](int c, int j) {
        need(&kv_done[j & 1], (j >> 1) & 1);
        fence_after();
        const float gm = G[min(kCh, (int)(k.end - k.t0) - c * kCh)];
        const uint32_t at = lanes + col0 + (OUT ? C::kv : C::kv - C::next_kv * (j & 1));
#pragma unroll
        for (int d = 0; d < CW; d += 16) {
          uint32_t r[16];
          tmem_ld16(at + d, r);
          ld_wait();
          if constexpr (PARTS == 3) {
            uint32_t r1[16];
            tmem_ld16(at + C::half + d, r1);
            ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) + __uint_as_float(r1[e]));
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) st[d + e] = fmaf(gm, st[d + e], __uint_as_float(r[e]));
        }
      };
      for (int c = 0; c < k.nch; ++c, ++it) {
        const int m = min(kCh, (int)(k.end - k.t0) - c * kCh), sv = it % NV;
        unsigned char* v = vs + sv * L::kTileV;
        need(&v_full[sv], (it / NV) & 1);
        if (k.ragged && c == k.nch - 1) {
          const int sk = it % NKQ;
          need(&k_full[sk], (it / NKQ) & 1);
          unsigned char* kt = ks + sk * L::kTileK;
          for (int e = tid; e < kCh * 8; e += 32 * kWorkers) {     // 16-byte units of a 64-column block
            if ((e >> 3) < m) continue;
            for (int d = 0; d < PARTS * DK / 64; ++d) *reinterpret_cast<uint4*>(kt + d * (kCh * 128) + e * 16) = make_uint4(0, 0, 0, 0);
            for (int d = 0; d < PARTS * DV / 64; ++d) *reinterpret_cast<uint4*>(v + d * (kCh * 128) + e * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        if constexpr (!OUT) {
          // the products of chunk c - 1 go on while w V of chunk c is formed
          if (it > 0) need(&w_free[0], (it - 1) & 1);
          scale(v, 0, m, [] {});
          if (it > 0) need(&w_free[1], (it - 1) & 1);
          scale(v, 1, m, [] {});
          if (c > 0) update(c - 1, it - 1);
          continue;
        }
        scale(v, 0, m, [] {});
        if (OUT && c > 0) outputs(k, c - 1, it - 1);
        need(&w_free[0], it & 1);
        scale(v, 1, m, [&] {
          if constexpr (OUT && PARTS == 1) {
            need(&qs0_done, it & 1);               // the product with S's first part
            publish(1);
          }
        });
        if constexpr (OUT) {
          need(&qk_done, it & 1);
          fence_after();
          // P block (quarter, grp): below the diagonal g^{i-j} = g^{i-j0-31} g^{j0+31-j}
          [[maybe_unused]] uint32_t p2[16];        // the block's third part
#pragma unroll
          for (int x = 0; x < 32; x += 16) {
            float f[16];
            if (grp <= quarter) {
              uint32_t r[16];
              tmem_ld16(lanes + C::scores + 32 * grp + x, r);
              ld_wait();
              if (grp < quarter) {
                const float gi = s.scale * G[row - 32 * grp - 31];
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                  const float4 g4 = *reinterpret_cast<const float4*>(&GR[x + e]);
                  f[e] = __uint_as_float(r[e]) * (gi * g4.x);
                  f[e + 1] = __uint_as_float(r[e + 1]) * (gi * g4.y);
                  f[e + 2] = __uint_as_float(r[e + 2]) * (gi * g4.z);
                  f[e + 3] = __uint_as_float(r[e + 3]) * (gi * g4.w);
                }
              } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) f[e] = x + e <= lane ? __uint_as_float(r[e]) * GD[31 + lane - x - e] : 0.f;
              }
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) f[e] = 0.f;
            }
            // two parts of 16 positions, over their own scores (the product takes 16 positions
            // of P at a time from anywhere), so no warp waits for the others' reads
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if constexpr (PARTS == 1) split2(f[2 * e], f[2 * e + 1], w[e], w[8 + e]);
              else split3(f[2 * e], f[2 * e + 1], w[e], w[8 + e], p2[x / 2 + e]);
            }
            tmem_st16(lanes + C::p + 32 * grp + x, w);
          }
          if constexpr (PARTS == 3) tmem_st16(lanes + C::p2 + 16 * grp, p2);
          st_wait();
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&p_ready);
        }
        update(c, it);
        if constexpr (OUT) {
          need(&qs_done, it & 1);                  // the state before is not read any more
          publish(0);
        }
      }
      if (OUT && k.nch > 0) outputs(k, k.nch - 1, it - 1);
      if (!OUT) update(k.nch - 1, it - 1);
      float* dst = nullptr;
      const int dst_ld = OUT ? s.state_ld : ws_ld;
      if constexpr (!OUT) dst = ws + (size_t)(k.seg + 1) * slot;
      else if (a.state_out && k.end == k.len) dst = a.state_out + k.bh * s.state_slot + k.v0;   // this segment holds the last position
      if (!dst) continue;
      if (vec_state) {
        for (int hc = 0; hc < 2; ++hc) {
          sync();
          if (grp / 2 == hc) {
#pragma unroll
            for (int e = 0; e < CW; e += 4)
              *reinterpret_cast<float4*>(stage + row * L::kLd + (grp & 1) * CW + e) = make_float4(st[e], st[e + 1], st[e + 2], st[e + 3]);
          }
          sync();
#pragma unroll
          for (int u = 0; u < 128 * PER / (32 * kWorkers); ++u) {
            const int e = tid + u * (32 * kWorkers), r = e / PER, c = hc * (DV / 2) + 4 * (e % PER);
            if (r < s.dk && c < k.dv)
              *reinterpret_cast<float4*>(dst + (size_t)r * dst_ld + c) = *reinterpret_cast<const float4*>(stage + r * L::kLd + 4 * (e % PER));
          }
        }
      } else if (row < s.dk) {
#pragma unroll
        for (int e = 0; e < CW; ++e)
          if (col0 + e < k.dv) dst[(size_t)row * dst_ld + col0 + e] = st[e];
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    const bool issuer = elect_one();
    constexpr uint32_t id_qk = idesc(128, 128), id_qs = idesc(128, DV, false, true), id_pv = idesc(128, DV, false, true),
                       id_kv = idesc(128, DV, true, true);
    const uint32_t wa = saddr(wv), sa = saddr(sop);
    // K^T (w V) over half of the chunk, smallest parts first; rows 64..127 of a
    // 64-dimensional K repeat the first ones and are not read.
    auto kv_half = [&](uint32_t ka, int half) {
      const uint32_t d = tmem + C::half * half + (OUT ? C::kv : C::kv - C::next_kv * (it & 1)), w = wa + (L::kHalves > 1 ? half * L::kHalf : 0);
#pragma unroll
      for (int c = 0; c < (PARTS == 3 ? 6 : 3); ++c) {
        const uint32_t kp = PARTS == 3 ? kPairA >> 2 * c & 3 : 0, wp = (PARTS == 3 ? kPairB : kSingleB) >> 2 * c & 3;
#pragma unroll
        for (int x = 0; x < kWHalf / 16; ++x)
          mma(d, desc_mn(ka + kp * L::kPlaneK + (half * kWHalf + 16 * x) * 128, DK == 128 ? kCh * 128 : 0),
              desc_mn(w + wp * L::kPart + 16 * x * 128, kWHalf * 128), id_kv, (PARTS == 1 && half > 0) || c > 0 || x > 0);
      }
    };
    constexpr int NC = PARTS == 3 ? 6 : 1;         // products of parts
    for (int i = blockIdx.x; i < tasks && alive; i += gridDim.x) {
      const LaTask k = la_task<OUT, PARTS>(s, p, a, i);
      for (int c = 0; c < k.nch; ++c, ++it) {
        const int sk = it % NKQ, sv = it % NV;
        const uint32_t ka = saddr(ks + sk * L::kTileK), qa = saddr(qs + sk * L::kTileK), va = saddr(vs + sv * L::kTileV);
        alive = wait(&k_full[sk], (it / NKQ) & 1) && wait(&w_ready[0], it & 1);
        if (!alive) break;
        fence_after();
        if (issuer) {
          kv_half(ka, 0);
          commit(&w_free[0]);
        }
        __syncwarp();
        if constexpr (OUT) {
          // the scores replace P, which the product before reads
          alive = wait(&q_full[sk], (it / NKQ) & 1) && (it == 0 || wait(&o_done, (it - 1) & 1));
          if (!alive) break;
          fence_after();
          if (issuer) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const uint32_t qp = NC > 1 ? kPairA >> 2 * c & 3 : 0, kp = NC > 1 ? kPairB >> 2 * c & 3 : 0;
#pragma unroll
              for (int x = 0; x < DK / 16; ++x) {
                const uint32_t o = (x / 4) * (kCh * 128) + (x % 4) * 32;
                mma(tmem + C::scores, desc_k(qa + qp * L::kPlaneK + o), desc_k(ka + kp * L::kPlaneK + o), id_qk, c > 0 || x > 0);
              }
            }
            commit(&qk_done);
          }
          __syncwarp();
          // the state before was published ahead of w_ready; its product replaces
          // outputs that have been read
          alive = it == 0 || wait(&o_read, (it - 1) & 1);
          if (!alive) break;
          fence_after();
          if (issuer) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const uint32_t qp = NC > 1 ? kPairA >> 2 * c & 3 : 0, sp = NC > 1 ? kPairB >> 2 * c & 3 : 0;
#pragma unroll
              for (int x = 0; x < DK / 16; ++x)
                mma(tmem + C::inter, desc_k(qa + qp * L::kPlaneK + (x / 4) * (kCh * 128) + (x % 4) * 32),
                    desc_mn(sa + sp * L::kStatePart + 16 * x * 128, DK * 128), id_qs, c > 0 || x > 0);
            }
            if constexpr (PARTS == 1) {
              commit(&qs0_done);                   // the other part follows in its place
            } else {
              commit(&qs_done);
              commit(&q_empty[sk]);
            }
          }
          __syncwarp();
        }
        alive = wait(&w_ready[1], it & 1);
        if (!alive) break;
        fence_after();
        if (issuer) {
          kv_half(ka, 1);
          if constexpr (!OUT) commit(&w_free[1]);
          commit(&kv_done[it & 1]);
          commit(&k_empty[sk]);
          if constexpr (!OUT) commit(&v_empty[sv]);
          if constexpr (OUT && PARTS == 1) {
#pragma unroll
            for (int x = 0; x < DK / 16; ++x)
              mma(tmem + C::inter, desc_k(qa + (x / 4) * (kCh * 128) + (x % 4) * 32), desc_mn(sa + 16 * x * 128, DK * 128), id_qs, 1);
            commit(&qs_done);
            commit(&q_empty[sk]);
          }
        }
        __syncwarp();
        if constexpr (OUT) {
          alive = wait(&p_ready, it & 1);
          if (!alive) break;
          fence_after();
          if (issuer) {
#pragma unroll
            for (int c = 0; c < (PARTS == 3 ? 6 : 2); ++c) {
              const uint32_t pp = PARTS == 3 ? kPairA >> 2 * c & 3 : 1 - c, vp = PARTS == 3 ? kPairB >> 2 * c & 3 : 0;
#pragma unroll
              for (int x = 0; x < kCh / 16; ++x)
                mma_ta(tmem + C::intra + C::half * (x / 4), tmem + (pp == 2 ? C::p2 + 8 * x : C::p + 16 * x + 8 * pp),
                       desc_mn(va + vp * L::kPlaneV + 16 * x * 128, kCh * 128), id_pv, c > 0 || (PARTS == 3 ? x % 4 : x) > 0);
            }
            commit(&o_done);
            if constexpr (!STAGED) commit(&v_empty[sv]);
          }
          __syncwarp();
        }
      }
    }
    if (!alive) give_up();
    // shared and tensor memory are released only once the MMAs issued are done
    if (issuer) commit(&drained);
    __syncwarp();
    bar_wait(&drained, 0, kDrainLimit);
  } else {
    // ------------------------------------------------------------ TMA
    // A chunk's loads go out as soon as the tiles' last readers are done, over the ends
    // of tasks: walks ahead (wk: chunks whose K and Q were asked for, wv_: V), behind
    // them the walk of the outputs (wo).
    const bool issuer = elect_one();
    struct Walk {
      int i, c, j;                                           // task, its chunk, the CTA's chunk
      LaTask k;
    };
    auto settle = [&](Walk& w) {                             // on to a task with a chunk left
      while (w.i < tasks && w.c >= w.k.nch) {
        w.i += gridDim.x;
        w.c = 0;
        if (w.i < tasks) w.k = la_task<OUT, PARTS>(s, p, a, w.i);
      }
    };
    auto next = [&](Walk& w) {
      ++w.c;
      ++w.j;
      settle(w);
    };
    Walk wk{(int)blockIdx.x, 0, 0, la_task<OUT, PARTS>(s, p, a, min((int)blockIdx.x, tasks - 1))};
    settle(wk);
    Walk wv_ = wk, wo = wk;
    auto load = [&](unsigned char* dst, int D, const CUtensorMap& map, uint64_t* bar, const Walk& w, int x0, int zb, int zh) {
      if (issuer) {
        bar_expect(bar, PARTS * D * 2 * kCh);
        for (int part = 0; part < PARTS; ++part)
          for (int d = 0; d < D; d += 64)
            tma_4d(dst + (part * D + d) / 64 * (kCh * 128), &map, bar, x0 + d, part * s.n + (int)w.k.t0 + w.c * kCh, zb, zh);
      }
      __syncwarp();
    };
    auto load_v = [&]() {
      load(vs + (wv_.j % NV) * L::kTileV, DV, vmap, &v_full[wv_.j % NV], wv_, wv_.k.v0, wv_.k.b * mul.vb, wv_.k.h * mul.vh);
      next(wv_);
    };
    auto load_k = [&]() {
      load(ks + (wk.j % NKQ) * L::kTileK, DK, kmap, &k_full[wk.j % NKQ], wk, 0, wk.k.b * mul.kb, wk.k.h * mul.kh);
    };
    auto load_q = [&]() {
      load(qs + (wk.j % NKQ) * L::kTileK, DK, qmap, &q_full[wk.j % NKQ], wk, 0, wk.k.b * mul.qb, wk.k.h * mul.qh);
    };
    for (int c = 0; c < NV; ++c) {
      if (wv_.i < tasks) load_v();
      if (c < NKQ && wk.i < tasks) {
        load_k();
        if constexpr (OUT) load_q();
        next(wk);
      }
    }
    for (; wo.i < tasks && alive; next(wo)) {                // what follows chunk wo.j
      const int j = wo.j;
      if (wk.i < tasks) {                                    // chunk j + NKQ
        // both before either is asked for: the copies that are waited for at the end are
        // those of whole chunks
        alive = wait(&k_empty[j % NKQ], (j / NKQ) & 1);
        if constexpr (OUT) alive = alive && wait(&q_empty[j % NKQ], (j / NKQ) & 1);
        if (!alive) break;
        load_k();
        if constexpr (OUT) load_q();
        next(wk);
      }
      if constexpr (STAGED) {
        alive = wait(&o_staged, j & 1);
        if (!alive) break;
        if (issuer && tile_out && !(wo.k.ragged && wo.c == wo.k.nch - 1)) {
          for (int d = 0; d < DV; d += 64)
            tma_store_4d(&omap, vs + (j % NV) * L::kTileV + (d / 64) * (kCh * 128), d, (int)wo.k.t0 + wo.c * kCh, wo.k.b, wo.k.h);
          bulk_commit();
          bulk_wait_read();                                  // the tile may be loaded into again
        }
        __syncwarp();
        if (wv_.i < tasks) load_v();                         // chunk j + NV
      } else if (wv_.i < tasks) {
        alive = wait(&v_empty[j % NV], (j / NV) & 1);
        if (!alive) break;
        load_v();
      }
    }
    if (!alive) give_up();
    // no copy of this CTA may still be in flight when it ends
    if (issuer) bulk_wait();
    __syncwarp();
    for (int x = max(0, wv_.j - NV); x < wv_.j; ++x) bar_wait(&v_full[x % NV], (x / NV) & 1, kDrainLimit);
    for (int x = max(0, wk.j - NKQ); x < wk.j; ++x) {
      bar_wait(&k_full[x % NKQ], (x / NKQ) & 1, kDrainLimit);
      if constexpr (OUT) bar_wait(&q_full[x % NKQ], (x / NKQ) & 1, kDrainLimit);
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 0) tmem_free(tmem, 512);
}

// Whether a tensor map can describe x: 16-byte aligned address and strides; a
// stride of 0 is one shared element, which positions cannot be.
bool mappable(const void* x, const int64_t (&st)[3], const LaShape& s) {
  const int64_t count[3] = {s.n, s.B, s.H};
  if ((uintptr_t)x & 15) return false;
  for (int i = 0; i < 3; ++i)
    if (count[i] > 1 && (st[i] % 8 != 0 || st[i] * 2 >= ((int64_t)1 << 40) || (i == 0 && st[i] == 0))) return false;
  return true;
}
bool map_heads(CUtensorMap* map, const void* x, const int64_t (&st)[3], const LaShape& s, int parts, int d, int* mb, int* mh) {
  *mb = s.B > 1 && st[1] != 0;
  *mh = s.H > 1 && st[2] != 0;
  const int64_t rows = (int64_t)parts * s.n;
  const uint64_t dims[4] = {(uint64_t)d, (uint64_t)rows, *mb ? (uint64_t)s.B : 1, *mh ? (uint64_t)s.H : 1};
  const uint64_t strides[3] = {rows > 1 ? (uint64_t)st[0] * 2 : 256, *mb ? (uint64_t)st[1] * 2 : 256, *mh ? (uint64_t)st[2] * 2 : 256};
  const uint32_t box[4] = {64, (uint32_t)kCh, 1, 1};
  return encode_map(map, x, 4, dims, strides, box);
}

// Inputs that no tensor map describes, and fp32 ones, as bf16 parts [part][n][B][H][d
// rounded up to 8]: 8 elements per thread. I: what counts them (64-bit divisions cost
// more than the memory accesses).
struct LaOperand {
  const void* src;
  __nv_bfloat16* dst;
  int64_t st[3];
  int d, vec;            // vec: rows start at 16-byte boundaries
};
struct LaOperands {
  LaOperand x[3];
  int64_t end[3];        // units of 8 elements up to and with each
};
template <typename T, typename I>
__global__ void __launch_bounds__(256) k_linattn_layout(LaOperands ops, int B, int H, int64_t rows) {
  pdl_launch_dependents();                 // the attention itself, which waits for this launch's end
  pdl_wait_primary();
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < ops.end[2]; u += (int64_t)gridDim.x * 256) {
    const int i = u < ops.end[0] ? 0 : u < ops.end[1] ? 1 : 2;
    const LaOperand& o = ops.x[i];
    const I v = (I)(i ? u - ops.end[i - 1] : u), per = (I)((o.d + 7) / 8);
    const I r = v / per;                   // (position, sequence, head)
    const I tb = r / (I)H, t = tb / (I)B;
    const int64_t h = r - tb * (I)H, b = tb - t * (I)B;
    const int k = (int)(v - r * per) * 8;
    const T* p = (const T*)o.src + (int64_t)t * o.st[0] + b * o.st[1] + h * o.st[2] + k;
    __nv_bfloat16* d = o.dst + (int64_t)r * (8 * (int)per) + k;
    if constexpr (sizeof(T) == 2) {
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k + e < o.d) w[e / 2] |= (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p) + e) << (16 * (e & 1));
      *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      float f[8];
      if (o.vec && k + 8 <= o.d) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(p)), y = __ldg(reinterpret_cast<const float4*>(p) + 1);
        f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
        f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = k + e < o.d ? __ldg(p + e) : 0.f;
      }
      uint32_t q[3][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split3(f[2 * e], f[2 * e + 1], q[0][e], q[1][e], q[2][e]);
#pragma unroll
      for (int x = 0; x < 3; ++x)
        *reinterpret_cast<uint4*>(d + x * rows * (8 * (int)per)) = make_uint4(q[x][0], q[x][1], q[x][2], q[x][3]);
    }
  }
}

// 16-byte address and strides of the dimensions that are stepped over.
bool aligned_heads(const void* x, const int64_t (&st)[3], const LaShape& s) {
  const int e = s.bf16 ? 8 : 4;
  const int64_t count[3] = {s.n, s.B, s.H};
  if ((uintptr_t)x & 15) return false;
  for (int i = 0; i < 3; ++i)
    if (count[i] > 1 && st[i] % e != 0) return false;
  return true;
}

template <int DK, int DV, int PARTS, bool ADD = false>
cudaError_t run(const LaShape& s, const LaPlan& p, const LaPtrs& a, int num_sms, cudaStream_t st) {
  CUtensorMap qm, km, vm, om{};
  LaMul mul{};
  int ob, oh;
  if (!map_heads(&qm, a.q, s.qs, s, PARTS, s.dk, &mul.qb, &mul.qh) || !map_heads(&km, a.k, s.ks, s, PARTS, s.dk, &mul.kb, &mul.kh) ||
      !map_heads(&vm, a.v, s.vs, s, PARTS, s.dv, &mul.vb, &mul.vh))
    return cudaErrorInvalidValue;
  const int vec_out = PARTS == 1 ? mappable(a.o, s.os, s) && map_heads(&om, a.o, s.os, s, 1, s.dv, &ob, &oh)
                                 : aligned_heads(a.o, s.os, s);
  const int tile_out = PARTS == 1 && vec_out && s.dv % 8 == 0;
  const int vec_state = s.dv % 4 == 0 && s.state_ld % 4 == 0 && ((uintptr_t)a.state_in & 15) == 0 && ((uintptr_t)a.state_out & 15) == 0;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int tasks = s.B * s.H * (PARTS == 3 ? (s.dv + 63) / 64 : 1) * p.G;
  cfg.gridDim = dim3((unsigned)(tasks < num_sms ? tasks : num_sms));
  cfg.blockDim = dim3(kLaTcThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (p.G > 1) {
    constexpr auto kern = k_linattn_tc<DK, DV, false, PARTS, false>;
    cfg.dynamicSmemBytes = LaSmem<DK, DV, false, PARTS>::bytes;
    if ((e = allow_smem<kern>(cfg.dynamicSmemBytes)) != cudaSuccess) return e;
    if ((e = cudaLaunchKernelEx(&cfg, kern, s, p, a, qm, km, vm, om, mul, vec_out, tile_out, vec_state, op_wait_limit())) != cudaSuccess)
      return e;
  }
  constexpr auto kern = k_linattn_tc<DK, DV, true, PARTS, ADD>;
  cfg.dynamicSmemBytes = LaSmem<DK, DV, true, PARTS>::bytes;
  if ((e = allow_smem<kern>(cfg.dynamicSmemBytes)) != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, kern, s, p, a, qm, km, vm, om, mul, vec_out, tile_out, vec_state, op_wait_limit());
}

size_t operand_bytes(const LaShape& s, int d) {
  return ((size_t)(s.bf16 ? 1 : 3) * s.n * s.B * s.H * ((d + 7) / 8 * 8) * 2 + 255) / 256 * 256;
}

}  // namespace

bool linattn_tc_fits(const LaShape& s) {
  return !s.bf16 || (s.dk <= 128 && s.dv <= 128);
}

// What fp32 launches work on: tiles fit shared memory up to 64 dimensions, blocks of value
// dimensions are like heads of their own, those of key dimensions follow one another.
LaShape linattn_tc_block(const LaShape& s) {
  LaShape b = s;
  if (s.bf16) return b;
  b.H *= (s.dv + 63) / 64;
  b.dk = s.dk < 64 ? s.dk : 64;
  b.dv = s.dv < 64 ? s.dv : 64;
  return b;
}

size_t linattn_tc_layout_bytes(const LaShape& s, const LaPtrs& a) {
  size_t n = 0;
  if (!s.bf16 || !mappable(a.q, s.qs, s)) n += operand_bytes(s, s.dk);
  if (!s.bf16 || !mappable(a.k, s.ks, s)) n += operand_bytes(s, s.dk);
  if (!s.bf16 || !mappable(a.v, s.vs, s)) n += operand_bytes(s, s.dv);
  return n;
}

// Segments: a CTA fills an SM, so B x H x G CTAs run in rounds of num_sms; the
// launch that forms the segments' states does about half the work of the other
// over all but the last segment. The G of least total time, in chunks.
LaPlan linattn_tc_plan(const LaShape& s, int num_sms) {
  const int64_t chunks = ((int64_t)s.n + kCh - 1) / kCh, bh = (int64_t)s.B * s.H;
  auto rounds = [&](int64_t ctas) { return (ctas + num_sms - 1) / num_sms; };
  int64_t best = 1;
  double least = 0;
  for (int64_t G = 1; G <= 64 && G <= chunks; ++G) {
    const int64_t c = (chunks + G - 1) / G;
    if ((chunks + c - 1) / c != G) continue;               // the same segments as a smaller G
    // each launch and each CTA's start costs about two chunks' time
    double t = (double)(rounds(bh * G) * (c + 2));
    if (G > 1) t += 0.5 * (double)(rounds(bh * (G - 1)) * (c + 2)) + 2;
    if (G == 1 || t < least) {
      least = t;
      best = G;
    }
  }
  const int64_t c = chunks > 0 ? (chunks + best - 1) / best : 1;
  return LaPlan{(int)best, (int)(c * kCh)};
}

cudaError_t launch_linattn_tc(const LaShape& shape, const LaPlan& p, const LaPtrs& ptrs, void* layout, int num_sms,
                              cudaStream_t st) {
  LaShape s = shape;
  LaPtrs a = ptrs;
  LaOperands ops{};
  unsigned char* at = (unsigned char*)layout;
  int64_t units = 0;
  int n = 0;
  const int64_t rows = (int64_t)s.n * s.B * s.H;
  auto lay = [&](const void*& x, int64_t (&xs)[3], int d) {
    if (s.bf16 && mappable(x, xs, s)) return;
    LaOperand& o = ops.x[n];
    o = LaOperand{x, (__nv_bfloat16*)at, {xs[0], xs[1], xs[2]}, d, aligned_heads(x, xs, s)};
    units += rows * ((d + 7) / 8);
    ops.end[n++] = units;
    at += operand_bytes(s, d);
    x = o.dst;
    xs[2] = (d + 7) / 8 * 8;
    xs[1] = xs[2] * s.H;
    xs[0] = xs[1] * s.B;
  };
  lay(a.q, s.qs, s.dk);
  lay(a.k, s.ks, s.dk);
  lay(a.v, s.vs, s.dv);
  if (n > 0) {
    for (int i = n; i < 3; ++i) ops.end[i] = units;
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
        s.bf16 ? cudaLaunchKernelEx(&cfg, narrow ? k_linattn_layout<__nv_bfloat16, uint32_t> : k_linattn_layout<__nv_bfloat16, uint64_t>,
                                    ops, s.B, s.H, rows)
               : cudaLaunchKernelEx(&cfg, narrow ? k_linattn_layout<float, uint32_t> : k_linattn_layout<float, uint64_t>, ops, s.B,
                                    s.H, rows);
    if (e != cudaSuccess) return e;
  }
  s.state_slot = (int64_t)s.dk * s.dv;
  s.state_ld = s.dv;
  if (!s.bf16) {
    // q . k is the sum over blocks of key dimensions, and so are the outputs (each block after
    // the first adds to them); the state's blocks are apart
    for (int k0 = 0; k0 < s.dk; k0 += 64) {
      LaShape t = s;
      LaPtrs b = a;
      t.dk = s.dk - k0 < 64 ? s.dk - k0 : 64;
      b.q = (const __nv_bfloat16*)a.q + k0;
      b.k = (const __nv_bfloat16*)a.k + k0;
      if (a.state_in) b.state_in = a.state_in + (size_t)k0 * s.dv;
      if (a.state_out) b.state_out = a.state_out + (size_t)k0 * s.dv;
      const cudaError_t e = k0 == 0 ? run<64, 64, 3>(t, p, b, num_sms, st) : run<64, 64, 3, true>(t, p, b, num_sms, st);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
  if (s.dk <= 64) return s.dv <= 64 ? run<64, 64, 1>(s, p, a, num_sms, st) : run<64, 128, 1>(s, p, a, num_sms, st);
  return s.dv <= 64 ? run<128, 64, 1>(s, p, a, num_sms, st) : run<128, 128, 1>(s, p, a, num_sms, st);
}

cudaError_t linattn_take_error(cudaStream_t st, int* flag) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(flag, g_linattn_error, sizeof(int), 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && *flag) {
    const int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_linattn_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  return e;
}

}  // namespace fi
