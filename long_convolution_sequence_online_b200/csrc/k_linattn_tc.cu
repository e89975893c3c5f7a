// Linear attention over prompts on the 5th-generation tensor cores: the chunked
// form (k_linattn.cu) with chunks of 128 positions, bf16 inputs by TMA,
// accumulators in tensor memory.
//
// One CTA runs the chunks of a segment of one (sequence, head) in order. Per
// chunk, with Q, K, V the 128-row tiles and S the state before it:
//     scores = Q K^T            -> P = scores * g^{i-j} for j <= i (bf16, in place)
//     inter  = Q S              (S rounded to bf16 as an operand)
//     intra  = P V              (P read from tensor memory)
//     KV     = K^T (w V)        w_j = g^{m-1-j}, w V as three bf16 parts
//     S     <- g^m S + KV       (fp32, in registers)
//     o      = scale (g^{i+1} inter + intra)
// Roundings below fp32: the result, P, and S where it enters Q S. P and S are
// rounded once each to the results' own type, so each adds an error of the size
// of the result's own rounding. The state itself must stay an fp32 sum, so w V
// is not rounded: three parts hold all 24 bits of it, the products with the
// bf16 K are exact, and every chunk's KV is accumulated on its own (the tensor
// core's sums are not rounded to nearest) and added to S in registers.
//
// Warps: 0-3 scores -> P, then the outputs; 4-11 the state; 12-15 w V; 16 issues
// the MMAs; 17 the TMA copies. Everything is handed over by mbarriers, so the
// MMAs of one chunk, the copies of the next and the warps' arithmetic overlap.
#include "op_internal.cuh"
#include "tc.cuh"

namespace fi {

namespace {

using namespace tc;

constexpr int kCh = 128;                 // positions per chunk
constexpr int kWHalf = 64;               // positions of w V in shared memory at a time
constexpr int kSlots = 4;                // tiles of Q, K, V in flight
constexpr int kOutWarps = 4, kStateWarps = 8, kScaleWarps = 4;
constexpr int kMmaWarp = kOutWarps + kStateWarps + kScaleWarps, kTmaWarp = kMmaWarp + 1;
constexpr int kLaTcThreads = 32 * (kTmaWarp + 1);

__device__ int g_linattn_error;          // a bounded wait gave up since the last check

// DK, DV: key and value dimensions padded to 64 or 128.
template <int DK, int DV>
struct LaSmem {
  static constexpr int kTileK = kCh * 2 * DK, kTileV = kCh * 2 * DV;
  static constexpr int kSlot = kTileK > kTileV ? kTileK : kTileV;
  static constexpr int kPart = kWHalf * 2 * DV;
  static constexpr int kState = DK * 2 * DV;
  static constexpr size_t bytes = 1024 + (size_t)kSlots * kSlot + 3 * kPart + kState;
};

// Coordinates of a tensor map [dim][position][sequence][head]; a stride of 0
// becomes a dimension of 1 and a coordinate of 0.
struct LaMul {
  int qb, qh, kb, kh, vb, vh;
};

// TMEM columns.
constexpr uint32_t kColP = 0, kColInter = 128, kColIntra = 256, kColKV = 384;

template <int DK, int DV, bool OUT>
__global__ void __launch_bounds__(kLaTcThreads, 1)
k_linattn_tc(LaShape s, LaPlan p, LaPtrs a, const __grid_constant__ CUtensorMap qmap,
             const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, LaMul mul, int vec_out,
             int vec_state, int wait_limit) {
  using L = LaSmem<DK, DV>;
  constexpr int TILES = OUT ? 3 : 2;     // per chunk: K, (Q,) V
  extern __shared__ unsigned char raw_smem[];
  __shared__ uint64_t full[kSlots], empty[kSlots], qk_done, p_ready, o_done, o_free, w_ready, w_free, kv_done, s_ready, fixed, drained;
  __shared__ float G[kCh + 1];           // g^0 .. g^128
  __shared__ __align__(16) float GR[32]; // g^31 .. g^0
  __shared__ uint32_t tmem_s;
  __shared__ int abort_s;
  unsigned char* slots = raw_smem + ((1024 - (saddr(raw_smem) & 1023)) & 1023);
  unsigned char* wv = slots + kSlots * L::kSlot;
  unsigned char* sop = wv + 3 * L::kPart;
  pdl_launch_dependents();
  pdl_wait_primary();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = blockIdx.x, b = bh / s.H, h = bh - b * s.H, seg = blockIdx.y;
  const int len = la_length(a.lengths, b, s.n);
  const int64_t t0 = (int64_t)seg * p.seg;
  const size_t slot = (size_t)s.dk * s.dv;
  float* ws = a.ws ? a.ws + (size_t)bh * p.G * slot : nullptr;
  const float* s_in = a.state_in ? a.state_in + (size_t)bh * slot : nullptr;
  if constexpr (!OUT) {
    if (seg == 0 && s_in)
      for (size_t e = tid; e < slot; e += kLaTcThreads) ws[e] = s_in[e];
    if (t0 + p.seg >= len) return;       // no segment after this one
  } else {
    if (t0 >= len && seg > 0) return;
  }
  const int end = (int)min((int64_t)len, t0 + p.seg);
  const int nch = (int)((end - t0 + kCh - 1) / kCh);
  const float ld2 = la_log2_decay(__ldg(a.log_decay + h));
  if (warp == 0) tmem_alloc(&tmem_s, 512);
  if (tid >= 64 && tid < 64 + kCh + 1) G[tid - 64] = la_pow(ld2, tid - 64);
  if (tid >= 256 && tid < 288) GR[tid - 256] = la_pow(ld2, 31 - (tid - 256));
  if (tid == 32) {
    for (int i = 0; i < kSlots; ++i) {
      bar_init(&full[i], 1);
      bar_init(&empty[i], 1);
    }
    bar_init(&qk_done, 1);
    bar_init(&p_ready, kOutWarps);
    bar_init(&o_done, 1);
    bar_init(&o_free, kOutWarps);
    bar_init(&w_ready, kScaleWarps);
    bar_init(&w_free, 1);
    bar_init(&kv_done, 1);
    bar_init(&s_ready, kStateWarps);
    bar_init(&fixed, kScaleWarps);
    bar_init(&drained, 1);
    abort_s = 0;
    bar_init_fence();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_s;
  volatile int* abort_flag = &abort_s;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, bar_wait(bar, parity, wait_limit, abort_flag));
  };
  auto give_up = [&]() {
    if (lane == 0) {
      *abort_flag = 1;
      atomicExch(&g_linattn_error, 1);
    }
  };
  auto tile_of = [&](int c, int which) { return c * TILES + which; };   // 0: K, 1: Q (OUT), last: V
  auto tile_at = [&](int t) { return slots + (t % kSlots) * L::kSlot; };
  // The last chunk of a sequence shorter than the batch: what stands behind its
  // end (anything, NaN too) is cleared in the tiles before they are multiplied.
  const bool ragged = end == len && len < s.n && (end - t0) % kCh != 0;

  if (warp < kOutWarps) {
    // ------------------------------------------------------------ P and the outputs
    if constexpr (OUT) {
      const int i = 32 * warp + lane;              // row of the chunk
      const uint32_t at = tmem + ((uint32_t)(32 * warp) << 16);
      bool alive = true;
      for (int c = 0; c < nch && alive; ++c) {
        const int m = min(kCh, (int)(end - t0) - c * kCh);
        alive = wait(&qk_done, c & 1);
        if (!alive) break;
        fence_after();
#pragma unroll 1
        for (int blk = 0; blk < 4; ++blk) {
          uint32_t out[16];
          if (blk <= warp) {
            uint32_t r[32];
            tmem_ld32(at + kColP + 32 * blk, r);
            ld_wait();
            if (blk < warp) {
              const float f = G[i - 32 * blk - 31];
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 g4 = *reinterpret_cast<const float4*>(&GR[e]);
                out[e / 2] = pack2(__uint_as_float(r[e]) * (f * g4.x), __uint_as_float(r[e + 1]) * (f * g4.y));
                out[e / 2 + 1] = pack2(__uint_as_float(r[e + 2]) * (f * g4.z), __uint_as_float(r[e + 3]) * (f * g4.w));
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 2)
                out[e / 2] = pack2(e <= lane ? __uint_as_float(r[e]) * G[(lane - e) & 31] : 0.f,
                                   e + 1 <= lane ? __uint_as_float(r[e + 1]) * G[(lane - e - 1) & 31] : 0.f);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) out[e] = 0;
          }
          tmem_st16(at + kColP + 16 * blk, out);
        }
        st_wait();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&p_ready);
        alive = wait(&o_done, c & 1);
        if (!alive) break;
        fence_after();
        const float fi_ = s.scale * G[i + 1], fo = s.scale;
        const int64_t t = t0 + (int64_t)c * kCh + i;
        __nv_bfloat16* op = (__nv_bfloat16*)a.o + b * s.os[1] + h * s.os[2] + t * s.os[0];
#pragma unroll 1
        for (int d = 0; d < DV; d += 32) {
          uint32_t r[32], q[32];
          tmem_ld32(at + kColInter + d, r);
          tmem_ld32(at + kColIntra + d, q);
          ld_wait();
          if (d + 32 >= DV) {
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(&o_free);
          }
          if (i < m) {
            if (vec_out) {
#pragma unroll
              for (int u = 0; u < 4; ++u)
                if (d + 8 * u < s.dv) {
                  uint32_t w[4];
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const int x = 8 * u + 2 * e;
                    w[e] = pack2(fmaf(fi_, __uint_as_float(r[x]), fo * __uint_as_float(q[x])),
                                 fmaf(fi_, __uint_as_float(r[x + 1]), fo * __uint_as_float(q[x + 1])));
                  }
                  *reinterpret_cast<uint4*>(op + d + 8 * u) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (d + e < s.dv)
                  op[d + e] = __float2bfloat16_rn(fmaf(fi_, __uint_as_float(r[e]), fo * __uint_as_float(q[e])));
            }
          }
        }
      }
      if (!alive) give_up();
    }
  } else if (warp < kOutWarps + kStateWarps) {
    // ------------------------------------------------------------ the state
    // Row 32 (warp % 4) + lane, columns [col0, + CW) of S in registers.
    constexpr int CW = DV / 2;
    const int quarter = warp & 3, half = (warp - kOutWarps) >> 2;
    const int row = 32 * quarter + lane, col0 = half * CW;
    const uint32_t at = tmem + ((uint32_t)(32 * quarter) << 16) + kColKV + col0;
    float st[CW];
#pragma unroll
    for (int e = 0; e < CW; ++e) st[e] = 0.f;
    if constexpr (OUT) {
      const float* src = p.G > 1 ? ws : s_in;
      if (src && row < s.dk)
        for (int g = s_in ? 0 : 1; g <= seg; ++g) {
          // slot 0: the state before the prompt; slot g: segment g - 1's contribution
          const float f = la_pow(ld2, (g == 0 ? seg : seg - g) * p.seg);
          const float* sp = src + (size_t)g * slot + (size_t)row * s.dv + col0;
          if (vec_state) {
#pragma unroll
            for (int e = 0; e < CW; e += 4)
              if (col0 + e < s.dv) {
                const float4 v = *reinterpret_cast<const float4*>(sp + e);
                st[e] = fmaf(f, v.x, st[e]);
                st[e + 1] = fmaf(f, v.y, st[e + 1]);
                st[e + 2] = fmaf(f, v.z, st[e + 2]);
                st[e + 3] = fmaf(f, v.w, st[e + 3]);
              }
          } else {
#pragma unroll
            for (int e = 0; e < CW; ++e)
              if (col0 + e < s.dv) st[e] = fmaf(f, sp[e], st[e]);
          }
        }
    }
    // S as the B operand of Q S: rows of 64 bf16 columns, 128-byte swizzle.
    auto publish = [&]() {
      if constexpr (OUT) {
        if (row < DK) {
#pragma unroll
          for (int e = 0; e < CW; e += 8) {
            const int col = col0 + e, unit = (col & 63) >> 3;
            unsigned char* dst = sop + (col >> 6) * (DK * 128) + row * 128 + ((unit ^ (row & 7)) << 4);
            *reinterpret_cast<uint4*>(dst) = make_uint4(pack2(st[e], st[e + 1]), pack2(st[e + 2], st[e + 3]),
                                                        pack2(st[e + 4], st[e + 5]), pack2(st[e + 6], st[e + 7]));
          }
        }
        fence_async();
      }
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&s_ready);
    };
    publish();
    bool alive = true;
    for (int c = 0; c < nch && alive; ++c) {
      const int m = min(kCh, (int)(end - t0) - c * kCh);
      alive = wait(&kv_done, c & 1);
      if (!alive) break;
      fence_after();
      const float gm = G[m];
#pragma unroll
      for (int e = 0; e < CW; e += 32) {
        uint32_t r[32];
        tmem_ld32(at + e, r);
        ld_wait();
#pragma unroll
        for (int x = 0; x < 32; ++x) st[e + x] = fmaf(gm, st[e + x], __uint_as_float(r[x]));
      }
      publish();
    }
    if (!alive) give_up();
    float* dst = nullptr;
    if constexpr (!OUT) dst = ws + (size_t)(seg + 1) * slot;
    else if (a.state_out && end == len) dst = a.state_out + (size_t)bh * slot;   // this segment holds the last position
    if (dst && row < s.dk) {
      dst += (size_t)row * s.dv + col0;
      if (vec_state) {
#pragma unroll
        for (int e = 0; e < CW; e += 4)
          if (col0 + e < s.dv) *reinterpret_cast<float4*>(dst + e) = make_float4(st[e], st[e + 1], st[e + 2], st[e + 3]);
      } else {
#pragma unroll
        for (int e = 0; e < CW; ++e)
          if (col0 + e < s.dv) dst[e] = st[e];
      }
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------------------ w V as three bf16 parts
    const int lt = tid - 32 * (kOutWarps + kStateWarps);   // 0..127
    constexpr int UNITS = kWHalf * DV / 8 / (32 * kScaleWarps);   // 16-byte units per thread and half
    bool alive = true;
    for (int c = 0; c < nch && alive; ++c) {
      const int m = min(kCh, (int)(end - t0) - c * kCh);
      const int tv = tile_of(c, TILES - 1), tk = tile_of(c, 0);
      unsigned char* v = tile_at(tv);
      alive = wait(&full[tv % kSlots], (tv / kSlots) & 1);
      if (!alive) break;
      if (ragged && c == nch - 1) {
        alive = wait(&full[tk % kSlots], (tk / kSlots) & 1);
        if (!alive) break;
        unsigned char* k = tile_at(tk);
        for (int e = lt; e < kCh * 8; e += 32 * kScaleWarps) {   // 16-byte units of a 64-column block
          if ((e >> 3) < m) continue;
          for (int d = 0; d < DK / 64; ++d) *reinterpret_cast<uint4*>(k + d * (kCh * 128) + e * 16) = make_uint4(0, 0, 0, 0);
          for (int d = 0; d < DV / 64; ++d) *reinterpret_cast<uint4*>(v + d * (kCh * 128) + e * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_async();
        asm volatile("bar.sync 1, %0;" ::"r"(32 * kScaleWarps) : "memory");
        if (lane == 0) bar_arrive(&fixed);
      }
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const int use = 2 * c + half;
        if (use > 0) {
          alive = wait(&w_free, (use - 1) & 1);
          if (!alive) break;
        }
#pragma unroll 4
        for (int u = 0; u < UNITS; ++u) {
          const int e = lt + u * (32 * kScaleWarps);       // unit of the half tile: 64-column block, row, unit
          const int blk = e / (kWHalf * 8), rem = e & (kWHalf * 8 - 1), row = half * kWHalf + (rem >> 3);
          const uint4 x = *reinterpret_cast<const uint4*>(v + blk * (kCh * 128) + half * (kWHalf * 128) + rem * 16);
          const float w = row < m ? G[m - 1 - row] : 0.f;
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
          uint32_t q0[4], q1[4], q2[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) split3(w * lo_f(xs[i]), w * hi_f(xs[i]), q0[i], q1[i], q2[i]);
          unsigned char* dst = wv + blk * (kWHalf * 128) + rem * 16;
          *reinterpret_cast<uint4*>(dst) = make_uint4(q0[0], q0[1], q0[2], q0[3]);
          *reinterpret_cast<uint4*>(dst + L::kPart) = make_uint4(q1[0], q1[1], q1[2], q1[3]);
          *reinterpret_cast<uint4*>(dst + 2 * L::kPart) = make_uint4(q2[0], q2[1], q2[2], q2[3]);
        }
        fence_async();
        __syncwarp();
        if (lane == 0) bar_arrive(&w_ready);
      }
    }
    if (!alive) give_up();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    const bool issuer = elect_one();
    constexpr uint32_t id_qk = idesc(128, 128), id_qs = idesc(128, DV, false, true), id_pv = idesc(128, DV, false, true),
                       id_kv = idesc(128, DV, true, true);
    const uint32_t wa = saddr(wv), sa = saddr(sop);
    bool alive = true;
    // K^T (w V) over half of the chunk, smallest parts first; rows 64..127 of a
    // 64-dimensional K repeat the first ones and are not read.
    auto kv_half = [&](int c, int half) {
      const uint32_t ka = saddr(tile_at(tile_of(c, 0)));
      if (!wait(&w_ready, half)) return false;             // uses 2c + half
      fence_after();
      if (issuer) {
#pragma unroll
        for (int part = 2; part >= 0; --part)
#pragma unroll
          for (int k = 0; k < kWHalf / 16; ++k)
            mma(tmem + kColKV, desc_mn(ka + (half * kWHalf + 16 * k) * 128, DK == 128 ? kCh * 128 : 0),
                desc_mn(wa + part * L::kPart + 16 * k * 128, kWHalf * 128), id_kv, half > 0 || part < 2 || k > 0);
        commit(&w_free);
        if (half == 1) commit(&kv_done);
      }
      __syncwarp();
      return true;
    };
    for (int c = 0; c < nch && alive; ++c) {
      const int tk = tile_of(c, 0), tv = tile_of(c, TILES - 1);
      alive = wait(&full[tk % kSlots], (tk / kSlots) & 1);
      if (alive && ragged && c == nch - 1) alive = wait(&fixed, 0);
      if (!alive) break;
      if constexpr (OUT) {
        const int tq = tile_of(c, 1);
        // the scores replace P, which the product before reads
        alive = wait(&full[tq % kSlots], (tq / kSlots) & 1) && (c == 0 || wait(&o_done, (c - 1) & 1));
        if (!alive) break;
        fence_after();
        const uint32_t ka = saddr(tile_at(tk)), qa = saddr(tile_at(tq)), va = saddr(tile_at(tv));
        if (issuer) {
#pragma unroll
          for (int k = 0; k < DK / 16; ++k) {
            const uint32_t o = (k / 4) * (kCh * 128) + (k % 4) * 32;
            mma(tmem + kColP, desc_k(qa + o), desc_k(ka + o), id_qk, k > 0);
          }
          commit(&qk_done);
        }
        __syncwarp();
        alive = wait(&s_ready, c & 1) && (c == 0 || wait(&o_free, (c - 1) & 1));
        if (!alive) break;
        fence_after();
        if (issuer) {
#pragma unroll
          for (int k = 0; k < DK / 16; ++k)
            mma(tmem + kColInter, desc_k(qa + (k / 4) * (kCh * 128) + (k % 4) * 32), desc_mn(sa + 16 * k * 128, DK * 128),
                id_qs, k > 0);
          commit(&empty[tq % kSlots]);
        }
        __syncwarp();
        alive = kv_half(c, 0) && wait(&p_ready, c & 1);
        if (!alive) break;
        fence_after();
        if (issuer) {
#pragma unroll
          for (int k = 0; k < kCh / 16; ++k)
            mma_ta(tmem + kColIntra, tmem + kColP + 8 * k, desc_mn(va + 16 * k * 128, kCh * 128), id_pv, k > 0);
          commit(&o_done);
        }
        __syncwarp();
      } else {
        alive = wait(&s_ready, c & 1) && kv_half(c, 0);
        if (!alive) break;
      }
      alive = kv_half(c, 1);
      if (!alive) break;
      if (issuer) {
        commit(&empty[tk % kSlots]);
        commit(&empty[tv % kSlots]);
      }
      __syncwarp();
    }
    if (!alive) give_up();
    // shared and tensor memory are released only once the MMAs issued are done
    if (issuer) commit(&drained);
    __syncwarp();
    bar_wait(&drained, 0, kDefaultWaitLimit);
  } else {
    // ------------------------------------------------------------ TMA producer
    const bool issuer = elect_one();
    bool alive = true;
    int t = 0;
    const int total = nch * TILES;
    for (; t < total && alive; ++t) {
      const int c = t / TILES, which = t - c * TILES, sl = t % kSlots;
      if (t >= kSlots) {
        alive = wait(&empty[sl], (t / kSlots - 1) & 1);
        if (!alive) break;
      }
      if (issuer) {
        const int pos = (int)t0 + c * kCh;
        unsigned char* dst = tile_at(t);
        const bool is_v = which == TILES - 1, is_k = which == 0;
        const int D = is_v ? DV : DK;
        bar_expect(&full[sl], D * 2 * kCh);
        const CUtensorMap* map = is_v ? &vmap : is_k ? &kmap : &qmap;
        const int mb = is_v ? mul.vb : is_k ? mul.kb : mul.qb, mh = is_v ? mul.vh : is_k ? mul.kh : mul.qh;
        for (int d = 0; d < D; d += 64) tma_4d(dst + (d / 64) * (kCh * 128), map, &full[sl], d, pos, b * mb, h * mh);
      }
      __syncwarp();
    }
    if (!alive) give_up();
    // no copy of this CTA may still be in flight when it ends
    for (int i = t > kSlots ? t - kSlots : 0; i < t; ++i) bar_wait(&full[i % kSlots], (i / kSlots) & 1, kDefaultWaitLimit);
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
bool map_heads(CUtensorMap* map, const void* x, const int64_t (&st)[3], const LaShape& s, int d, int* mb, int* mh) {
  *mb = s.B > 1 && st[1] != 0;
  *mh = s.H > 1 && st[2] != 0;
  const uint64_t dims[4] = {(uint64_t)d, (uint64_t)s.n, *mb ? (uint64_t)s.B : 1, *mh ? (uint64_t)s.H : 1};
  const uint64_t strides[3] = {s.n > 1 ? (uint64_t)st[0] * 2 : 256, *mb ? (uint64_t)st[1] * 2 : 256, *mh ? (uint64_t)st[2] * 2 : 256};
  const uint32_t box[4] = {64, (uint32_t)kCh, 1, 1};
  return encode_map(map, x, 4, dims, strides, box);
}

template <int DK, int DV>
cudaError_t run(const LaShape& s, const LaPlan& p, const LaPtrs& a, cudaStream_t st) {
  constexpr size_t smem = LaSmem<DK, DV>::bytes;
  CUtensorMap qm, km, vm;
  LaMul mul{};
  if (!map_heads(&qm, a.q, s.qs, s, s.dk, &mul.qb, &mul.qh) || !map_heads(&km, a.k, s.ks, s, s.dk, &mul.kb, &mul.kh) ||
      !map_heads(&vm, a.v, s.vs, s, s.dv, &mul.vb, &mul.vh))
    return cudaErrorInvalidValue;
  const bool out16 = ((uintptr_t)a.o & 15) == 0 && s.dv % 8 == 0 && (s.n == 1 || s.os[0] % 8 == 0) &&
                     (s.B == 1 || s.os[1] % 8 == 0) && (s.H == 1 || s.os[2] % 8 == 0);
  const bool state16 = s.dv % 4 == 0 && ((uintptr_t)a.state_in & 15) == 0 && ((uintptr_t)a.state_out & 15) == 0;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(s.B * s.H), (unsigned)p.G);
  cfg.blockDim = dim3(kLaTcThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (p.G > 1) {
    if ((e = allow_smem<k_linattn_tc<DK, DV, false>>(smem)) != cudaSuccess) return e;
    if ((e = cudaLaunchKernelEx(&cfg, k_linattn_tc<DK, DV, false>, s, p, a, qm, km, vm, mul, (int)out16, (int)state16,
                                (int)kDefaultWaitLimit)) != cudaSuccess)
      return e;
  }
  if ((e = allow_smem<k_linattn_tc<DK, DV, true>>(smem)) != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, k_linattn_tc<DK, DV, true>, s, p, a, qm, km, vm, mul, (int)out16, (int)state16,
                            (int)kDefaultWaitLimit);
}

}  // namespace

bool linattn_tc_fits(const LaShape& s, const LaPtrs& a) {
  return s.bf16 && s.n > 0 && s.dk <= 128 && s.dv <= 128 && mappable(a.q, s.qs, s) && mappable(a.k, s.ks, s) &&
         mappable(a.v, s.vs, s);
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

cudaError_t launch_linattn_tc(const LaShape& s, const LaPlan& p, const LaPtrs& a, cudaStream_t st) {
  if (s.dk <= 64) return s.dv <= 64 ? run<64, 64>(s, p, a, st) : run<64, 128>(s, p, a, st);
  return s.dv <= 64 ? run<128, 64>(s, p, a, st) : run<128, 128>(s, p, a, st);
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
