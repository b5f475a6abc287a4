// Decode of one new token per sequence over a paged cache in bf16 (sm_100a).
//
// A step reads every visible key and value once and does little with each:
// 2 GS products per element for GS query heads, far below what the memory
// system lets through, so the kernel is built around an unbroken stream of
// tiles.  The GPU's whole work is one list of 64-key tiles, cut into equal
// runs, one per SM; a CTA goes through its run with one ring of TMA stages
// that is not drained between sequences or heads (jl_paged.cuh has the plan).
//
//   warp 8     producer: looks the pages of the next tiles up and loads their
//              K and V by TMA (SWIZZLE_128B boxes of up to 64 rows; a tile of
//              16-key pages is four boxes of each).
//   warps 9-10 angles: the bifocal turn n(j0) - n(i) of each 16-key block's
//              first key: cosine and sine per channel pair.
//   warps 0-7  16 keys of every second tile each: scores, weights and weighted
//              values, with the warp's own running maximum and sum; merged when
//              the run leaves a (sequence, kv head).
//
// Products are m16n8k16 in registers: keys x channels by channels x heads for
// the scores, channels x keys by keys x heads for the outputs.  They need neither
// tensor memory nor a trip of the turned keys through shared memory: a key's
// channel k and its partner k + D/2 sit in the same lane (the operand of step x
// and that of step x + D/32), so the rotation happens on the operand's own
// registers.  At the memory's pace a tile leaves an SM some 1400 cycles.
//
// Precision: turned keys are split into two bf16, hi + lo, and both are
// multiplied, so they are held to 2^-17; softmax weights are split into three,
// which hold all their bits (three for the keys as well: 124 us against 112 at
// 128K); scores, maxima, sums and outputs are fp32.
#include "jl_paged.cuh"
#include "jl_ptx.cuh"

namespace jl {
namespace pgt {

constexpr int NCW = 8;                      // consumer warps
constexpr int WARP_LOAD = NCW, WARP_ANGLE = NCW + 1;
constexpr int THREADS = (NCW + 3) * 32;
constexpr int CTAS = 148;
constexpr int ERR_TIMEOUT = 64;
constexpr int NBLK = PD_TILE / PD_BLK;      // 16-key blocks of a tile
constexpr float LN2 = 0.69314718055994531f;

template <int D>
struct Geo {
  static constexpr int HALF = D / 2;
  static constexpr int NH = D / 64;                    // 64-channel boxes of a row
  static constexpr int KV = PD_TILE * D * 2;           // K or V of a tile
  // Ring stages: an even number, so that a stage's tiles all go to the same four
  // consumer warps.  (With an odd one the two groups take turns on a stage, a
  // group sees every second phase of its barrier only, and the parity it waits
  // for is already true while the other group's load is still under way.)
  static constexpr int NST = D == 128 ? 4 : 10;
  static_assert(NST % 2 == 0, "a stage belongs to one consumer group");
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = NST * KV;
  static constexpr int ANG = NBLK * HALF * 8;          // a stage's angles
  static constexpr int OFF_ANG = 2 * NST * KV;
  static constexpr int OFF_TAB = OFF_ANG + NST * ANG;  // turns by 0 .. 15 positions
  static constexpr int OFF_RED = OFF_TAB + PD_BLK * HALF * 8;
  static constexpr int RS = D + 4;                     // row stride of the merge buffer: heads 2 apart 8 banks apart
  static constexpr int SMEM = OFF_RED + NCW * PD_HEADS * RS * 4 + 1024;
};
static_assert(Geo<128>::SMEM <= 227 * 1024 && Geo<64>::SMEM <= 227 * 1024, "shared memory");

__device__ __forceinline__ void tma_load5(const CUtensorMap *map, uint64_t *bar, uint32_t dst, int c0, int c1, int c2,
                                          int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(map), "r"(su32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}
// What the roles' bounded waits share, in shared memory.
struct Waits {
  volatile int abort;
  int err;
  unsigned long long limit;  // ns
};
// Bounded waits whose probe may suspend the warp for up to SUSPEND_NS (a hint)
// before it gives the answer: warps that poll take issue slots from those that
// turn keys (128K at head_dim 64: 78.9 us with the default, 77.0 us so).
constexpr uint32_t SUSPEND_NS = 2000;
__device__ __forceinline__ bool mbar_try_long(uint64_t *b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(su32(b)), "r"(parity), "r"(SUSPEND_NS)
      : "memory");
  return ok != 0;
}
template <bool LONG>
static __device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity, Waits *w) {
  const uint64_t t0 = gtime();
  const uint64_t limit = w->limit;
  for (;;) {
    if (LONG ? mbar_try_long(bar, parity) : mbar_test(bar, parity)) return true;
    if (w->abort) return false;
    if (gtime() - t0 > limit) {
      w->abort = 1;
      atomicOr(&w->err, ERR_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_long(uint64_t *bar, uint32_t parity, Waits *w) {
  if (mbar_try_long(bar, parity)) return true;
  return wait_slow<true>(bar, parity, w);
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void lds_u64x2(uint32_t a, uint64_t &x, uint64_t &y) {
  asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "r"(a));
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// an 8 x 8 matrix of 16-bit elements, transposed over the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Packed fp32 pairs, kept as 64-bit registers from the load to the last use:
// one instruction computes both lanes.
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t bf2_f2(uint32_t w) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(w << 16), "r"(w & 0xffff0000u));
  return d;
}
__device__ __forceinline__ uint32_t f2_bf2(uint64_t f) {
  uint32_t d;
  asm("{\n\t.reg .f32 x, y;\n\tmov.b64 {x, y}, %1;\n\tcvt.rn.bf16x2.f32 %0, y, x;\n\t}" : "=r"(d) : "l"(f));
  return d;
}
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
// x as hi + lo, two bf16 pairs
__device__ __forceinline__ void split2(uint64_t x, uint32_t &hi, uint32_t &lo) {
  hi = f2_bf2(x);
  lo = f2_bf2(sub2(x, bf2_f2(hi)));
}
// Two weights x, y >= 0 as three bf16 pairs, whose sums they are: 3 x 8 bits by
// truncation.  No part is negative, and none is 0 where the weight is not (but at
// least 2^-126, the smallest that a weight is): each part's product with an
// infinite value then is that infinity, not 0 inf or an infinity of the other sign.
__device__ __forceinline__ void split3(float x, float y, uint32_t (&p)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
    p[i] = __byte_perm(a, b, 0x7632);
    x -= __uint_as_float(a & 0xffff0000u);
    y -= __uint_as_float(b & 0xffff0000u);
  }
  uint32_t least;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(least) : "r"(p[0]), "r"(0x00800080u));  // 2^-126
  asm("max.bf16x2 %0, %0, %1;" : "+r"(p[1]) : "r"(least));
  asm("max.bf16x2 %0, %0, %1;" : "+r"(p[2]) : "r"(least));
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
paged_decode_tc_kernel(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV,
                       const __grid_constant__ PagedDecodeArgs p, const __grid_constant__ TurnFreq turn) {
  using GG = Geo<D>;
  constexpr int HALF = GG::HALF, NST = GG::NST;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_full[NST], bar_empty[NST];
  __shared__ int s_j0[NST][NBLK], s_rho[NST][NBLK];  // a block's first key, and its remainder by G
  __shared__ float red_ml[NCW][PD_HEADS][2];
  __shared__ Waits waits;
  __shared__ int issued, announced[2];  // tiles whose loads were issued; the first tile of each group whose angles were not announced
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = (su32(smem_raw) + 1023u) & ~1023u;
  uint8_t *gbase = smem_raw + (sbase - su32(smem_raw));

  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&bar_full[s], 2);       // producer, angles
      mbar_init(&bar_empty[s], NBLK);   // the four consumer warps of the tile
    }
    waits.abort = waits.err = 0;
    issued = announced[0] = announced[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // turns by r = 0 .. 15 positions: {cos, cos, sin, sin} of two neighbouring
  // pairs, the 64-byte halves of odd rows swapped so that two rows meet in
  // different banks
  constexpr int TT = THREADS / HALF * HALF;  // a thread's turns are all of one frequency
  const unsigned long long tf = turn.v[threadIdx.x % HALF];
  for (int idx = threadIdx.x < TT ? threadIdx.x : PD_BLK * HALF; idx < PD_BLK * HALF; idx += TT) {
    const int r = idx / HALF, k = idx % HALF;
    float c, s;
    turn_cs(r, tf, c, s);
    float *to = reinterpret_cast<float *>(gbase + GG::OFF_TAB + r * HALF * 8 + (((k >> 1) * 16) ^ ((r & 1) * 64)));
    to[k & 1] = c;
    to[2 + (k & 1)] = s;
  }
  let_next_kernel_come();
  wait_for_kernel_before();
  if (threadIdx.x == 0) waits.limit = *(volatile unsigned long long *)&g_wait_limit_ns;
  const PagedRun run = paged_plan<THREADS>(p);
  __syncthreads();

  PagedWalk w(p, run);
  if (run.b >= 0) {
    if (warp == WARP_LOAD) {
      // ======================= producer =======================
      const int rows = min(1 << p.page_log2, PD_TILE);  // rows of a box
      const int per = rows / PD_BLK;                    // blocks of a box
      const bool leads = (lane & 3) % per == 0;         // this lane's block is the first of its box
      const uint32_t to = sbase + (lane & 3) / per * rows * D * 2;
      int it = 0;
      bool ok = true;
      while (ok && w.next(p)) {
        const int kvh = w.pair / p.HB;
        for (int u = w.u0; u < w.u1 && ok; u += 8) {
          // lane: block lane % 4 of tile u + lane / 4
          int page = 0, j0 = -1;
          if (u + (lane >> 2) < w.u1) j0 = paged_block(p, w.s, w.b, kvh, u + (lane >> 2), lane & 3, page);
          // a box is loaded where any of its blocks is wanted; page and slot are those of the first such block
          const unsigned want = __ballot_sync(0xffffffffu, j0 >= 0) >> lane & ((1u << per) - 1u);
          const int src = lane + (want ? __ffs(want) - 1 : 0);
          const int bp = __shfl_sync(0xffffffffu, page, src), bj = __shfl_sync(0xffffffffu, j0, src);
          const int slot = (bj & ((1 << p.page_log2) - 1)) & ~(rows - 1);
          const unsigned boxes = __ballot_sync(0xffffffffu, leads && want != 0);
          for (int x = 0; x < 8 && u + x < w.u1; ++x, ++it) {
            const int st = it % NST;
            if (it >= NST) ok = wait_long(&bar_empty[st], ((it / NST) - 1) & 1, &waits);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const bool mine = (lane >> 2) == x;
            if (mine) s_j0[st][lane & 3] = j0;
            __syncwarp();
            const int n = __popc(boxes >> (4 * x) & 15u);
            if (lane == 0) {
              if (n > 0) mbar_expect_tx(&bar_full[st], (uint32_t)(n * rows * D * 2 * 2));
              else mbar_arrive(&bar_full[st]);
            }
            __syncwarp();
            if (mine && leads && want != 0) {
              tma_load5(&mK, &bar_full[st], to + GG::OFF_K + st * GG::KV, 0, kvh, slot, bp, 0);
              tma_load5(&mV, &bar_full[st], to + GG::OFF_V + st * GG::KV, 0, kvh, slot, bp, 0);
            }
          }
        }
      }
      if (lane == 0) issued = it;
    } else if (warp >= WARP_ANGLE) {
      // ======================= angles =======================
      // one warp per consumer group (so that it too sees every phase of its
      // stages); the angles are formed before the stage is free for them
      const int par = warp - WARP_ANGLE;
      unsigned long long tw[HALF / 32];
#pragma unroll
      for (int e = 0; e < HALF / 32; ++e) tw[e] = turn.v[lane + 32 * e];
      int it = 0;
      bool ok = true;
      while (ok && w.next(p)) {
        const int kvh = w.pair / p.HB;
        const int G = p.plain ? 1 : (int)group_size(w.s.L, p.w_pre);
        const int ni = corr_n(w.s.L - 1, G);
        const int j_local = (int)max(0LL, (long long)w.s.L - (long long)p.w0);
        for (int u = w.u0; u < w.u1 && ok; u += 8) {
          int page, j0 = -1;
          if (G > 1 && u + (lane >> 2) < w.u1) j0 = paged_block(p, w.s, w.b, kvh, u + (lane >> 2), lane & 3, page);
          if (j0 >= j_local) j0 = -1;  // a local block
          const int f = j0 >= 0 ? j0 / G : 0, n = j0 - f - ni, rho = j0 - f * G;
          const unsigned want = __ballot_sync(0xffffffffu, j0 >= 0);
          for (int x = 0; x < 8 && u + x < w.u1; ++x, ++it) {
            if ((it & 1) != par) continue;
            const int st = it % NST;
            const bool any = (want >> (4 * x)) & 15u;
            float c[NBLK][HALF / 32], s[NBLK][HALF / 32];
            if (any) {
#pragma unroll
              for (int blk = 0; blk < NBLK; ++blk) {
                const int nb = __shfl_sync(0xffffffffu, n, 4 * x + blk);
#pragma unroll
                for (int e = 0; e < HALF / 32; ++e) turn_cs(nb, tw[e], c[blk][e], s[blk][e]);
              }
            }
            if (it >= NST) ok = wait_long(&bar_empty[st], ((it / NST) - 1) & 1, &waits);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (any) {
              if ((lane >> 2) == x) s_rho[st][lane & 3] = rho;
#pragma unroll
              for (int blk = 0; blk < NBLK; ++blk)
#pragma unroll
                for (int e = 0; e < HALF / 32; ++e) {
                  const int k = lane + 32 * e;
                  float *to = reinterpret_cast<float *>(gbase + GG::OFF_ANG + st * GG::ANG + blk * HALF * 8) +
                              (k >> 1) * 4 + (k & 1);
                  to[0] = c[blk][e];
                  to[2] = s[blk][e];
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_full[st]);
          }
        }
      }
      if (lane == 0) announced[par] = it;
    } else {
      // ======================= consumers =======================
      const int blk = warp & 3, par = warp >> 2;
      const int q4 = lane & 3, row = lane >> 2;
      const float scale = rsqrtf((float)D) * 1.4426950408889634f;
      // ldmatrix addresses in a tile, of keys x channels and (V, transposed on the
      // way) channels x keys operands; a box of `rows` keys has 64 channels of each
      // key in turn, then the other 64
      const int lm = lane >> 3, lr = lane & 7;
      const int rows = min(1 << p.page_log2, PD_TILE);
      const uint32_t half_b = D == 128 ? rows * 128 : 0;
      const uint32_t blk_at = (uint32_t)(blk * PD_BLK / rows * rows * D * 2 + (blk * PD_BLK % rows + lr) * 128);
      const uint32_t k_at = blk_at + (lm & 1) * 1024, v_at = blk_at + (lm >> 1) * 1024;
      const int k_ch = lm >> 1, v_ch = lm & 1;  // 8-channel chunk of a 16-channel step
      int it = 0;
      bool ok = true;
      // the hardware suspends for longer than a limit below SUSPEND_NS, whatever the
      // hint: such a one is kept by looks at the group's first tile that do not suspend
      if (waits.limit < SUSPEND_NS && run.t1 - run.t0 > par) ok = wait_slow<false>(&bar_full[par], 0, &waits);
      while (w.next(p)) {
        const int kvh = w.pair / p.HB, hb = w.pair % p.HB;
        const int gh = min(PD_HEADS, p.GS - hb * PD_HEADS);
        const int h0 = kvh * p.GS + hb * PD_HEADS;
        const int L = w.s.L, jw = w.s.jw;
        const int G = p.plain ? 1 : (int)group_size(L, p.w_pre);
        const int j_local = G > 1 ? (int)max(0LL, (long long)L - (long long)p.w0) : 0;
        // n(j0 + x) - n(j0) = x - floor((rho + x) / G), rho = j0 mod G, x < 16:
        // by 2^16 / G rounded up where G < 32 (exact for numerators below 2^11), else at most one
        const uint32_t inv_g = G < 32 ? (65535u + G) / G : 0u;
        auto turn_in = [&](int rho, int x) { return x - (G < 32 ? (int)(((rho + x) * inv_g) >> 16) : rho + x >= G); };
        // query operand: column = head `row`, channels 16 x + 2 q4 + {0, 1} and + 8
        uint32_t qf[D / 16][2];
        {
          const uint32_t *q = reinterpret_cast<const uint32_t *>((const __nv_bfloat16 *)p.q +
                                                                 ((size_t)w.b * p.Hq + h0 + row) * D);
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            qf[x][0] = row < gh ? q[8 * x + q4] : 0u;
            qf[x][1] = row < gh ? q[8 * x + 4 + q4] : 0u;
          }
        }
        // outputs, transposed: channels 16 x + row and + 8 of heads 2 q4 + {0, 1}; maximum of and this lane's
        // part of the sum for those heads
        float o[D / 16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int x = 0; x < D / 16; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;

        for (int u = w.u0; u < w.u1; ++u, ++it) {
          if ((it & 1) != par) continue;
          const int st = it % NST;
          if (ok) ok = wait_long(&bar_full[st], (it / NST) & 1, &waits);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) continue;  // the run is walked to its end, so that the merges' barriers are met
          const int j0 = s_j0[st][blk];
          if (j0 >= 0) {
            const uint32_t kt = sbase + GG::OFF_K + st * GG::KV + k_at;
            const uint32_t vt = sbase + GG::OFF_V + st * GG::KV + v_at;
            // scores of keys `row` (0, 1) and row + 8 (2, 3) for heads 2 q4 and 2 q4 + 1
            float sc[4];
            auto plain_scores = [&]() {
              float c[4] = {}, d[4] = {};
#pragma unroll
              for (int x = 0; x < D / 16; ++x) {
                uint32_t kf[4];
                ldsm4(kt + (x >> 2) * half_b + ((((x & 3) * 2 + k_ch) ^ lr) << 4), kf);
                mma(x & 1 ? d : c, kf[0], kf[1], kf[2], kf[3], qf[x][0], qf[x][1]);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) sc[e] = c[e] + d[e];
            };
            if (j0 >= j_local) {
              plain_scores();
            } else {
              // positions by which this lane's two keys (row and row + 8) turn beyond the block's first
              const int rho = s_rho[st][blk];
              const int r0 = turn_in(rho, row), r1 = turn_in(rho, row + 8);
              const uint32_t ang = sbase + GG::OFF_ANG + st * GG::ANG + blk * HALF * 8 + q4 * 16;
              const uint32_t tab = sbase + GG::OFF_TAB;
              const uint32_t t0 = tab + r0 * HALF * 8, t1 = tab + r1 * HALF * 8;
              const uint32_t x0 = (r0 & 1) * 64, x1 = (r1 & 1) * 64;
              float c[4] = {}, cl[4] = {};
#pragma unroll
              for (int x = 0; x < D / 32; ++x) {
                // channels 16 x .. + 15 and their partners
                uint32_t ka[4], kb[4];
                ldsm4(kt + (((x * 2 + k_ch) ^ lr) << 4), ka);
                if constexpr (D == 128)
                  ldsm4(kt + half_b + (((x * 2 + k_ch) ^ lr) << 4), kb);
                else
                  ldsm4(kt + (((4 + x * 2 + k_ch) ^ lr) << 4), kb);
                uint32_t ah[4], al[4], bh[4], bl[4];
#pragma unroll
                for (int y = 0; y < 2; ++y) {  // channels + 8 y
                  const uint32_t at = (x * 16 + y * 8) * 8;
                  uint64_t fc, fs;
                  lds_u64x2(ang + at, fc, fs);
#pragma unroll
                  for (int nb = 0; nb < 2; ++nb) {  // keys + 8 nb
                    const int i = 2 * y + nb;
                    uint64_t gc, gs;
                    lds_u64x2((nb ? t1 : t0) + ((at + q4 * 16) ^ (nb ? x1 : x0)), gc, gs);
                    const uint64_t co = sub2(mul2(fc, gc), mul2(fs, gs));
                    const uint64_t si = fma2(fs, gc, mul2(fc, gs));
                    const uint64_t a = bf2_f2(ka[i]), b = bf2_f2(kb[i]);
                    split2(fma2(a, co, mul2(b, si)), ah[i], al[i]);
                    split2(sub2(mul2(b, co), mul2(a, si)), bh[i], bl[i]);
                  }
                }
                mma(c, ah[0], ah[1], ah[2], ah[3], qf[x][0], qf[x][1]);
                mma(cl, al[0], al[1], al[2], al[3], qf[x][0], qf[x][1]);
                mma(c, bh[0], bh[1], bh[2], bh[3], qf[D / 32 + x][0], qf[D / 32 + x][1]);
                mma(cl, bl[0], bl[1], bl[2], bl[3], qf[D / 32 + x][0], qf[D / 32 + x][1]);
              }
              // where an element is infinite its high half alone says so: what is left of it
              // is inf - inf, and a low half times an infinite query may be 0 inf
#pragma unroll
              for (int e = 0; e < 4; ++e) cl[e] = isnan(c[e] + cl[e]) ? c[e] : c[e] + cl[e];
              if (j0 + PD_BLK > j_local) {  // the one block with keys of both kinds
                plain_scores();
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (j0 + row + 8 * (e >> 1) < j_local) sc[e] = cl[e];
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[e] = cl[e];
              }
            }
            // mask, in units of log2 e
            const bool part = j0 + PD_BLK > L || j0 < jw;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              sc[e] *= scale;
              const int j = j0 + row + 8 * (e >> 1);
              if (part && (j >= L || j < jw)) sc[e] = -INFINITY;
            }
            float top[2], f[2];
            bool grow = false;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              top[h] = max_nan(sc[h], sc[2 + h]);
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) top[h] = max_nan(top[h], __shfl_xor_sync(0xffffffffu, top[h], x));
              // the maximum is only moved when it has grown by more than 2^8
              const bool g = !(top[h] <= m[h] + 8.f) && !(top[h] == -INFINITY);
              f[h] = 1.f;
              if (g) {
                f[h] = m[h] == -INFINITY ? 0.f : ex2(m[h] - top[h]);
                m[h] = top[h];
              }
              grow = grow || g;
            }
            if (__any_sync(0xffffffffu, grow)) {
              l[0] *= f[0], l[1] *= f[1];
#pragma unroll
              for (int x = 0; x < D / 16; ++x) o[x][0] *= f[0], o[x][1] *= f[1], o[x][2] *= f[0], o[x][3] *= f[1];
            }
            // weights, in three parts, turned into the second operand of the products with the values
            const float m0 = m[0] == -INFINITY ? 0.f : m[0], m1 = m[1] == -INFINITY ? 0.f : m[1];
            uint32_t pw[2][3];
#pragma unroll
            for (int nb = 0; nb < 2; ++nb) {
              const float e0 = ex2(sc[2 * nb] - m0), e1 = ex2(sc[2 * nb + 1] - m1);
              l[0] += e0, l[1] += e1;
              split3(e0, e1, pw[nb]);
#pragma unroll
              for (int i = 0; i < 3; ++i) pw[nb][i] = transpose8(pw[nb][i]);
            }
            uint32_t keep[2] = {0xffffffffu, 0xffffffffu};  // of keys 2 q4 + {0, 1} (+ 8)
            if (part) {
#pragma unroll
              for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int j = j0 + 8 * nb + 2 * q4 + e;
                  if (j >= L || j < jw) keep[nb] &= e == 0 ? 0xffff0000u : 0x0000ffffu;
                }
            }
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
              uint32_t vf[4];
              ldsm4t(vt + (x >> 2) * half_b + ((((x & 3) * 2 + v_ch) ^ lr) << 4), vf);
              if (part) {  // rows past the length may hold anything, and 0 NaN is NaN
                vf[0] &= keep[0], vf[1] &= keep[0];
                vf[2] &= keep[1], vf[3] &= keep[1];
              }
#pragma unroll
              for (int i = 0; i < 3; ++i) mma(o[x], vf[0], vf[1], vf[2], vf[3], pw[0][i], pw[1][i]);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_empty[st]);
        }

        // merge the warps' results of this piece
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], x);
          if (row == 0) red_ml[warp][2 * q4 + h][0] = m[h], red_ml[warp][2 * q4 + h][1] = l[h];
        }
        float *red = reinterpret_cast<float *>(gbase + GG::OFF_RED);
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            red[(warp * PD_HEADS + 2 * q4 + (e & 1)) * GG::RS + 16 * x + row + 8 * (e >> 1)] = o[x][e];
        asm volatile("bar.sync 1, %0;" ::"n"(NCW * 32) : "memory");
        const bool whole = w.u0 == 0 && w.u1 == w.s.tiles;
        const size_t slot = 2 * (size_t)blockIdx.x + (w.u0 > 0 ? 0 : 1);
        for (int idx = threadIdx.x; idx < gh * (D / 2); idx += NCW * 32) {
          const int g = idx / (D / 2), d = idx % (D / 2) * 2;
          float M = -INFINITY;
#pragma unroll
          for (int x = 0; x < NCW; ++x) M = max_nan(M, red_ml[x][g][0]);
          float sum = 0.f;
          float2 acc = make_float2(0.f, 0.f);
          if (M != -INFINITY)
#pragma unroll
            for (int x = 0; x < NCW; ++x) {
              const float f = exp2f(red_ml[x][g][0] - M);
              const float2 y = *reinterpret_cast<const float2 *>(red + (x * PD_HEADS + g) * GG::RS + d);
              sum = fmaf(f, red_ml[x][g][1], sum);
              acc.x = fmaf(f, y.x, acc.x);
              acc.y = fmaf(f, y.y, acc.y);
            }
          if (whole) {
            const size_t bh = (size_t)w.b * p.Hq + h0 + g;
            const float r = M != -INFINITY ? 1.f / sum : 0.f;
            reinterpret_cast<uint32_t *>(p.out)[(bh * D + d) / 2] = f2_bf2(pack2(acc.x * r, acc.y * r));
            if (p.lse != nullptr && d == 0) p.lse[bh] = M != -INFINITY ? (M + log2f(sum)) * LN2 : -INFINITY;
          } else {
            *reinterpret_cast<float2 *>(p.part_o + (slot * PD_HEADS + g) * D + d) = acc;
            if (d == 0) {
              p.part_ml[(slot * PD_HEADS + g) * 2] = M;
              p.part_ml[(slot * PD_HEADS + g) * 2 + 1] = sum;
            }
          }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(NCW * 32) : "memory");
      }
    }
  }
  __syncthreads();
  // after a timeout, let the loads in flight land; a stage whose angles were not
  // announced is announced here, so that its barrier waits for the loads alone
  if (threadIdx.x == 0 && waits.abort)
    for (int x = max(0, issued - NST); x < issued; ++x) {
      if (x >= announced[x & 1]) mbar_arrive(&bar_full[x % NST]);
      wait_drain(&bar_full[x % NST], (x / NST) & 1, &waits.err, ERR_TIMEOUT);
    }
  if (threadIdx.x == 0) p.cta_err[blockIdx.x] = waits.err;
}

static bool make_pool_map(CUtensorMap *m, const void *base, const PagedDecodeArgs &a, int D) {
  // a pool viewed as (channel of 64, head, slot, page, 64 channels)
  static EncodeTiledFn enc = get_encode_tiled();
  if (enc == nullptr) return false;
  const int P = 1 << a.page_log2;
  const cuuint64_t dims[5] = {64, (cuuint64_t)a.Hkv, (cuuint64_t)P, (cuuint64_t)a.n_pages, (cuuint64_t)D / 64};
  const cuuint64_t strides[4] = {(cuuint64_t)D * 2, (cuuint64_t)a.Hkv * D * 2, (cuuint64_t)a.page_stride * 2, 128};
  const cuuint32_t box[5] = {64, 1, (cuuint32_t)(P < PD_TILE ? P : PD_TILE), 1, (cuuint32_t)D / 64};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace pgt

int paged_decode_tc_ctas() { return pgt::CTAS; }

cudaError_t launch_paged_decode_tc(int D, const PagedDecodeArgs &a, const TurnFreq &turn, cudaStream_t st) {
  CUtensorMap mK, mV;
  if (!pgt::make_pool_map(&mK, a.k, a, D) || !pgt::make_pool_map(&mV, a.v, a, D)) return cudaErrorInvalidValue;
  cudaError_t e;
  if (D == 128) {
    e = cudaFuncSetAttribute(pgt::paged_decode_tc_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             pgt::Geo<128>::SMEM);
    if (e != cudaSuccess) return e;
    return launch_overlapped(pgt::paged_decode_tc_kernel<128>, pgt::CTAS, pgt::THREADS, pgt::Geo<128>::SMEM, st, mK, mV, a,
                             turn);
  } else {
    e = cudaFuncSetAttribute(pgt::paged_decode_tc_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             pgt::Geo<64>::SMEM);
    if (e != cudaSuccess) return e;
    return launch_overlapped(pgt::paged_decode_tc_kernel<64>, pgt::CTAS, pgt::THREADS, pgt::Geo<64>::SMEM, st, mK, mV, a,
                             turn);
  }
}

// Test hook: the limit of the bounded waits of this file's kernels.
cudaError_t set_wait_limit_paged(unsigned long long ns) {
  return cudaMemcpyToSymbol(g_wait_limit_ns, &ns, sizeof(ns));
}

}  // namespace jl
