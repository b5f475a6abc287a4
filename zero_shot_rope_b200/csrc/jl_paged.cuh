// Shared declarations of the paged-cache operators: append, page selection
// and decode.
//
// The cache is a pool of pages [n_pages, P, Hkv, D] (K and V each; the first
// stride is the caller's), P a power of two from 16 to 256.  Logical page c
// of sequence b, its keys cP .. cP + P - 1, is pool page table[b, c].
#pragma once

#include <utility>

#include "jl_common.cuh"

namespace jl {

// Minimum / maximum that keep a NaN: a NaN key must show in its page's range and
// in the output, not vanish from a comparison.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Rotation frequencies in turns per position, as fractions of 2^64: the angle
// of n positions, modulo a turn, is one integer product, which wraps where the
// angle does.
struct TurnFreq {
  unsigned long long v[JL_MAX_HALF];
};

// cos and sin of n positions' angle.  The product's two top bits (rounded) are
// the quadrant, the rest an angle within an eighth of a turn, whose sine and
// cosine are the Taylor series in fp32 (to r^9 and r^10: truncated at 2e-9 and
// 2e-10).  Off by less than 3 2^-24 from those of the exact product of n and the
// frequency, up to 2^64 radians a position; about 25 instructions, against some 60 of 64-bit
// arithmetic in angle_cs.
__host__ __device__ __forceinline__ void turn_cs(int32_t n, unsigned long long w, float &c, float &s) {
  const unsigned long long x = (unsigned long long)(long long)n * w;
  const uint32_t t = (uint32_t)(x >> 32);
  const uint32_t quad = t + 0x20000000u;              // nearest quarter turn, in the two top bits
  const int32_t f = (int32_t)(t - (quad & 0xc0000000u));  // the rest: -2^29 .. 2^29 - 1
  const float r = (float)f * 1.46291807926715968105e-9f;  // 2 pi / 2^32
  const float r2 = r * r;
  float ps = 2.7557319223985893e-6f;  // 1/9!
  ps = fmaf(ps, r2, -1.9841269841269841e-4f);
  ps = fmaf(ps, r2, 8.3333333333333333e-3f);
  ps = fmaf(ps, r2, -1.6666666666666667e-1f);
  const float sr = fmaf(r * r2, ps, r);
  float pc = -2.7557319223985888e-7f;  // -1/10!
  pc = fmaf(pc, r2, 2.4801587301587302e-5f);
  pc = fmaf(pc, r2, -1.3888888888888889e-3f);
  pc = fmaf(pc, r2, 4.1666666666666667e-2f);
  pc = fmaf(pc, r2, -0.5f);
  const float cr = fmaf(pc, r2, 1.f);
  const bool swap = quad & 0x40000000u;
  const float a = swap ? sr : cr, b = swap ? cr : sr;
  // quadrants 0..3: (cr, sr), (-sr, cr), (-cr, -sr), (sr, -cr)
  c = ((quad >> 30) + 1) & 2 ? -a : a;
  s = quad & 0x80000000u ? -b : b;
}

constexpr int PG_MIN_LOG2 = 4, PG_MAX_LOG2 = 8;  // page sizes 16 .. 256

// ------------------------------------------------------------------ decode
// Keys are processed in tiles of 64 consecutive cache slots, each made of four
// 16-key blocks; a block lies inside one page (P >= 16).
constexpr int PD_TILE = 64;
constexpr int PD_BLK = 16;
constexpr int PD_HEADS = 8;     // query heads a CTA serves at a time (of one kv head)
constexpr int PD_MAX_CTAS = 296;  // two per SM (the CUDA-core kernel); the tensor-core kernel runs one

struct PagedDecodeArgs {
  const void *q, *k, *v;          // k, v: the pools
  const int32_t *table;           // [B, max_pages], row stride table_stride
  long long table_stride;
  const int32_t *seqlens;
  const int32_t *list;            // [B, Hkv, n_list] logical pages, or NULL: every page
  int n_list, max_pages, page_log2, n_pages;
  long long page_stride;          // elements between pages of a pool
  int B, Hq, Hkv, GS, HB;         // HB: blocks of PD_HEADS query heads per kv head
  long long w_pre;
  int w0, window, plain;
  float *part_o;                  // [2 * CTAs][PD_HEADS][D]
  float *part_ml;                 // [2 * CTAs][PD_HEADS][2]
  long long *tab;                 // [B + 1] first tile of each sequence
  int *err;                       // the call's error word, and one for each CTA behind it
  int *cta_err;
  void *out;
  float *lse;
};

// What a sequence's length means for the decode.
struct PagedSeq {
  int L, jw, j_first, tiles;      // length, first visible key, first key of tile 0, tiles per (kv head, head block)
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedDecodeArgs &p, int b) {
  PagedSeq s;
  s.L = p.seqlens[b];
  if (s.L < 0 || (long long)s.L > ((long long)p.max_pages << p.page_log2)) s.L = 0;  // outside the contract: no key
  s.jw = p.window > 0 ? max(0, s.L - p.window) : 0;
  if (p.list != nullptr) {
    s.j_first = 0;
    s.tiles = s.L > 0 ? (int)((((long long)p.n_list << p.page_log2) + PD_TILE - 1) / PD_TILE) : 0;
  } else {
    s.j_first = s.jw & ~(PD_TILE - 1);
    s.tiles = (int)(((long long)s.L - s.j_first + PD_TILE - 1) / PD_TILE);
  }
  return s;
}

// First key of 16-key block `blk` of tile u, and its pool row block: the page
// in `page` (its slot is the key index mod P).  -1: nothing to read there (past
// the length, before the window, no such page).
__device__ __forceinline__ int paged_block(const PagedDecodeArgs &p, const PagedSeq &s, int b, int kvh, int u, int blk,
                                           int &page) {
  int j0;
  const long long at = (long long)u * PD_TILE + blk * PD_BLK;
  if (p.list != nullptr) {
    const long long e = at >> p.page_log2;
    if (e >= p.n_list) return -1;
    const int c = p.list[((long long)b * p.Hkv + kvh) * p.n_list + e];
    if (c < 0 || c >= p.max_pages) return -1;
    j0 = (c << p.page_log2) + (int)(at & ((1 << p.page_log2) - 1));
  } else {
    j0 = s.j_first + (int)at;
  }
  if (j0 >= s.L || j0 + PD_BLK <= s.jw) return -1;
  page = p.table[(long long)b * p.table_stride + (j0 >> p.page_log2)];
  if (page < 0 || page >= p.n_pages) return -1;
  return j0;
}

// The work list: the tiles of all sequences in order (sequence, then kv head,
// then head block, then tile), cut into equal runs, one per CTA.  A run meets
// at most two (kv head, head block) pairs of a sequence that it does not
// cover whole: the one it starts in and the one it ends in.  Their partial
// results go to the CTA's two slots; pairs covered whole are finished in place.
struct PagedRun {
  long long base;    // first tile of sequence b
  long long t0, t1;  // this CTA's tiles
  int b;             // sequence of tile t0
};

__device__ __forceinline__ long long div_up(long long n, int d) {
  if (n < (1ll << 31)) return (unsigned)(n + d - 1) / (unsigned)d;
  return (n + d - 1) / d;
}

// This CTA's run, from the lengths on the device, so that a captured step
// replays with the lengths of the moment.  CTA 0 also leaves the first tile of
// every sequence in p.tab for the combine.  Up to 32 sequences: every warp by
// itself.  More: the whole block, which has to call it together.
template <int NT>
__device__ __forceinline__ PagedRun paged_plan(const PagedDecodeArgs &p) {
  const unsigned full = 0xffffffffu;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pairs = p.Hkv * p.HB;
  auto warp_scan = [&](long long x) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(full, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  PagedRun r;
  if (p.B <= 32) {
    const long long n = lane < p.B ? (long long)paged_seq(p, lane).tiles * pairs : 0;
    const long long last = warp_scan(n), first = last - n, total = __shfl_sync(full, last, 31);
    if (blockIdx.x == 0 && warp == 0) {
      if (lane < p.B) p.tab[lane] = first;
      if (lane == 0) p.tab[p.B] = total;
    }
    const long long chunk = div_up(total, gridDim.x);
    r.t0 = (long long)blockIdx.x * chunk;
    r.t1 = r.t0 + chunk < total ? r.t0 + chunk : total;
    r.b = __ffs(__ballot_sync(full, r.t0 >= first && r.t0 < last)) - 1;
    r.base = __shfl_sync(full, first, max(r.b, 0));
    return r;
  }
  __shared__ long long s_warp[NT / 32], s_first;
  __shared__ int s_b;
  auto scan = [&](long long x, long long &total) {  // inclusive over the block
    x = warp_scan(x);
    __syncthreads();
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    total = 0;
    long long before = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) before += s_warp[w];
      total += s_warp[w];
    }
    return x + before;
  };
  long long mine = 0, total;
  for (int b = tid; b < p.B; b += NT) mine += (long long)paged_seq(p, b).tiles * pairs;
  scan(mine, total);
  const long long chunk = div_up(total, gridDim.x);
  r.t0 = (long long)blockIdx.x * chunk;
  r.t1 = r.t0 + chunk < total ? r.t0 + chunk : total;
  if (tid == 0) s_b = -1;
  __syncthreads();
  long long carry = 0;
  for (int b0 = 0; b0 < p.B; b0 += NT) {
    const int b = b0 + tid;
    const long long n = b < p.B ? (long long)paged_seq(p, b).tiles * pairs : 0;
    long long sum;
    const long long first = carry + scan(n, sum) - n;
    if (b < p.B) {
      if (blockIdx.x == 0) p.tab[b] = first;
      if (r.t0 >= first && r.t0 < first + n) {
        s_b = b;
        s_first = first;
      }
    }
    carry += sum;
    if (blockIdx.x != 0 && carry > r.t0) break;  // uniform over the block
  }
  if (blockIdx.x == 0 && tid == 0) p.tab[p.B] = carry;
  __syncthreads();
  r.b = s_b;
  r.base = s_first;
  return r;
}

// The run's tiles piece by piece (a piece: tiles u0 .. u1 - 1 of one (kv head,
// head block) of sequence b), as every warp walks them.
struct PagedWalk {
  long long base, t, t1;
  int b, pairs;
  PagedSeq s;
  int pair, u0, u1;
  __device__ __forceinline__ PagedWalk(const PagedDecodeArgs &p, const PagedRun &r)
      : base(r.base), t(r.t0), t1(r.b >= 0 ? r.t1 : r.t0), b(r.b), pairs(p.Hkv * p.HB) {}
  __device__ __forceinline__ bool next(const PagedDecodeArgs &p) {
    while (t < t1) {
      s = paged_seq(p, b);
      const long long n = (long long)s.tiles * pairs;
      if (t >= base + n) {
        base += n;
        ++b;
        continue;
      }
      const long long at = t - base;
      pair = at < (1ll << 31) ? (int)((unsigned)at / (unsigned)s.tiles) : (int)(at / s.tiles);
      u0 = (int)(at - (long long)pair * s.tiles);
      u1 = (int)(t1 - t < s.tiles - u0 ? u0 + (t1 - t) : s.tiles);
      t += u1 - u0;
      return true;
    }
    return false;
  }
};

// ------------------------------------------------------- dependent launches
// The paged-cache kernels are launched so that their set-up overlaps the end of
// the kernel before them (programmatic dependent launch): each waits for all of
// that kernel's work before it touches global memory, and lets the next one's
// blocks come as soon as its own are placed.
__device__ __forceinline__ void wait_for_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_come() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A &&...args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

// The tensor-core kernel (bf16): the partial results only; paged_decode_tc_ctas() runs.
int paged_decode_tc_ctas();
cudaError_t launch_paged_decode_tc(int D, const PagedDecodeArgs &a, const TurnFreq &turn, cudaStream_t st);
cudaError_t launch_paged_decode(bool bf16, int D, const PagedDecodeArgs &a, const TurnFreq &turn, cudaStream_t st);

// ------------------------------------------------------------------ append
struct PagedAppendArgs {
  const void *k, *v, *q;
  void *k_pages, *v_pages, *summary, *q_out;
  const int32_t *table;
  long long table_stride;
  const int32_t *cu, *seqlens;
  int max_pages, page_log2, n_pages, T, max_new, Hkv, GS;
  int heads;  // kv heads of a CTA
  long long page_stride;
};
cudaError_t launch_paged_append(bool bf16, int D, bool rotate, const PagedAppendArgs &a, const TurnFreq &turn,
                                int batch, cudaStream_t st);

// ------------------------------------------------------------------ select
struct PagedSelectArgs {
  const void *q, *summary;
  const int32_t *table;
  long long table_stride;
  const int32_t *seqlens;
  int B, Hkv, GS, max_pages, page_log2, n_pages, n_select, n_first, n_last;
  long long w_pre;
  int w0, plain;
  int32_t *list;
  // [B, Hkv, max_pages] each: a page's fp32 score (twice it); for pairs of pages,
  // a bound of the sum of squares of their key ranges; 1 for a chosen page; the
  // undecided pages and their scores in 64 bits
  float *score, *size, *mark;
  int32_t *amb;
  double *fine;
};
cudaError_t launch_paged_select(bool bf16, int D, const PagedSelectArgs &a, const InvFreq &inv, const TurnFreq &turn,
                                cudaStream_t st);

}  // namespace jl
