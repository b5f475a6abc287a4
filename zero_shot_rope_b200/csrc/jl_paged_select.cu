// Selection of the cache pages that the new token of each sequence reads
// (sm_100a).
//
// Each page carries, per kv head and channel, the least and the greatest value
// of its keys.  For a query turned by the bifocal shift of the page's middle
// key, q' = R(n(m) - n(i)) q (no turn for a local page), every key of the page
// whose own shift is that one scores at most
//     sum_d max(q'_d min_d, q'_d max_d),
// and the page's score is the largest such bound over the kv head's query
// heads.  The list holds the first and the newest pages, then the highest
// scores.
//
// Which pages are chosen does not depend on rounding: scores are formed in
// fp32, and only those too near the last chosen one to be told apart there are
// formed again in 64 bits (select_kernel).
#include "jl_paged.cuh"

namespace jl {

namespace pgs {


// PPL pairs per lane, as fp32: elements PPL l .. of a row's halves
template <typename T, int PPL>
__device__ __forceinline__ void load_pairs(const T *row, int half, int lane, float (&a)[PPL], float (&b)[PPL]) {
  if constexpr (PPL == 2 && sizeof(T) == 4) {
    const float2 x = *reinterpret_cast<const float2 *>(row + 2 * lane);
    const float2 y = *reinterpret_cast<const float2 *>(row + half + 2 * lane);
    a[0] = x.x, a[1] = x.y, b[0] = y.x, b[1] = y.y;
  } else if constexpr (PPL == 2) {
    const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(row + 2 * lane));
    const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(row + half + 2 * lane));
    a[0] = x.x, a[1] = x.y, b[0] = y.x, b[1] = y.y;
  } else {
    a[0] = to_f(row[lane]);
    b[0] = to_f(row[half + lane]);
  }
}

// pages of sequence b; 0 for a length outside the contract
__device__ __forceinline__ int pages_of(const PagedSelectArgs &p, int b) {
  const int L = p.seqlens[b];
  if (L < 0 || (long long)L > ((long long)p.max_pages << p.page_log2)) return 0;
  return (int)(((long long)L + (1 << p.page_log2) - 1) >> p.page_log2);
}
// and what its pages' turns depend on
struct Seq {
  int L, pages, G, ni, j_local;
};
__device__ __forceinline__ Seq seq_of(const PagedSelectArgs &p, int b) {
  Seq s;
  s.pages = pages_of(p, b);
  s.L = s.pages > 0 ? p.seqlens[b] : 0;
  s.G = p.plain ? 1 : (int)group_size(s.L, p.w_pre);
  s.ni = s.L > 0 ? corr_n(s.L - 1, s.G) : 0;
  s.j_local = (int)max(0LL, (long long)s.L - (long long)p.w0);
  return s;
}
// positions by which the query is turned for page c: n(m) - n(i), 0 if local
__device__ __forceinline__ int page_turn(const PagedSelectArgs &p, const Seq &s, int c) {
  const int m = (c << p.page_log2) + (1 << p.page_log2) / 2;
  return s.G > 1 && m < s.j_local ? corr_n(m, s.G) - s.ni : 0;
}
__device__ __forceinline__ int pool_page(const PagedSelectArgs &p, int b, int c) {
  const int page = p.table[(long long)b * p.table_stride + c];
  return page >= 0 && page < p.n_pages ? page : -1;
}

// packed fp32 pairs
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
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
__device__ __forceinline__ float2 unpack2(uint64_t d) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(d));
  return f;
}
// N values (2 or 4) from 2 N or 4 N aligned bytes
template <typename T, int N>
__device__ __forceinline__ void load_n(const T *p, float (&x)[N]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float2 v = *reinterpret_cast<const float2 *>(p + e);
      x[e] = v.x, x[e + 1] = v.y;
    }
  } else {
    uint32_t w[N / 2];
    if constexpr (N == 4) {
      const uint2 v = *reinterpret_cast<const uint2 *>(p);
      w[0] = v.x, w[1] = v.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
#pragma unroll
    for (int e = 0; e < N; e += 2) x[e] = __uint_as_float(w[e / 2] << 16), x[e + 1] = __uint_as_float(w[e / 2] & 0xffff0000u);
  }
}

// Twice the scores, in fp32.  A CTA takes the key ranges of 8 pages and up to 8
// kv heads, 64 KB at most, all asked for at once (a page's heads lie side by
// side); the pages' angles are formed meanwhile, once for all heads.  Then warps
// go through the heads with the head's queries in registers, two pages at a
// time, one per half warp.  A lane has the sums of GP heads, which are added up
// over the lanes together: with each shuffle it hands over half of what it holds
// and keeps the other half.
constexpr int SCORE_HEADS = 8;
constexpr int SP = 8;
template <typename T, int D>
__host__ __device__ constexpr int score_smem() { return SP * SCORE_HEADS * 2 * D * (int)sizeof(T); }

template <typename T, int D, int GP, int NT_SCORE>
__global__ void __launch_bounds__(NT_SCORE, 512 / NT_SCORE)
score_kernel(const __grid_constant__ PagedSelectArgs p, const __grid_constant__ TurnFreq turn) {
  constexpr int HALF = D / 2, PPL = HALF / 16, NW = NT_SCORE / 32;
  extern __shared__ __align__(16) uint8_t range_s[];  // [SP][heads][2][D]
  __shared__ float4 ang[SP][HALF / 2];                // of two neighbouring pairs: cos, cos, sin, sin
  __shared__ const uint8_t *from_s[SP];  // a page's ranges, NULL: not there
  __shared__ int turn_s[SP], np_s;
  const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = blockIdx.x * SP;
  const int h_first = blockIdx.z * SCORE_HEADS, heads = min(SCORE_HEADS, p.Hkv - h_first);
  // (a thread's angles are all of one frequency, read once: lanes that read
  // different constants take turns)
  static_assert(NT_SCORE % HALF == 0, "one frequency per thread");
  const unsigned long long w = turn.v[threadIdx.x % HALF];
  let_next_kernel_come();
  wait_for_kernel_before();
  if (warp == 0) {
    const int c = c0 + lane;
    const int page = lane < SP && c < p.max_pages ? pool_page(p, b, c) : -1;
    const Seq s = seq_of(p, b);
    const int np = s.pages <= p.n_select ? 0 : min(SP, s.pages - c0);  // no more pages than the list: all of them are in it
    if (lane < SP) {
      turn_s[lane] = lane < np ? page_turn(p, s, c) : 0;
      from_s[lane] = lane < np && page >= 0
                         ? (const uint8_t *)p.summary + ((size_t)page * p.Hkv + h_first) * 2 * D * sizeof(T)
                         : nullptr;
    }
    if (lane == 0) np_s = np;
  }
  __syncthreads();
  const int np = np_s;
  if (np <= 0) return;
  {
    const int per = heads * 2 * D * (int)sizeof(T);  // bytes of a page
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(range_s);
#pragma unroll
    for (int c = 0; c < SP; ++c) {
      const uint8_t *from = from_s[c];
      for (int x = threadIdx.x * 16; x < per; x += NT_SCORE * 16) {  // a page that is not there: zeros
        const bool there = from != nullptr;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + c * per + x),
                     "l"(there ? from + x : (const uint8_t *)p.summary), "r"(there ? 16 : 0)
                     : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
#pragma unroll
  for (int x = threadIdx.x; x < SP * HALF; x += NT_SCORE) {
    const int c = x / HALF, k = x % HALF;
    float co, si;
    turn_cs(turn_s[c], w, co, si);
    float *to = reinterpret_cast<float *>(&ang[c][k / 2]) + (k & 1);
    to[0] = co;
    to[2] = si;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  const T *q = (const T *)p.q + (size_t)b * p.Hkv * p.GS * D;
  const int sub = lane >> 4, k0 = (lane & 15) * PPL;  // page of the two, first pair of this lane
  // a unit: two pages of a head; a warp takes a run of units, head by head
  const int per_head = SP / 2, units = heads * per_head, u1 = units * (warp + 1) / NW;
  uint64_t qa[GP][PPL / 2], qb[GP][PPL / 2];
  int held = -1;         // the head whose queries they are
  float size[2 * PPL];   // the largest |min|, |max| of each channel over the pages of that head seen so far
  auto put_size = [&](int h, int first, int n) {  // of page pairs first .. first + n - 1 of the CTA
    float sq = 0.f;
#pragma unroll
    for (int e = 0; e < 2 * PPL; ++e) {
      size[e] = max_nan(size[e], __shfl_xor_sync(0xffffffffu, size[e], 16));
      sq = fmaf(size[e], size[e], sq);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    if (lane < n && 2 * (first + lane) < np) p.size[((size_t)b * p.Hkv + h) * p.max_pages + c0 / 2 + first + lane] = sq;
  };
  auto load_q = [&](int h, int g0) {
#pragma unroll
    for (int g = 0; g < GP; ++g) {  // a head twice is no other maximum
      const T *row = q + (size_t)(h * p.GS + min(g0 + g, p.GS - 1)) * D + k0;
      float x[PPL], y[PPL];
      load_n<T, PPL>(row, x);
      load_n<T, PPL>(row + HALF, y);
#pragma unroll
      for (int e = 0; e < PPL / 2; ++e) qa[g][e] = pack2(x[2 * e], x[2 * e + 1]), qb[g][e] = pack2(y[2 * e], y[2 * e + 1]);
    }
  };
  for (int u = units * warp / NW; u < u1; ++u) {
    const int h = h_first + u / per_head, x0 = (u % per_head) * 2;
    if (held != h) {
      held = h;
      load_q(h, 0);
#pragma unroll
      for (int e = 0; e < 2 * PPL; ++e) size[e] = 0.f;
    }
    const int x = x0 + sub;
    // 2 max(t lo, t hi) = t (hi + lo) + |t| (hi - lo)
    uint64_t mid_a[PPL / 2], mid_b[PPL / 2], rad_a[PPL / 2], rad_b[PPL / 2];
    {
      const T *row = reinterpret_cast<const T *>(range_s) + (x * heads + h - h_first) * 2 * D + k0;
      float la[PPL], lb[PPL], ha[PPL], hb[PPL];
      load_n<T, PPL>(row, la);
      load_n<T, PPL>(row + HALF, lb);
      load_n<T, PPL>(row + D, ha);
      load_n<T, PPL>(row + D + HALF, hb);
#pragma unroll
      for (int e = 0; e < PPL; ++e) {
        size[2 * e] = max_nan(size[2 * e], max_nan(fabsf(la[e]), fabsf(ha[e])));
        size[2 * e + 1] = max_nan(size[2 * e + 1], max_nan(fabsf(lb[e]), fabsf(hb[e])));
      }
#pragma unroll
      for (int e = 0; e < PPL / 2; ++e) {
        mid_a[e] = pack2(ha[2 * e] + la[2 * e], ha[2 * e + 1] + la[2 * e + 1]);
        rad_a[e] = pack2(ha[2 * e] - la[2 * e], ha[2 * e + 1] - la[2 * e + 1]);
        mid_b[e] = pack2(hb[2 * e] + lb[2 * e], hb[2 * e + 1] + lb[2 * e + 1]);
        rad_b[e] = pack2(hb[2 * e] - lb[2 * e], hb[2 * e + 1] - lb[2 * e + 1]);
      }
    }
    uint64_t co[PPL / 2], si[PPL / 2], ns[PPL / 2];
#pragma unroll
    for (int e = 0; e < PPL / 2; ++e) {
      const float4 f = ang[x][k0 / 2 + e];
      co[e] = pack2(f.x, f.y), si[e] = pack2(f.z, f.w), ns[e] = si[e] ^ 0x8000000080000000ull;
    }
    float best = -INFINITY;
    for (int g0 = 0; g0 < p.GS; g0 += GP) {
      if (p.GS > GP) load_q(h, g0);
      float v[GP];
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        uint64_t y = 0ull;
#pragma unroll
        for (int e = 0; e < PPL / 2; ++e) {
          // <R(-turn) k, q> = <k, R(turn) q>
          const uint64_t ta = fma2(qa[g][e], co[e], mul2(qb[g][e], ns[e]));
          const uint64_t tb = fma2(qb[g][e], co[e], mul2(qa[g][e], si[e]));
          y = fma2(ta, mid_a[e], y);
          y = fma2(tb, mid_b[e], y);
          y = fma2(ta & 0x7fffffff7fffffffull, rad_a[e], y);
          y = fma2(tb & 0x7fffffff7fffffffull, rad_b[e], y);
        }
        const float2 f = unpack2(y);
        v[g] = f.x + f.y;
      }
      int o = 8;
#pragma unroll
      for (int n = GP; n > 1; n >>= 1, o >>= 1)
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
          const bool up = lane & o;
          const float keep = up ? v[i + n / 2] : v[i], give = up ? v[i] : v[i + n / 2];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
      float y = v[0];
#pragma unroll
      for (; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
      best = fmaxf(best, isfinite(y) ? y : INFINITY);
    }
    // lane bits from the top: page, head, copies
#pragma unroll
    for (int o = 8; o > 8 / GP; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
    if ((lane & 15) == 0 && x < np)
      p.score[((size_t)b * p.Hkv + h) * p.max_pages + c0 + x] = from_s[x] != nullptr ? best : -INFINITY;
    if (u + 1 == u1 || (u + 1) % per_head == 0) {  // the warp's last unit of this head
      const int first = max(units * warp / NW - (h - h_first) * per_head, 0);
      put_size(h, first, x0 / 2 + 1 - first);
    }
  }
}

// The score of one page in 64 bits (by one warp).  Not finite (NaN or infinite
// keys): first of all.
template <typename T, int D>
__device__ double score64(const PagedSelectArgs &p, const InvFreq &inv, const Seq &s, int b, int h, int c, int lane) {
  constexpr int PPL = D / 64, HALF = D / 2;
  const int page = pool_page(p, b, c);
  if (page < 0) return -INFINITY;
  const T *row = (const T *)p.summary + ((size_t)page * p.Hkv + h) * 2 * D;
  const T *q = (const T *)p.q + ((size_t)b * p.Hkv + h) * p.GS * D;
  const int turn = page_turn(p, s, c);
  double cs[PPL], sn[PPL], lo[2 * PPL], hi[2 * PPL];
#pragma unroll
  for (int e = 0; e < PPL; ++e) {
    const int k = PPL * lane + e;
    sincos_fp64((double)turn * inv.v[k], sn[e], cs[e]);
    lo[2 * e] = to_f(row[k]), hi[2 * e] = to_f(row[D + k]);
    lo[2 * e + 1] = to_f(row[HALF + k]), hi[2 * e + 1] = to_f(row[D + HALF + k]);
  }
  double best = -INFINITY;
  for (int g = 0; g < p.GS; ++g) {
    double x = 0.0;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < PPL; ++e) {
      const int k = PPL * lane + e;
      const double qa = to_f(q[(size_t)g * D + k]), qb = to_f(q[(size_t)g * D + HALF + k]);
      const double ta = qa * cs[e] - qb * sn[e], tb = qb * cs[e] + qa * sn[e];
      const double pa = ta * lo[2 * e], pb = ta * hi[2 * e], pc = tb * lo[2 * e + 1], pd = tb * hi[2 * e + 1];
      x += (pa > pb ? pa : pb) + (pc > pd ? pc : pd);
      bad = bad || isnan(pa) || isnan(pb) || isnan(pc) || isnan(pd);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (!isfinite(x) || __any_sync(0xffffffffu, bad)) return INFINITY;
    best = fmax(best, x);
  }
  return best;
}

// order-preserving whole numbers of floating values (no NaN among them)
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x == 0.0 ? 0.0 : x);
  return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}
__device__ __forceinline__ float unorder(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// The k-th largest (k >= 1) of the keys key(0 .. n-1), by the whole block: one
// digit of eight bits at a time, from the top.  *above: how many are larger.
template <int NT_SEL, typename K, typename F>
__device__ K kth_largest(F key, int n, int k, int *above) {
  __shared__ int hist[256];
  __shared__ int s_digit, s_left;
  const int tid = threadIdx.x;
  K prefix = 0;
  int left = k;
  for (int shift = 8 * (int)sizeof(K) - 8; shift >= 0; shift -= 8) {
    for (int x = tid; x < 256; x += NT_SEL) hist[x] = 0;
    __syncthreads();
    for (int x = tid; x < n; x += NT_SEL) {
      const K v = key(x);
      if (shift + 8 >= 8 * (int)sizeof(K) || (v >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&hist[(int)(v >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid < 32) {
      // lane: digits 255 - 8 lane downwards
      int c[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += c[e] = hist[255 - 8 * tid - e];
      int before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (tid >= o) before += y;
      }
      before -= sum;
      if (before < left && left <= before + sum) {
        int e = 0;
        while (before + c[e] < left) before += c[e++];
        s_digit = 255 - 8 * tid - e;
        s_left = left - before;
      }
    }
    __syncthreads();
    prefix |= (K)s_digit << shift;
    left = s_left;
    __syncthreads();
  }
  *above = k - left;
  return prefix;
}

// exclusive prefix sum of x over the block; *total: the sum
template <int NT_SEL>
__device__ int block_scan(int x, int *total) {
  __shared__ int s_warp[NT_SEL / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = y;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < NT_SEL / 32; ++w) {
    if (w < warp) before += s_warp[w];
    sum += s_warp[w];
  }
  *total = sum;
  return before + y - x;
}

// Of R keys per thread (whole numbers, 0: none): the k-th largest, by the whole
// block, two bits at a time from the first in which they differ.  Once exactly k
// keys are at or above a threshold, the least of them is it.
template <int NT_SEL, int R>
__device__ uint32_t kth_largest_held(const uint32_t (&key)[R], int k) {
  constexpr int NW = NT_SEL / 32;
  __shared__ uint64_t s_count[2][NW];
  __shared__ uint32_t s_least[NW], s_range[2][NW];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t lo = 0xffffffffu, hi = 0;
#pragma unroll
  for (int x = 0; x < R; ++x) {
    if (key[x] != 0) lo = min(lo, key[x]);
    hi = max(hi, key[x]);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) s_range[0][warp] = lo, s_range[1][warp] = hi;
  __syncthreads();
  lo = __reduce_min_sync(0xffffffffu, lane < NW ? s_range[0][lane] : 0xffffffffu);
  hi = __reduce_max_sync(0xffffffffu, lane < NW ? s_range[1][lane] : 0u);
  if (lo == hi) return lo;
  const int first = (31 - __clz(lo ^ hi)) & ~1;  // the two bits from here: the first that differ among them
  uint32_t prefix = first == 30 ? 0u : hi >> (first + 2) << (first + 2);
  for (int shift = first, round = 0; shift >= 0; shift -= 2, round ^= 1) {
    // how many keys are at or above prefix + 1, 2, 3 << shift
    int n1 = 0, n2 = 0, n3 = 0;
#pragma unroll
    for (int x = 0; x < R; ++x) {
      n1 += key[x] >= prefix + (1u << shift);
      n2 += key[x] >= prefix + (2u << shift);
      n3 += key[x] >= prefix + (3u << shift);
    }
    const uint32_t n12 = __reduce_add_sync(0xffffffffu, (uint32_t)(n1 | n2 << 16));
    const uint32_t nn3 = __reduce_add_sync(0xffffffffu, (uint32_t)n3);
    if (lane == 0) s_count[round][warp] = (uint64_t)nn3 << 32 | n12;
    __syncthreads();
    const uint64_t y = lane < NW ? s_count[round][lane] : 0;
    const uint32_t a12 = __reduce_add_sync(0xffffffffu, (uint32_t)y);
    const uint32_t a3 = __reduce_add_sync(0xffffffffu, (uint32_t)(y >> 32));
    const uint32_t a1 = a12 & 0xffffu, a2 = a12 >> 16, want = (uint32_t)k;
    const uint32_t digit = a3 >= want ? 3 : a2 >= want ? 2 : a1 >= want ? 1 : 0;
    prefix += digit << shift;
    if (digit > 0 && (digit == 3 ? a3 : digit == 2 ? a2 : a1) == want) break;
  }
  uint32_t least = 0xffffffffu;
#pragma unroll
  for (int x = 0; x < R; ++x)
    if (key[x] >= prefix && key[x] != 0) least = min(least, key[x]);
  least = __reduce_min_sync(0xffffffffu, least);
  if (lane == 0) s_least[warp] = least;
  __syncthreads();
  return __reduce_min_sync(0xffffffffu, lane < NW ? s_least[lane] : 0xffffffffu);
}

// One (sequence, kv head).  With T the k-th largest fp32 score and eps a bound
// of every fp32 score's error, the k-th largest true score is within eps of T:
// a page scored above T + 2 eps is surely chosen, one below T - 2 eps surely
// not, and the few between are decided by their scores in 64 bits (equal ones:
// the lower page first).  Where all of those are needed anyway, as nearly
// always, nothing is left to decide; a sequence of up to R pages per thread then
// has its scores read once and kept in registers.
//
// eps: a score is a sum of D terms |q'_d m_d|, m_d the larger of |min_d| and
// |max_d|, whose sizes add up to at most |q| |m| (2-norms; turning leaves |q|
// as it is).  Relative to that, with u = 2^-24: the turned query is off by at
// most 7u (cosine and sine within 3u, one product, one sum), hi + lo and
// hi - lo by 1u each, and a term goes through at most 8 + 5 further sums:
// 22u = 1.32e-6.  1.9e-6 is used (and twice that for twice the score), as the norms and thresholds are rounded too;
// 2e-18 makes up for squares and 1e-36 for products below the normal range.  The
// angles in 64 bits are themselves products rounded to 2^-53, which moves the turned
// query by at most L 2^-53 times the highest frequency (far below 1.9e-6 unless
// positions are near 2^30 or the base is below 1).
template <typename T, int D, int NT_SEL, int R>
__global__ void __launch_bounds__(NT_SEL)
select_kernel(const __grid_constant__ PagedSelectArgs p, const __grid_constant__ InvFreq inv) {
  constexpr int NW = NT_SEL / 32;
  constexpr int FEW = 64;  // undecided pages that are settled in shared memory
  __shared__ float s_max[2][NW];
  __shared__ int s_und[FEW];
  __shared__ double s_fine[FEW];
  __shared__ bool s_take[FEW];
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  let_next_kernel_come();
  wait_for_kernel_before();
  const int pages = pages_of(p, b);
  const size_t row = (size_t)b * p.Hkv + h;
  int32_t *list = p.list + row * p.n_select;
  if (pages <= p.n_select) {
    for (unsigned x = tid; x < (unsigned)p.n_select; x += NT_SEL) list[x] = x < (unsigned)pages ? (int)x : -1;
    return;
  }
  float *score = p.score + row * p.max_pages;
  // candidates: the pages between the first ones and the newest
  const int lo = p.n_first, n = pages - p.n_first - p.n_last, k = p.n_select - p.n_first - p.n_last;
  const bool held = pages <= R * NT_SEL;
  // thread: pages R tid .. R tid + R - 1
  float mine[R];
  uint32_t key[R];
  if (held) {
#pragma unroll
    for (int x = 0; x < R; ++x) mine[x] = R * tid + x < pages ? score[R * tid + x] : -INFINITY;
  }
  float above_t = INFINITY, below_t = INFINITY;  // chosen above the one, undecided from the other on
  if (k > 0) {
    // eps
    float size = 0.f;
    for (int x = tid; x < (pages + 1) / 2; x += NT_SEL) size = max_nan(size, p.size[row * p.max_pages + x]);
    float qs = 0.f;
    const T *q = (const T *)p.q + row * p.GS * D;
    for (int g = warp; g < p.GS; g += NW) {
      float x = 0.f;
#pragma unroll
      for (int d = lane; d < D; d += 32) x = fmaf(to_f(q[g * D + d]), to_f(q[g * D + d]), x);
      qs = max_nan(qs, warp_sum(x));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) size = max_nan(size, __shfl_xor_sync(0xffffffffu, size, o));
    if (lane == 0) s_max[0][warp] = size, s_max[1][warp] = qs;
    float t;
    if (held) {
#pragma unroll
      for (int x = 0; x < R; ++x) {
        const int c = R * tid + x;
        key[x] = c >= lo && c < lo + n ? order_key(mine[x]) : 0u;
      }
      t = unorder(kth_largest_held<NT_SEL, R>(key, k));
    } else {
      int above;
      t = unorder(kth_largest<NT_SEL, uint32_t>([&](int x) { return order_key(score[lo + x]); }, n, k, &above));
    }
    __syncthreads();
    float m2 = 0.f, q2 = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) m2 = max_nan(m2, s_max[0][w]), q2 = max_nan(q2, s_max[1][w]);
    const float rel = 3.8e-6f + 2.4e-16f * (float)p.seqlens[b] * (float)fmax(inv.v[0], inv.v[D / 2 - 1]);
    const float eps = rel * (sqrtf(q2) + 2e-18f) * (sqrtf(m2) + 2e-18f) + 1e-36f;
    if (eps < 1e30f) {  // no square or score near overflow, nothing infinite or NaN
      above_t = t + 2.f * eps;
      below_t = t - 2.f * eps;
    } else {  // fp32 says nothing here: all undecided
      below_t = -INFINITY;
    }
  }
  if (held) {
    bool yes[R], near_s[R];
    int sure = 0, maybe = 0;
#pragma unroll
    for (int x = 0; x < R; ++x) {
      const int c = R * tid + x;
      const bool in = c < pages, forced = in && (c < lo || c >= lo + n);
      const bool top = in && k > 0 && mine[x] > above_t, near = in && k > 0 && !top && mine[x] >= below_t;
      near_s[x] = near && !forced;
      yes[x] = forced || top || near;
      sure += forced || top;
      maybe += near_s[x];
    }
    int both;
    const int at = block_scan<NT_SEL>(sure | maybe << 16, &both);
    if ((both & 0xffff) + (both >> 16) == p.n_select) {
      int out = (at & 0xffff) + (at >> 16);
#pragma unroll
      for (int x = 0; x < R; ++x)
        if (yes[x]) list[out++] = R * tid + x;
      return;
    }
    const int und = both >> 16, need = p.n_select - (both & 0xffff);
    if (und <= FEW) {
      int x1 = at >> 16;
#pragma unroll
      for (int x = 0; x < R; ++x)
        if (near_s[x]) s_und[x1++] = R * tid + x;
      __syncthreads();
      for (int x = warp; x < und; x += NW) {
        const double v = score64<T, D>(p, inv, seq_of(p, b), b, h, s_und[x], lane);
        if (lane == 0) s_fine[x] = v;
      }
      __syncthreads();
      if (tid < und) {  // in ascending order of page: the lower wins a tie
        int rank = 0;
        for (int y = 0; y < und; ++y) rank += s_fine[y] > s_fine[tid] || (s_fine[y] == s_fine[tid] && y < tid);
        s_take[tid] = rank < need;
      }
      __syncthreads();
      x1 = at >> 16;
      int n_yes = 0;
#pragma unroll
      for (int x = 0; x < R; ++x) {
        if (near_s[x]) yes[x] = s_take[x1++];
        n_yes += yes[x];
      }
      int sum, out = block_scan<NT_SEL>(n_yes, &sum);
#pragma unroll
      for (int x = 0; x < R; ++x)
        if (yes[x]) list[out++] = R * tid + x;
      return;
    }
  }
  float *mark = p.mark + row * p.max_pages;
  double *fine = p.fine + row * p.max_pages;
  int32_t *amb = p.amb + row * p.max_pages;
  int sure = 0, und = 0;
  for (int x0 = 0; x0 < pages; x0 += NT_SEL) {
    const int c = x0 + tid;
    bool yes = false, maybe = false;
    if (c < pages) {
      const bool forced = c < lo || c >= pages - p.n_last;
      const float v = score[c];
      yes = forced || (k > 0 && v > above_t);
      maybe = !yes && k > 0 && v >= below_t;
      mark[c] = yes ? 1.f : 0.f;
    }
    int sum;
    const int at = block_scan<NT_SEL>(maybe ? 1 : 0, &sum);
    if (maybe) amb[und + at] = c;
    und += sum;
    block_scan<NT_SEL>(yes ? 1 : 0, &sum);
    sure += sum;
  }
  __syncthreads();
  const int need = p.n_select - sure;  // of the und undecided ones, in ascending order of page
  if (need == und) {
    for (int x = tid; x < und; x += NT_SEL) mark[amb[x]] = 1.f;
  } else if (need > 0) {
    for (int x = warp; x < und; x += NT_SEL / 32) {
      const double v = score64<T, D>(p, inv, seq_of(p, b), b, h, amb[x], lane);
      if (lane == 0) fine[x] = v;
    }
    __syncthreads();
    int above;
    const uint64_t kt = kth_largest<NT_SEL, uint64_t>([&](int x) { return order_key(fine[x]); }, und, need, &above);
    int equal = need - above;  // of those equal to the last chosen, the first
    for (int x0 = 0; x0 < und; x0 += NT_SEL) {
      const int x = x0 + tid;
      const uint64_t v = x < und ? order_key(fine[x]) : 0;
      const bool eq = x < und && v == kt;
      int sum;
      const int at = block_scan<NT_SEL>(eq ? 1 : 0, &sum);
      if (x < und && (v > kt || (eq && at < equal))) mark[amb[x]] = 1.f;
      equal -= min(equal, sum);
    }
  }
  __syncthreads();
  int out = 0;
  for (int x0 = 0; x0 < pages; x0 += NT_SEL) {
    const int c = x0 + tid;
    const bool yes = c < pages && mark[c] != 0.f;
    int sum;
    const int at = block_scan<NT_SEL>(yes ? 1 : 0, &sum);
    if (yes) list[out + at] = c;
    out += sum;
  }
}

template <typename T, int D>
cudaError_t launch(const PagedSelectArgs &args, const InvFreq &inv, const TurnFreq &turn, cudaStream_t st) {
  PagedSelectArgs a = args;
  const int gp = a.GS == 1 ? 1 : a.GS == 2 ? 2 : a.GS <= 4 ? 4 : 8;
  if (a.max_pages > a.n_select) {  // some sequence may have more pages than the list
    // Many CTAs: 128 threads each, so that four of them share an SM and one
    // loads while another computes (32 sequences up to 32K: 34 us against 41).
    // Fewer than four per SM: 256 threads, for the time of one (128K: 14 us
    // against 18).
    const dim3 grid((a.max_pages + SP - 1) / SP, a.B, (a.Hkv + SCORE_HEADS - 1) / SCORE_HEADS);
    const bool many = (long long)grid.x * grid.y * grid.z >= 4 * 148;
#define JL_SCORE(GP) (many ? score_kernel<T, D, GP, 128> : score_kernel<T, D, GP, 256>)
    const auto kernel = gp == 1 ? JL_SCORE(1) : gp == 2 ? JL_SCORE(2) : gp == 4 ? JL_SCORE(4) : JL_SCORE(8);
#undef JL_SCORE
    constexpr int smem = score_smem<T, D>();
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = launch_overlapped(kernel, grid, many ? 128 : 256, smem, st, a, turn);
    if (e != cudaSuccess) return e;
  }
  // few pages: few threads, whose barriers are short, each with four pages in
  // registers (one sequence, both kernels: 512 pages 11.8 us, with 512 threads 13.4; 2048
  // pages 12.4 us, with 1024 threads 15.1; 4096 pages 21.8 us, with eight pages a
  // thread 24.8)
  const dim3 grid(a.Hkv, a.B);
  if (a.max_pages <= 512) return launch_overlapped(select_kernel<T, D, 128, 4>, grid, 128, 0, st, a, inv);
  if (a.max_pages <= 2048) return launch_overlapped(select_kernel<T, D, 512, 4>, grid, 512, 0, st, a, inv);
  if (a.max_pages <= 4096) return launch_overlapped(select_kernel<T, D, 1024, 4>, grid, 1024, 0, st, a, inv);
  return launch_overlapped(select_kernel<T, D, 1024, 8>, grid, 1024, 0, st, a, inv);
}

}  // namespace pgs

cudaError_t launch_paged_select(bool bf16, int D, const PagedSelectArgs &a, const InvFreq &inv, const TurnFreq &turn,
                                cudaStream_t st) {
  if (D == 128)
    return bf16 ? pgs::launch<__nv_bfloat16, 128>(a, inv, turn, st) : pgs::launch<float, 128>(a, inv, turn, st);
  return bf16 ? pgs::launch<__nv_bfloat16, 64>(a, inv, turn, st) : pgs::launch<float, 64>(a, inv, turn, st);
}

}  // namespace jl
