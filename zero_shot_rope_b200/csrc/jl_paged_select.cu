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

constexpr int NT_SCORE = 256;
constexpr int NT_SEL = 512;

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

struct Seq {
  int L, pages, G, ni, j_local;
};
__device__ __forceinline__ Seq seq_of(const PagedSelectArgs &p, int b) {
  Seq s;
  s.L = p.seqlens[b];
  if (s.L < 0 || (long long)s.L > ((long long)p.max_pages << p.page_log2)) s.L = 0;  // outside the contract: no page
  s.pages = (int)(((long long)s.L + (1 << p.page_log2) - 1) >> p.page_log2);
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

// Scores in fp32.  A CTA takes 16 pages of a sequence: first their angles, once
// for all heads, then warps go through the kv heads with the head's queries in
// registers, UP pages at a time.  UP pages x GP heads are 16 sums (or fewer) per
// lane, which are added up over the lanes together: with each shuffle a lane
// hands over half of what it holds and keeps the other half.
constexpr int SCORE_PAGES = 16;
__host__ __device__ constexpr int pages_at_once(int gp) { return gp <= 4 ? 4 : 2; }

template <typename T, int D, int GP>
__global__ void __launch_bounds__(NT_SCORE)
score_kernel(const __grid_constant__ PagedSelectArgs p, const __grid_constant__ TurnFreq turn) {
  constexpr int PPL = D / 64, HALF = D / 2, UP = pages_at_once(GP), NV = UP * GP, NW = NT_SCORE / 32;
  __shared__ __align__(16) float2 ang[SCORE_PAGES][HALF];
  __shared__ int pool[SCORE_PAGES];
  const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = blockIdx.x * SCORE_PAGES;
  let_next_kernel_come();
  wait_for_kernel_before();
  const Seq s = seq_of(p, b);
  if (s.pages <= p.n_select) return;  // all of them are listed
  if (c0 >= s.pages) return;
  if (threadIdx.x < SCORE_PAGES)
    pool[threadIdx.x] = c0 + threadIdx.x < s.pages ? pool_page(p, b, c0 + threadIdx.x) : -1;
#pragma unroll
  for (int x = threadIdx.x; x < SCORE_PAGES * HALF; x += NT_SCORE) {
    const int c = x / HALF, k = x % HALF;
    float co, si;
    turn_cs(c0 + c < s.pages ? page_turn(p, s, c0 + c) : 0, turn.v[k], co, si);
    ang[c][k] = make_float2(co, si);
  }
  __syncthreads();
  const T *q = (const T *)p.q + (size_t)b * p.Hkv * p.GS * D;
  const int per_head = SCORE_PAGES / UP;
  const long long units = (long long)p.Hkv * per_head;
  const int u1 = (int)(units * (warp + 1) / NW);
  float qa[GP][PPL], qb[GP][PPL];
  int held = -1;  // the head whose queries they are
  for (int u = (int)(units * warp / NW); u < u1; ++u) {
    const int h = u / per_head, x0 = (u % per_head) * UP;
    if (c0 + x0 >= s.pages) continue;
    float la[UP][PPL], lb[UP][PPL], ha[UP][PPL], hb[UP][PPL];
    uint32_t mx = 0;
#pragma unroll
    for (int x = 0; x < UP; ++x) {
      const int page = pool[x0 + x];
      if (page >= 0) {
        const T *row = (const T *)p.summary + ((size_t)page * p.Hkv + h) * 2 * D;
        load_pairs<T, PPL>(row, HALF, lane, la[x], lb[x]);
        load_pairs<T, PPL>(row + D, HALF, lane, ha[x], hb[x]);
      } else {
#pragma unroll
        for (int e = 0; e < PPL; ++e) la[x][e] = lb[x][e] = ha[x][e] = hb[x][e] = 0.f;
      }
    }
    float best = -INFINITY;
    for (int g0 = 0; g0 < p.GS; g0 += GP) {
      if (held != h || p.GS > GP) {
#pragma unroll
        for (int g = 0; g < GP; ++g)  // a head twice is no other maximum
          load_pairs<T, PPL>(q + (size_t)(h * p.GS + min(g0 + g, p.GS - 1)) * D, HALF, lane, qa[g], qb[g]);
        held = h;
      }
      float v[NV];
#pragma unroll
      for (int x = 0; x < UP; ++x) {
        float2 cs[PPL];
#pragma unroll
        for (int e = 0; e < PPL; ++e) cs[e] = ang[x0 + x][PPL * lane + e];
#pragma unroll
        for (int g = 0; g < GP; ++g) {
          float y = 0.f;
#pragma unroll
          for (int e = 0; e < PPL; ++e) {
            // <R(-turn) k, q> = <k, R(turn) q>
            const float ta = fmaf(qa[g][e], cs[e].x, -(qb[g][e] * cs[e].y));
            const float tb = fmaf(qb[g][e], cs[e].x, qa[g][e] * cs[e].y);
            y = fmaf(ta, ta >= 0.f ? ha[x][e] : la[x][e], y);
            y = fmaf(tb, tb >= 0.f ? hb[x][e] : lb[x][e], y);
          }
          v[x * GP + g] = y;
        }
      }
      int o = 16;
#pragma unroll
      for (int n = NV; n > 1; n >>= 1, o >>= 1)
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
    for (int o = 16 / UP; o > 16 / NV; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
#pragma unroll
    for (int x = 0; x < UP; ++x)
#pragma unroll
      for (int e = 0; e < PPL; ++e) {
        // magnitudes as bits: a NaN stays above every number
        mx = max(max(mx, __float_as_uint(fabsf(la[x][e]))), __float_as_uint(fabsf(ha[x][e])));
        mx = max(max(mx, __float_as_uint(fabsf(lb[x][e]))), __float_as_uint(fabsf(hb[x][e])));
      }
    mx = __reduce_max_sync(0xffffffffu, mx);
    const size_t at = ((size_t)b * p.Hkv + h) * p.max_pages;
    const int x = lane / (32 / UP);
    if (lane % (32 / UP) == 0 && c0 + x0 + x < s.pages) p.score[at + c0 + x0 + x] = pool[x0 + x] >= 0 ? best : -INFINITY;
    if (lane == 0) p.mx[at + (c0 + x0) / UP] = __uint_as_float(mx);
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
  double best = -INFINITY;
  for (int g = 0; g < p.GS; ++g) {
    double x = 0.0;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < PPL; ++e) {
      const int k = PPL * lane + e;
      double sn, cs;
      sincos_fp64((double)turn * inv.v[k], sn, cs);
      const double qa = to_f(q[(size_t)g * D + k]), qb = to_f(q[(size_t)g * D + HALF + k]);
      const double ta = qa * cs - qb * sn, tb = qb * cs + qa * sn;
      const double pa = ta * to_f(row[k]), pb = ta * to_f(row[D + k]);
      const double pc = tb * to_f(row[HALF + k]), pd = tb * to_f(row[D + HALF + k]);
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
template <typename K, typename F>
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
// block, two bits at a time from the top.  Once exactly k keys are at or above
// a threshold, the least of them is it.
template <int R>
__device__ uint32_t kth_largest_held(const uint32_t (&key)[R], int k) {
  constexpr int NW = NT_SEL / 32;
  __shared__ uint64_t s_count[2][NW];
  __shared__ uint32_t s_least[NW];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t prefix = 0;
  for (int shift = 30, round = 0; shift >= 0; shift -= 2, round ^= 1) {
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
// always, nothing is left to decide; a sequence of up to R x 512 pages then has
// its scores read once and kept in registers.
//
// eps: with Mx the largest |min|, |max| of a page and Q the sum over channels
// of the length of the query's pair (which no rotation changes), a score is a
// sum of D terms |q'_d m_d| whose sizes add up to at most Q Mx.  Relative to
// that, with u = 2^-24: the turned query is off by at most 7u (cosine and sine
// within 3u, one product, one sum), taking the wrong side of a q' within its own
// error of zero costs at most 14u, and a term goes through at most 4 + 5 further
// roundings: 30u < 2^-19.  2^-18 is used: Q, Mx and the thresholds are rounded too.
template <typename T, int D, int R>
__global__ void __launch_bounds__(NT_SEL)
select_kernel(const __grid_constant__ PagedSelectArgs p, const __grid_constant__ InvFreq inv) {
  constexpr int NW = NT_SEL / 32;
  __shared__ float s_max[2][NW];
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  let_next_kernel_come();
  wait_for_kernel_before();
  const Seq s = seq_of(p, b);
  const size_t row = (size_t)b * p.Hkv + h;
  int32_t *list = p.list + row * p.n_select;
  if (s.pages <= p.n_select) {
    for (int x = tid; x < p.n_select; x += NT_SEL) list[x] = x < s.pages ? x : -1;
    return;
  }
  float *score = p.score + row * p.max_pages;
  // candidates: the pages between the first ones and the newest
  const int lo = p.n_first, n = s.pages - p.n_first - p.n_last, k = p.n_select - p.n_first - p.n_last;
  const bool held = s.pages <= R * NT_SEL;
  // thread: pages R tid .. R tid + R - 1
  float mine[R];
  uint32_t key[R];
  if (held) {
#pragma unroll
    for (int x = 0; x < R; ++x) mine[x] = R * tid + x < s.pages ? score[R * tid + x] : -INFINITY;
  }
  float above_t = INFINITY, below_t = INFINITY;  // chosen above the one, undecided from the other on
  if (k > 0) {
    // eps
    uint32_t mx = 0;
    const int groups = (s.pages + p.mx_pages - 1) / p.mx_pages;
    for (int x = tid; x < groups; x += NT_SEL) mx = max(mx, __float_as_uint(p.mx[row * p.max_pages + x]));
    float qs = 0.f;
    const T *q = (const T *)p.q + row * p.GS * D;
    for (int g = warp; g < p.GS; g += NW) {
      float x = 0.f;
#pragma unroll
      for (int d = lane; d < D / 2; d += 32) {
        const float u = to_f(q[g * D + d]), v = to_f(q[g * D + D / 2 + d]);
        x += 2.f * sqrtf(u * u + v * v);
      }
      qs = max_nan(qs, warp_sum(x));
    }
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (lane == 0) s_max[0][warp] = __uint_as_float(mx), s_max[1][warp] = qs;
    float t;
    if (held) {
#pragma unroll
      for (int x = 0; x < R; ++x) {
        const int c = R * tid + x;
        key[x] = c >= lo && c < lo + n ? order_key(mine[x]) : 0u;
      }
      t = unorder(kth_largest_held<R>(key, k));
    } else {
      int above;
      t = unorder(kth_largest<uint32_t>([&](int x) { return order_key(score[lo + x]); }, n, k, &above));
    }
    __syncthreads();
    float Mx = 0.f, Q = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) Mx = max_nan(Mx, s_max[0][w]), Q = max_nan(Q, s_max[1][w]);
    const float eps = 3.9e-6f * Q * Mx + 1e-36f;  // (1e-36: products below the normal range)
    if (eps < 1e30f) {                            // no score near overflow, and nothing infinite or NaN
      above_t = t + 2.f * eps;
      below_t = t - 2.f * eps;
    } else {  // fp32 says nothing here: all undecided
      below_t = -INFINITY;
    }
  }
  if (held) {
    bool yes[R];
    int sure = 0, maybe = 0;
#pragma unroll
    for (int x = 0; x < R; ++x) {
      const int c = R * tid + x;
      const bool in = c < s.pages, forced = in && (c < lo || c >= lo + n);
      const bool top = in && k > 0 && mine[x] > above_t, near = in && k > 0 && !top && mine[x] >= below_t;
      yes[x] = forced || top || near;
      sure += forced || top;
      maybe += !forced && near;
    }
    int both;
    const int at = block_scan(sure | maybe << 16, &both);
    if ((both & 0xffff) + (both >> 16) == p.n_select) {
      int out = (at & 0xffff) + (at >> 16);
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
  for (int x0 = 0; x0 < s.pages; x0 += NT_SEL) {
    const int c = x0 + tid;
    bool yes = false, maybe = false;
    if (c < s.pages) {
      const bool forced = c < lo || c >= s.pages - p.n_last;
      const float v = score[c];
      yes = forced || (k > 0 && v > above_t);
      maybe = !yes && k > 0 && v >= below_t;
      mark[c] = yes ? 1.f : 0.f;
    }
    int sum;
    const int at = block_scan(maybe ? 1 : 0, &sum);
    if (maybe) amb[und + at] = c;
    und += sum;
    block_scan(yes ? 1 : 0, &sum);
    sure += sum;
  }
  __syncthreads();
  const int need = p.n_select - sure;  // of the und undecided ones, in ascending order of page
  if (need == und) {
    for (int x = tid; x < und; x += NT_SEL) mark[amb[x]] = 1.f;
  } else if (need > 0) {
    for (int x = warp; x < und; x += NT_SEL / 32) {
      const double v = score64<T, D>(p, inv, s, b, h, amb[x], lane);
      if (lane == 0) fine[x] = v;
    }
    __syncthreads();
    int above;
    const uint64_t kt = kth_largest<uint64_t>([&](int x) { return order_key(fine[x]); }, und, need, &above);
    int equal = need - above;  // of those equal to the last chosen, the first
    for (int x0 = 0; x0 < und; x0 += NT_SEL) {
      const int x = x0 + tid;
      const uint64_t v = x < und ? order_key(fine[x]) : 0;
      const bool eq = x < und && v == kt;
      int sum;
      const int at = block_scan(eq ? 1 : 0, &sum);
      if (x < und && (v > kt || (eq && at < equal))) mark[amb[x]] = 1.f;
      equal -= min(equal, sum);
    }
  }
  __syncthreads();
  int out = 0;
  for (int x0 = 0; x0 < s.pages; x0 += NT_SEL) {
    const int c = x0 + tid;
    const bool yes = c < s.pages && mark[c] != 0.f;
    int sum;
    const int at = block_scan(yes ? 1 : 0, &sum);
    if (yes) list[out + at] = c;
    out += sum;
  }
}

template <typename T, int D>
cudaError_t launch(const PagedSelectArgs &args, const InvFreq &inv, const TurnFreq &turn, cudaStream_t st) {
  PagedSelectArgs a = args;
  const int gp = a.GS == 1 ? 1 : a.GS == 2 ? 2 : a.GS <= 4 ? 4 : 8;
  a.mx_pages = pages_at_once(gp);
  if (a.max_pages > a.n_select) {  // some sequence may have more pages than the list
    const auto kernel = gp == 1   ? score_kernel<T, D, 1>
                        : gp == 2 ? score_kernel<T, D, 2>
                        : gp == 4 ? score_kernel<T, D, 4>
                                  : score_kernel<T, D, 8>;
    const cudaError_t e = launch_overlapped(kernel, dim3((a.max_pages + SCORE_PAGES - 1) / SCORE_PAGES, a.B), NT_SCORE, 0,
                                            st, a, turn);
    if (e != cudaSuccess) return e;
  }
  const auto kernel = a.max_pages <= 4 * NT_SEL ? select_kernel<T, D, 4> : select_kernel<T, D, 16>;
  return launch_overlapped(kernel, dim3(a.Hkv, a.B), NT_SEL, 0, st, a, inv);
}

}  // namespace pgs

cudaError_t launch_paged_select(bool bf16, int D, const PagedSelectArgs &a, const InvFreq &inv, const TurnFreq &turn,
                                cudaStream_t st) {
  if (D == 128)
    return bf16 ? pgs::launch<__nv_bfloat16, 128>(a, inv, turn, st) : pgs::launch<float, 128>(a, inv, turn, st);
  return bf16 ? pgs::launch<__nv_bfloat16, 64>(a, inv, turn, st) : pgs::launch<float, 64>(a, inv, turn, st);
}

}  // namespace jl
