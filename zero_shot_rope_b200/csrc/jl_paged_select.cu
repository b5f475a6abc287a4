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
#pragma unroll
  for (int e = 0; e < PPL; ++e) {
    a[e] = to_f(row[PPL * lane + e]);
    b[e] = to_f(row[half + PPL * lane + e]);
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

// Scores in fp32.  One warp per page, all kv heads, so a page's angles are
// formed once; the turned query goes through registers head by head.
template <typename T, int D>
__global__ void __launch_bounds__(NT_SCORE)
score_kernel(const __grid_constant__ PagedSelectArgs p, const __grid_constant__ InvFreq inv) {
  constexpr int PPL = D / 64, HALF = D / 2;
  const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Seq s = seq_of(p, b);
  if (s.pages <= p.n_select) return;  // all of them are listed
  const T *q = (const T *)p.q + (size_t)b * p.Hkv * p.GS * D;
  const int step = gridDim.x * (NT_SCORE / 32);
  for (int c = blockIdx.x * (NT_SCORE / 32) + warp; c < s.pages; c += step) {
    const int page = pool_page(p, b, c);
    const int turn = page_turn(p, s, c);
    float co[PPL], si[PPL];
#pragma unroll
    for (int e = 0; e < PPL; ++e) angle_cs(turn, inv.v[PPL * lane + e], co[e], si[e]);
    for (int h = 0; h < p.Hkv; ++h) {
      float score = -INFINITY;
      uint32_t mx = 0;
      if (page >= 0) {
        const T *row = (const T *)p.summary + ((size_t)page * p.Hkv + h) * 2 * D;
        float la[PPL], lb[PPL], ha[PPL], hb[PPL];
        load_pairs<T, PPL>(row, HALF, lane, la, lb);
        load_pairs<T, PPL>(row + D, HALF, lane, ha, hb);
#pragma unroll
        for (int e = 0; e < PPL; ++e) {
          // magnitudes as bits: a NaN stays above every number
          mx = max(max(mx, __float_as_uint(fabsf(la[e]))), __float_as_uint(fabsf(ha[e])));
          mx = max(max(mx, __float_as_uint(fabsf(lb[e]))), __float_as_uint(fabsf(hb[e])));
        }
        for (int g = 0; g < p.GS; ++g) {
          float qa[PPL], qb[PPL], x = 0.f;
          load_pairs<T, PPL>(q + (size_t)(h * p.GS + g) * D, HALF, lane, qa, qb);
#pragma unroll
          for (int e = 0; e < PPL; ++e) {
            // <R(-turn) k, q> = <k, R(turn) q>
            const float ta = fmaf(qa[e], co[e], -(qb[e] * si[e]));
            const float tb = fmaf(qb[e], co[e], qa[e] * si[e]);
            x = fmaf(ta, ta >= 0.f ? ha[e] : la[e], x);
            x = fmaf(tb, tb >= 0.f ? hb[e] : lb[e], x);
          }
          x = warp_sum(x);
          score = isfinite(x) ? fmaxf(score, x) : INFINITY;
          if (score == INFINITY) break;
        }
      }
      mx = __reduce_max_sync(0xffffffffu, mx);
      if (lane == 0) {
        const size_t at = ((size_t)b * p.Hkv + h) * p.max_pages + c;
        p.score[at] = score;
        p.mx[at] = __uint_as_float(mx);
      }
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

// One (sequence, kv head).  With T the k-th largest fp32 score and eps a bound
// of every fp32 score's error, the k-th largest true score is within eps of T:
// a page scored above T + 2 eps is surely chosen, one below T - 2 eps surely
// not, and the few between are decided by their scores in 64 bits (equal ones:
// the lower page first).
//
// eps: with Mx the largest |min|, |max| of a page and Q the sum over channels
// of the length of the query's pair (which no rotation changes), a score is a
// sum of D terms |q'_d m_d| whose sizes add up to at most Q Mx.  Relative to
// that, with u = 2^-24: the turned query is off by at most 4u (cosine and sine
// rounded, one product, one sum), taking the wrong side of a q' within its own
// error of zero costs at most 8u, and a term goes through at most 4 + 5 further
// roundings: 21u < 2^-19.
template <typename T, int D>
__global__ void __launch_bounds__(NT_SEL)
select_kernel(const __grid_constant__ PagedSelectArgs p, const __grid_constant__ InvFreq inv) {
  __shared__ float s_max[2][NT_SEL / 32];
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Seq s = seq_of(p, b);
  const size_t row = (size_t)b * p.Hkv + h;
  int32_t *list = p.list + row * p.n_select;
  if (s.pages <= p.n_select) {
    for (int x = tid; x < p.n_select; x += NT_SEL) list[x] = x < s.pages ? x : -1;
    return;
  }
  float *score = p.score + row * p.max_pages;
  float *mark = p.mx + row * p.max_pages;
  double *fine = p.fine + row * p.max_pages;
  int32_t *amb = p.amb + row * p.max_pages;
  // candidates: the pages between the first ones and the newest
  const int lo = p.n_first, n = s.pages - p.n_first - p.n_last, k = p.n_select - p.n_first - p.n_last;
  float above_t = INFINITY, below_t = INFINITY;  // chosen above the one, undecided from the other on
  if (k > 0) {
    int above;
    const float t = unorder(kth_largest<uint32_t>([&](int x) { return order_key(score[lo + x]); }, n, k, &above));
    // eps
    uint32_t mx = 0;
    for (int x = tid; x < n; x += NT_SEL) mx = max(mx, __float_as_uint(mark[lo + x]));
    float qs = 0.f;
    const T *q = (const T *)p.q + row * p.GS * D;
    for (int g = warp; g < p.GS; g += NT_SEL / 32) {
      float x = 0.f;
      for (int d = lane; d < D / 2; d += 32) {
        const float u = to_f(q[g * D + d]), v = to_f(q[g * D + D / 2 + d]);
        x += 2.f * sqrtf(u * u + v * v);
      }
      qs = max_nan(qs, warp_sum(x));
    }
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (lane == 0) s_max[0][warp] = __uint_as_float(mx), s_max[1][warp] = qs;
    __syncthreads();
    float Mx = 0.f, Q = 0.f;
#pragma unroll
    for (int w = 0; w < NT_SEL / 32; ++w) Mx = max_nan(Mx, s_max[0][w]), Q = max_nan(Q, s_max[1][w]);
    // (2^-18.9: Q itself is rounded; 1e-36: products below the normal range)
    const float eps = 2.05e-6f * Q * Mx + 1e-36f;
    if (eps < 1e30f) {  // no score near overflow, and nothing infinite or NaN
      above_t = t + 2.f * eps;
      below_t = t - 2.f * eps;
    } else {  // fp32 says nothing here: all undecided
      below_t = -INFINITY;
    }
  }
  // above_t, below_t are rounded too: by 2^-24 of |t| + 2 eps, well inside the
  // slack of eps (|t| <= Q Mx)
  __syncthreads();
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
cudaError_t launch(const PagedSelectArgs &a, const InvFreq &inv, cudaStream_t st) {
  if (a.max_pages > a.n_select) {  // some sequence may have more pages than the list
    // about eight waves of eight warps per SM over the whole batch
    const int per = NT_SCORE / 32;
    const int most = (a.max_pages + per - 1) / per;
    int x = (148 * 8 + a.B - 1) / a.B;
    x = x < most ? x : most;
    score_kernel<T, D><<<dim3(x, a.B), NT_SCORE, 0, st>>>(a, inv);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  select_kernel<T, D><<<dim3(a.Hkv, a.B), NT_SEL, 0, st>>>(a, inv);
  return cudaGetLastError();
}

}  // namespace pgs

cudaError_t launch_paged_select(bool bf16, int D, const PagedSelectArgs &a, const InvFreq &inv, cudaStream_t st) {
  if (D == 128)
    return bf16 ? pgs::launch<__nv_bfloat16, 128>(a, inv, st) : pgs::launch<float, 128>(a, inv, st);
  return bf16 ? pgs::launch<__nv_bfloat16, 64>(a, inv, st) : pgs::launch<float, 64>(a, inv, st);
}

}  // namespace jl
