// Append to a paged cache (sm_100a): rotates new keys (and queries) by their
// absolute positions, writes keys and values into their pages, and keeps each
// page's per-channel key range (minimum and maximum), from which pages are
// later scored without reading them.
//
// Token at position p, pair (x_k, x_{k + D/2}), angle a = p theta^(-2k/D):
//   (x_k cos a - x_{k+D/2} sin a,  x_{k+D/2} cos a + x_k sin a)
// in fp32 from angles formed in 64 bits, rounded once to the cache's type.
#include "jl_paged.cuh"

namespace jl {

namespace pga {

constexpr int NT = 128;
constexpr int CHUNK = 64;  // tokens whose angles are held at a time

template <typename T>
struct Vec;  // 16 bytes of a row
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void load(const float *p, float (&x)[4]) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  }
  static __device__ __forceinline__ void store(float *p, const float (&x)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// CTA (page of the sequence's new tokens, kv head, sequence): that page's new
// tokens for one kv head and its query heads, so a page's range is reduced by
// one CTA, without atomics.  Thread: 16 bytes of the first half of a row and
// the partner 16 bytes of the second, tokens tl, tl + TL, ...
template <typename T, int D, bool ROT>
__global__ void __launch_bounds__(NT)
paged_append_kernel(const __grid_constant__ PagedAppendArgs a, const __grid_constant__ InvFreq inv) {
  constexpr int N = Vec<T>::N, HALF = D / 2, CT = HALF / N, TL = NT / CT;
  __shared__ float2 cs[ROT ? CHUNK : 1][HALF];
  __shared__ float red[2][NT / 32][D];
  const int b = blockIdx.z, kvh = blockIdx.y;
  let_next_kernel_come();
  wait_for_kernel_before();
  const int c0 = a.cu[b], n = a.cu[b + 1] - c0, L = a.seqlens[b];
  // outside the contract: the sequence is left alone
  if (c0 < 0 || n <= 0 || n > a.max_new || n > L || c0 > a.T - n) return;
  const int P = 1 << a.page_log2;
  const int lp = ((L - n) >> a.page_log2) + blockIdx.x;  // logical page
  const long long pb = (long long)lp << a.page_log2;
  if (pb >= L) return;
  const int ja = (int)max(pb, (long long)(L - n)), je = (int)min(pb + P, (long long)L);  // this page's new tokens
  int page = lp < a.max_pages ? a.table[(long long)b * a.table_stride + lp] : -1;
  if (page >= a.n_pages) page = -1;  // no such page: only the queries are written
  const int tl = threadIdx.x / CT, ch = threadIdx.x % CT;
  const int Hq = a.Hkv * a.GS;
  float lo[2][N], hi[2][N];
#pragma unroll
  for (int e = 0; e < N; ++e) lo[0][e] = lo[1][e] = INFINITY, hi[0][e] = hi[1][e] = -INFINITY;

  for (int j0 = ja; j0 < je; j0 += CHUNK) {
    const int m = min(CHUNK, je - j0);
    if constexpr (ROT) {
      // thread: one pair's angles of a run of tokens; the first in 64 bits,
      // the next by 64-bit steps of one position
      constexpr int RUNS = NT / HALF;
      const int k = threadIdx.x % HALF, r = threadIdx.x / HALF;
      const int per = (m + RUNS - 1) / RUNS, x0 = r * per, x1 = min(m, x0 + per);
      __syncthreads();
      if (x0 < x1) {
        double c, s, c1, s1;
        sincos_fp64((double)(j0 + x0) * inv.v[k], s, c);
        sincos_fp64(inv.v[k], s1, c1);
        for (int x = x0; x < x1; ++x) {
          cs[x][k] = make_float2((float)c, (float)s);
          const double cn = c * c1 - s * s1;
          s = s * c1 + c * s1;
          c = cn;
        }
      }
      __syncthreads();
    }
    for (int x = tl; x < m; x += TL) {
      const int j = j0 + x;
      const size_t tok = (size_t)c0 + (size_t)(j - (L - n));
      float co[N], si[N];
      if constexpr (ROT) {
#pragma unroll
        for (int e = 0; e < N; ++e) co[e] = cs[x][ch * N + e].x, si[e] = cs[x][ch * N + e].y;
      }
      auto turn = [&](float (&u)[N], float (&v)[N]) {
        if constexpr (ROT) {
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const float t = fmaf(u[e], co[e], -(v[e] * si[e]));
            v[e] = fmaf(v[e], co[e], u[e] * si[e]);
            u[e] = t;
          }
        }
      };
      if (page >= 0) {
        const size_t src = (tok * a.Hkv + kvh) * D + ch * N;
        const size_t dst = (size_t)page * a.page_stride + ((size_t)(j & (P - 1)) * a.Hkv + kvh) * D + ch * N;
        float u[N], v[N];
        Vec<T>::load((const T *)a.k + src, u);
        Vec<T>::load((const T *)a.k + src + HALF, v);
        turn(u, v);
#pragma unroll
        for (int e = 0; e < N; ++e) {  // the range is that of the stored values
          u[e] = to_f(from_f<T>(u[e]));
          v[e] = to_f(from_f<T>(v[e]));
          lo[0][e] = min_nan(lo[0][e], u[e]), hi[0][e] = max_nan(hi[0][e], u[e]);
          lo[1][e] = min_nan(lo[1][e], v[e]), hi[1][e] = max_nan(hi[1][e], v[e]);
        }
        Vec<T>::store((T *)a.k_pages + dst, u);
        Vec<T>::store((T *)a.k_pages + dst + HALF, v);
        *reinterpret_cast<uint4 *>((T *)a.v_pages + dst) = *reinterpret_cast<const uint4 *>((const T *)a.v + src);
        *reinterpret_cast<uint4 *>((T *)a.v_pages + dst + HALF) =
            *reinterpret_cast<const uint4 *>((const T *)a.v + src + HALF);
      }
      if (ROT && a.q != nullptr) {
        for (int g = 0; g < a.GS; ++g) {
          const size_t at = (tok * Hq + (size_t)kvh * a.GS + g) * D + ch * N;
          float u[N], v[N];
          Vec<T>::load((const T *)a.q + at, u);
          Vec<T>::load((const T *)a.q + at + HALF, v);
          turn(u, v);
          Vec<T>::store((T *)a.q_out + at, u);
          Vec<T>::store((T *)a.q_out + at + HALF, v);
        }
      }
    }
  }

  if (a.summary == nullptr || page < 0) return;  // uniform over the CTA
  // lanes of a warp with the same chunk, then the warps
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int e = 0; e < N; ++e) {
#pragma unroll
      for (int o = CT; o < 32; o <<= 1) {
        lo[h][e] = min_nan(lo[h][e], __shfl_xor_sync(0xffffffffu, lo[h][e], o));
        hi[h][e] = max_nan(hi[h][e], __shfl_xor_sync(0xffffffffu, hi[h][e], o));
      }
      if ((threadIdx.x & 31) < CT) {
        red[0][threadIdx.x >> 5][h * HALF + ch * N + e] = lo[h][e];
        red[1][threadIdx.x >> 5][h * HALF + ch * N + e] = hi[h][e];
      }
    }
  __syncthreads();
  for (int idx = threadIdx.x; idx < 2 * D; idx += NT) {
    const int side = idx / D, d = idx % D;
    float x = red[side][0][d];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) x = side == 0 ? min_nan(x, red[0][w][d]) : max_nan(x, red[1][w][d]);
    T *to = (T *)a.summary + (((size_t)page * a.Hkv + kvh) * 2 + side) * D + d;
    if (ja > pb) x = side == 0 ? min_nan(x, to_f(*to)) : max_nan(x, to_f(*to));  // the page had tokens before
    *to = from_f<T>(x);
  }
}

template <typename T, int D>
cudaError_t launch(bool rotate, const PagedAppendArgs &a, const InvFreq &inv, int batch, cudaStream_t st) {
  const int P = 1 << a.page_log2;
  const dim3 grid((unsigned)(((long long)a.max_new + 2 * P - 2) / P), a.Hkv, batch);
  const auto kernel = rotate ? paged_append_kernel<T, D, true> : paged_append_kernel<T, D, false>;
  return launch_overlapped(kernel, grid, NT, 0, st, a, inv);
}

}  // namespace pga

cudaError_t launch_paged_append(bool bf16, int D, bool rotate, const PagedAppendArgs &a, const InvFreq &inv, int batch,
                                cudaStream_t st) {
  if (D == 128)
    return bf16 ? pga::launch<__nv_bfloat16, 128>(rotate, a, inv, batch, st)
                : pga::launch<float, 128>(rotate, a, inv, batch, st);
  return bf16 ? pga::launch<__nv_bfloat16, 64>(rotate, a, inv, batch, st)
              : pga::launch<float, 64>(rotate, a, inv, batch, st);
}

}  // namespace jl
