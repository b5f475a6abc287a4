// Append to a paged cache (sm_100a): rotates new keys (and queries) by their
// absolute positions, writes keys and values into their pages, and keeps each
// page's per-channel key range (minimum and maximum), from which pages are
// later scored without reading them.
//
// Token at position p, pair (x_k, x_{k + D/2}), angle a = p theta^(-2k/D):
//   (x_k cos a - x_{k+D/2} sin a,  x_{k+D/2} cos a + x_k sin a)
// in fp32, the angle as a 64-bit fraction of a turn, rounded once to the cache's
// type.
#include "jl_paged.cuh"

namespace jl {

namespace pga {

constexpr int CHUNK = 64;  // tokens whose angles are held at a time

template <typename T>
struct Vec;  // 16 bytes of a row
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(uint4 v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// CTA (page of the sequence's new tokens, a.heads kv heads, sequence): a page's
// new tokens, so that its ranges are reduced by one CTA, without atomics, and
// its angles are formed once for all heads.  Keys and values: a thread has 16
// bytes of the first half of a row and the partner 16 bytes of the second, of
// one head, for every TL-th token, and keeps their range in registers.  A token's
// heads lie side by side, so a warp's accesses do too.  Queries: the same 16 +
// 16 bytes of any (token, head).  The kernel does little but move rows, so a
// thread asks for its next UNROLL rows before it works on the last ones, and two
// CTAs share an SM: 32K tokens of 16/8 heads in 106 us, 5.1 TB/s, where a plain
// copy of as many bytes takes 89 us.
constexpr int MAX_HEADS = 8;
constexpr int UNROLL = 2;

template <typename T, int D, bool ROT, int NT>
__global__ void __launch_bounds__(NT, 512 / NT)
paged_append_kernel(const __grid_constant__ PagedAppendArgs a, const __grid_constant__ TurnFreq turn) {
  constexpr int N = Vec<T>::N, HALF = D / 2, CT = HALF / N;
  // the angles of CHUNK tokens (two neighbouring pairs: cos, cos, sin, sin), then the threads' ranges
  constexpr int ANG = ROT ? CHUNK * HALF * 8 : 0, RED = NT * 4 * N * 4;
  __shared__ __align__(16) uint8_t smem[ANG > RED ? ANG : RED];
  float4(*cs)[HALF / 2] = reinterpret_cast<float4(*)[HALF / 2]>(smem);
  float(*red)[NT] = reinterpret_cast<float(*)[NT]>(smem);
  const int b = blockIdx.z, h0 = blockIdx.y * a.heads, heads = min(a.heads, a.Hkv - h0);
  // (a thread's angles are all of one frequency, read once: lanes that read
  // different constants take turns)
  static_assert(NT % HALF == 0, "one frequency per thread");
  const unsigned long long w = ROT ? turn.v[threadIdx.x % HALF] : 0;
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
  const int cols = heads * CT, TL = NT / cols;
  const int col = threadIdx.x % cols, tl = threadIdx.x / cols;  // (threads past cols TL have no keys)
  const int ch = col % CT;
  float lo[2][N], hi[2][N];
#pragma unroll
  for (int e = 0; e < N; ++e) lo[0][e] = lo[1][e] = INFINITY, hi[0][e] = hi[1][e] = -INFINITY;
  auto rotate = [&](int x, int chunk, float (&u)[N], float (&v)[N]) {
    if constexpr (ROT) {
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const float4 f = cs[x][(chunk * N + e) / 2];
        float t = fmaf(u[e], f.x, -(v[e] * f.z));
        v[e] = fmaf(v[e], f.x, u[e] * f.z);
        u[e] = t;
        t = fmaf(u[e + 1], f.y, -(v[e + 1] * f.w));
        v[e + 1] = fmaf(v[e + 1], f.y, u[e + 1] * f.w);
        u[e + 1] = t;
      }
    }
  };

  for (int done = 0; done < je - ja; done += CHUNK) {  // (counted from ja: positions go up to 2^31 - 2)
    const int j0 = ja + done, m = min(CHUNK, je - j0);
    const size_t tok0 = (size_t)c0 + (size_t)(j0 - (L - n));
    if constexpr (ROT) {
      __syncthreads();
      for (int idx = threadIdx.x; idx < m * HALF; idx += NT) {
        const int x = idx / HALF, k = idx % HALF;
        float c, s;
        turn_cs(j0 + x, w, c, s);
        float *to = reinterpret_cast<float *>(&cs[x][k / 2]) + (k & 1);
        to[0] = c;
        to[2] = s;
      }
      __syncthreads();
    }
    if (page >= 0 && tl < TL) {
      const size_t from = (tok0 * a.Hkv + h0) * D + (size_t)(col / CT) * D + ch * N, step = (size_t)a.Hkv * D;
      const size_t to = (size_t)page * a.page_stride + ((size_t)(j0 & (P - 1)) * a.Hkv + h0) * D +
                        (size_t)(col / CT) * D + ch * N;
      uint4 buf[2][UNROLL / 2][4];
      auto load = [&](uint4 (&r)[UNROLL / 2][4], int x0) {
#pragma unroll
        for (int y = 0; y < UNROLL / 2; ++y) {
          const size_t at = from + (size_t)(x0 + y * TL) * step;
          if (x0 + y * TL < m) {
            r[y][0] = *reinterpret_cast<const uint4 *>((const T *)a.k + at);
            r[y][1] = *reinterpret_cast<const uint4 *>((const T *)a.k + at + HALF);
            r[y][2] = *reinterpret_cast<const uint4 *>((const T *)a.v + at);
            r[y][3] = *reinterpret_cast<const uint4 *>((const T *)a.v + at + HALF);
          }
        }
      };
      auto use = [&](const uint4 (&r)[UNROLL / 2][4], int x0) {
#pragma unroll
        for (int y = 0; y < UNROLL / 2; ++y) {
          const int x = x0 + y * TL;
          if (x >= m) break;
          const size_t at = to + (size_t)x * step;
          *reinterpret_cast<uint4 *>((T *)a.v_pages + at) = r[y][2];
          *reinterpret_cast<uint4 *>((T *)a.v_pages + at + HALF) = r[y][3];
          float u[N], v[N];
          Vec<T>::unpack(r[y][0], u);
          Vec<T>::unpack(r[y][1], v);
          rotate(x, ch, u, v);
          const uint4 pu = Vec<T>::pack(u), pv = Vec<T>::pack(v);
          *reinterpret_cast<uint4 *>((T *)a.k_pages + at) = pu;
          *reinterpret_cast<uint4 *>((T *)a.k_pages + at + HALF) = pv;
          Vec<T>::unpack(pu, u);  // the range is that of the stored values
          Vec<T>::unpack(pv, v);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            lo[0][e] = min_nan(lo[0][e], u[e]), hi[0][e] = max_nan(hi[0][e], u[e]);
            lo[1][e] = min_nan(lo[1][e], v[e]), hi[1][e] = max_nan(hi[1][e], v[e]);
          }
        }
      };
      const int batch = TL * UNROLL / 2;
      load(buf[0], tl);
      for (int x0 = tl; x0 < m; x0 += 2 * batch) {
        load(buf[1], x0 + batch);
        use(buf[0], x0);
        load(buf[0], x0 + 2 * batch);
        use(buf[1], x0 + batch);
      }
    }
    if (ROT && a.q != nullptr) {
      // pieces of a token's heads; a thread has one (or every NT-th) of every QL-th token
      const int row = heads * a.GS * CT, wide = min(row, NT), QL = NT / wide, ql = threadIdx.x / wide;
      const size_t step = (size_t)a.Hkv * a.GS * D;
      for (int i = threadIdx.x % wide; ql < QL && i < row; i += wide) {
        const size_t from = tok0 * step + ((size_t)h0 * a.GS + i / CT) * D + i % CT * N;
        uint4 buf[2][UNROLL][2];
        auto load = [&](uint4 (&r)[UNROLL][2], int x0) {
#pragma unroll
          for (int y = 0; y < UNROLL; ++y)
            if (x0 + y * QL < m) {
              r[y][0] = *reinterpret_cast<const uint4 *>((const T *)a.q + from + (size_t)(x0 + y * QL) * step);
              r[y][1] = *reinterpret_cast<const uint4 *>((const T *)a.q + from + (size_t)(x0 + y * QL) * step + HALF);
            }
        };
        auto use = [&](const uint4 (&r)[UNROLL][2], int x0) {
#pragma unroll
          for (int y = 0; y < UNROLL; ++y) {
            const int x = x0 + y * QL;
            if (x >= m) break;
            float u[N], v[N];
            Vec<T>::unpack(r[y][0], u);
            Vec<T>::unpack(r[y][1], v);
            rotate(x, i % CT, u, v);
            *reinterpret_cast<uint4 *>((T *)a.q_out + from + (size_t)x * step) = Vec<T>::pack(u);
            *reinterpret_cast<uint4 *>((T *)a.q_out + from + (size_t)x * step + HALF) = Vec<T>::pack(v);
          }
        };
        load(buf[0], ql);
        for (int x0 = ql; x0 < m; x0 += 2 * QL * UNROLL) {
          load(buf[1], x0 + QL * UNROLL);
          use(buf[0], x0);
          load(buf[0], x0 + 2 * QL * UNROLL);
          use(buf[1], x0 + QL * UNROLL);
        }
      }
    }
  }

  if (a.summary == nullptr || page < 0) return;  // uniform over the CTA
  __syncthreads();
  const int live = min(TL, je - ja);  // token lanes that had one
  if (tl < live) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      red[e][threadIdx.x] = lo[0][e], red[N + e][threadIdx.x] = lo[1][e];
      red[2 * N + e][threadIdx.x] = hi[0][e], red[3 * N + e][threadIdx.x] = hi[1][e];
    }
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < heads * 2 * D; idx += NT) {
    const int h = idx / (2 * D), side = idx / D % 2, d = idx % D;
    const int slot = side * 2 * N + d / HALF * N + d % N, at = h * CT + d % HALF / N;
    float x = red[slot][at];
    for (int y = 1; y < live; ++y) x = side == 0 ? min_nan(x, red[slot][at + y * cols]) : max_nan(x, red[slot][at + y * cols]);
    T *to = (T *)a.summary + (((size_t)page * a.Hkv + h0 + h) * 2 + side) * D + d;
    if (ja > pb) x = side == 0 ? min_nan(x, to_f(*to)) : max_nan(x, to_f(*to));  // the page had tokens before
    *to = from_f<T>(x);
  }
}

template <typename T, int D>
cudaError_t launch(bool rotate, const PagedAppendArgs &args, const TurnFreq &turn, int batch, cudaStream_t st) {
  PagedAppendArgs a = args;
  const int P = 1 << a.page_log2;
  const long long slots = ((long long)a.max_new + 2 * P - 2) / P;
  // all heads of a page in one CTA, up to 8, unless there are too few CTAs to fill
  // the GPU (22 sequences of 181 tokens, 12/4 heads, 128-key pages: 20 us against
  // 43; one token of one sequence: 3.7 against 5.1)
  a.heads = a.Hkv < MAX_HEADS ? a.Hkv : MAX_HEADS;
  while (a.heads > 1 && slots * batch * ((a.Hkv + a.heads - 1) / a.heads) < 2 * 148) a.heads = (a.heads + 1) / 2;
  const dim3 grid((unsigned)slots, (a.Hkv + a.heads - 1) / a.heads, batch);
  // a page of few rows keeps few threads busy, and more CTAs fit (32K tokens of 2/1
  // heads in 16-key pages, fp32, 768 pieces: 30 us against 39; 64 x 150 tokens of
  // 8/2 heads, 1280 pieces: 12 us against 9, so those keep 256 threads)
  const long long pieces = (long long)(P < a.max_new ? P : a.max_new) * a.heads * (1 + a.GS) * D * sizeof(T) / 32;
  if (pieces <= 1024) {
    const auto kernel = rotate ? paged_append_kernel<T, D, true, 128> : paged_append_kernel<T, D, false, 128>;
    return launch_overlapped(kernel, grid, 128, 0, st, a, turn);
  }
  const auto kernel = rotate ? paged_append_kernel<T, D, true, 256> : paged_append_kernel<T, D, false, 256>;
  return launch_overlapped(kernel, grid, 256, 0, st, a, turn);
}

}  // namespace pga

cudaError_t launch_paged_append(bool bf16, int D, bool rotate, const PagedAppendArgs &a, const TurnFreq &turn,
                                int batch, cudaStream_t st) {
  if (D == 128)
    return bf16 ? pga::launch<__nv_bfloat16, 128>(rotate, a, turn, batch, st)
                : pga::launch<float, 128>(rotate, a, turn, batch, st);
  return bf16 ? pga::launch<__nv_bfloat16, 64>(rotate, a, turn, batch, st)
              : pga::launch<float, 64>(rotate, a, turn, batch, st);
}

}  // namespace jl
