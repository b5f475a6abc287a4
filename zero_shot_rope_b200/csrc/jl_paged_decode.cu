// Decode of one new token per sequence over a paged cache (sm_100a): the fp32
// kernel and the combine.
//
// The attention is jl_bifocal_decode's: with i = L - 1, G = G(L) and
// n(p) = p - floor(p / G), key j is scored as
//     s_j = <q, R(-(n(j) - n(i))) k_j> / sqrt(D)   for i - j >= w0  (remote)
//     s_j = <q, k_j> / sqrt(D)                     for i - j <  w0  (local)
// and out = softmax(s) V over the visible keys: those below L, within the
// window if there is one, in the listed pages if there is a list.
#include "jl_paged.cuh"

namespace jl {

namespace pgd {

constexpr int NT = 256;
constexpr int NW = NT / 32;
constexpr float LN2 = 0.69314718055994531f;
constexpr float LOG2E_F = 1.4426950408889634f;

// PPL rotation pairs per lane: lane l holds elements PPL l .. PPL l + PPL - 1 of the
// first half of a row and the same of the second
template <int PPL>
__device__ __forceinline__ void load_pairs(const float *row, int half, int lane, float (&a)[PPL], float (&b)[PPL]) {
  if constexpr (PPL == 2) {
    const float2 x = *reinterpret_cast<const float2 *>(row + 2 * lane);
    const float2 y = *reinterpret_cast<const float2 *>(row + half + 2 * lane);
    a[0] = x.x, a[1] = x.y, b[0] = y.x, b[1] = y.y;
  } else {
    a[0] = row[lane];
    b[0] = row[half + lane];
  }
}

// One warp takes 8 keys (half a 16-key block) of every tile and keeps its own
// running maximum, sum and output; the warps are merged when the CTA leaves a
// (sequence, kv head, head block).  Each warp has its own ring of STAGES x 8 keys
// and values in shared memory, filled by asynchronous copies two tiles ahead (and
// the page looked up before that), so warps never wait for one another on the
// way.  A lane has four channels (two at head_dim 64) of all eight keys.
// The 8 keys x 4 heads partial scores are added up over the lanes together (with
// each shuffle a lane hands over half of what it holds), which leaves one whole
// score in each lane: every exponential is taken once.  The weights go through
// shared memory to all lanes.  Four heads at a time bound the registers.
constexpr int STAGES = 3;
constexpr int ring_bytes(int D) { return STAGES * NW * 8 * 2 * D * 4; }
constexpr int ctas_per_sm(int D) { return D == 64 ? 2 : 1; }  // by their rings: 96 and 192 KB

template <int D, int GP>
__global__ void __launch_bounds__(NT, ctas_per_sm(D))
paged_decode_kernel(const __grid_constant__ PagedDecodeArgs p, const __grid_constant__ TurnFreq turn) {
  constexpr int PPL = D / 64, HALF = D / 2, KW = 8;
  constexpr int GC = GP < 4 ? GP : 4, NC = GP / GC;  // heads at a time, and how often
  constexpr int NV = KW * GC;                        // their scores: NV lanes (and copies)
  __shared__ float red_ml[NW][GP][2];
  extern __shared__ __align__(16) float ring[];  // [STAGES][NW][K, V][KW][D], at the end of a piece the warps' outputs
  float(*red_o)[GP][D] = reinterpret_cast<float(*)[GP][D]>(ring);
  __shared__ __align__(16) float w_s[NW][KW][GC], f_s[NW][GC];
  let_next_kernel_come();
  wait_for_kernel_before();
  const PagedRun run = paged_plan<NT>(p);
  if (threadIdx.x == 0) p.cta_err[blockIdx.x] = 0;  // this kernel has no waits that could run out
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float scale = rsqrtf((float)D) * LOG2E_F;
  // this lane's score: key lk, head lg of the four
  const int lk = lane / (32 / KW), lg = lane / (32 / NV) % GC;
  unsigned long long w[PPL];
  float c1[PPL], s1[PPL];  // rotation by one position
#pragma unroll
  for (int e = 0; e < PPL; ++e) {
    w[e] = turn.v[PPL * lane + e];
    turn_cs(1, w[e], c1[e], s1[e]);
  }

  PagedWalk walk(p, run);
  while (walk.next(p)) {
    const PagedSeq &s = walk.s;
    const int b = walk.b, pair = walk.pair, u0 = walk.u0, u1 = walk.u1;
    const int kvh = pair / p.HB, hb = pair % p.HB;
    const int gh = min(PD_HEADS, p.GS - hb * PD_HEADS);
    const int h0 = kvh * p.GS + hb * PD_HEADS;  // first query head
    const int G = p.plain ? 1 : (int)group_size(s.L, p.w_pre);
    const int ni = corr_n(s.L - 1, G);
    const int j_local = (int)max(0LL, (long long)s.L - (long long)p.w0);

    float qa[GP][PPL], qb[GP][PPL], oa[GP][PPL], ob[GP][PPL];
    float m[NC], l[NC];  // of head lg (+ 4): maximum, and this lane's part of the sum
#pragma unroll
    for (int g = 0; g < GP; ++g) {
#pragma unroll
      for (int e = 0; e < PPL; ++e) qa[g][e] = qb[g][e] = oa[g][e] = ob[g][e] = 0.f;
      if (g < gh) {
        load_pairs<PPL>((const float *)p.q + ((size_t)b * p.Hq + h0 + g) * D, HALF, lane, qa[g], qb[g]);
#pragma unroll
        for (int e = 0; e < PPL; ++e) qa[g][e] *= scale, qb[g][e] *= scale;
      }
    }
#pragma unroll
    for (int x = 0; x < NC; ++x) m[x] = -INFINITY, l[x] = 0.f;

    // the warp's first key in tile u and its place in the pools
    auto look = [&](int u, int &j0, size_t &row) {
      int page;
      j0 = u < u1 ? paged_block(p, s, b, kvh, u, warp >> 1, page) : -1;
      if (j0 < 0) return;
      j0 += (warp & 1) * KW;
      if (j0 >= s.L || j0 + KW <= s.jw) {
        j0 = -1;
        return;
      }
      row = (size_t)page * p.page_stride + ((size_t)(j0 & ((1 << p.page_log2) - 1)) * p.Hkv + kvh) * D;
    };
    auto fetch = [&](int st, int j0, size_t row) {
      if (j0 >= 0) {
        constexpr int PIECES = D / 4;  // 16-byte pieces of a row
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(ring + ((st * NW + warp) * 2) * KW * D);
#pragma unroll
        for (int i = 0; i < KW * PIECES / 32; ++i) {
          const int x = (i * 32 + lane) / PIECES, c = (i * 32 + lane) % PIECES;
          const int n = j0 + x < s.L && j0 + x >= s.jw ? 16 : 0;  // other rows may hold anything: zeros
          const size_t at = n ? row + (size_t)x * p.Hkv * D + c * 4 : 0;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + (x * D + c * 4) * 4),
                       "l"((const float *)p.k + at), "r"(n)
                       : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + ((KW + x) * D + c * 4) * 4),
                       "l"((const float *)p.v + at), "r"(n)
                       : "memory");
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int ja, jb, jc;
    size_t row;
    look(u0, ja, row);
    fetch(0, ja, row);
    look(u0 + 1, jb, row);
    fetch(1, jb, row);
    int st = 0;
    for (int u = u0; u < u1; ++u) {
      look(u + 2, jc, row);
      const int j0 = ja;
      ja = jb, jb = jc;
      const int st0 = st, st2 = st == 0 ? 2 : st - 1;  // this tile's stage, and that of two tiles on
      st = st == 2 ? 0 : st + 1;
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();
      if (j0 < 0) {
        fetch(st2, jc, row);
        continue;
      }
      const float *kt = ring + (st0 * NW + warp) * 2 * KW * D, *vt = kt + KW * D;
      float ka[KW][PPL], kb[KW][PPL];
#pragma unroll
      for (int x = 0; x < KW; ++x) load_pairs<PPL>(kt + x * D, HALF, lane, ka[x], kb[x]);
      if (G > 1 && j0 < j_local) {
        // the angle of the first key, the next ones a step of one position or
        // none (j + 1 a multiple of G) further
        float c[PPL], sn[PPL];
        const int f = j0 / G;
        int rho = j0 - f * G;
#pragma unroll
        for (int e = 0; e < PPL; ++e) turn_cs(j0 - f - ni, w[e], c[e], sn[e]);
#pragma unroll
        for (int x = 0; x < KW; ++x) {
          if (j0 + x < j_local)
#pragma unroll
            for (int e = 0; e < PPL; ++e) rot_back(ka[x][e], kb[x][e], c[e], sn[e]);
          if (++rho == G) {
            rho = 0;
          } else {
#pragma unroll
            for (int e = 0; e < PPL; ++e) {
              const float cn = c[e] * c1[e] - sn[e] * s1[e];
              sn[e] = fmaf(sn[e], c1[e], c[e] * s1[e]);
              c[e] = cn;
            }
          }
        }
      }
#pragma unroll
      for (int y = 0; y < NC; ++y) {
        float d[NV];
#pragma unroll
        for (int x = 0; x < KW; ++x)
#pragma unroll
          for (int g = 0; g < GC; ++g) {
            float t = 0.f;
#pragma unroll
            for (int e = 0; e < PPL; ++e)
              t = fmaf(qa[y * GC + g][e], ka[x][e], fmaf(qb[y * GC + g][e], kb[x][e], t));
            d[x * GC + g] = t;
          }
        int o = 16;
#pragma unroll
        for (int n = NV; n > 1; n >>= 1, o >>= 1)
#pragma unroll
          for (int i = 0; i < n / 2; ++i) {
            const bool up = lane & o;
            const float keep = up ? d[i + n / 2] : d[i], give = up ? d[i] : d[i + n / 2];
            d[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        float sc = d[0];
#pragma unroll
        for (; o > 0; o >>= 1) sc += __shfl_xor_sync(0xffffffffu, sc, o);
        if (j0 + lk >= s.L || j0 + lk < s.jw) sc = -INFINITY;
        float top = sc;
#pragma unroll
        for (int x = 16; x >= 32 / KW; x >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, x));
        // the maximum is only moved when it has grown by more than 2^8
        const bool grow = !(top <= m[y] + 8.f) && !(top == -INFINITY);
        const bool any = __any_sync(0xffffffffu, grow);
        float f = 1.f;
        if (grow) {
          f = m[y] == -INFINITY ? 0.f : exp2f(m[y] - top);
          m[y] = top;
        }
        const float pr = exp2f(sc - (m[y] == -INFINITY ? 0.f : m[y]));
        l[y] = fmaf(l[y], f, pr);
        __syncwarp();
        w_s[warp][lk][lg] = pr;
        if (any) f_s[warp][lg] = f;
        __syncwarp();
        if (any) {
#pragma unroll
          for (int g = 0; g < GC; ++g) {
            const float fg = f_s[warp][g];
#pragma unroll
            for (int e = 0; e < PPL; ++e) oa[y * GC + g][e] *= fg, ob[y * GC + g][e] *= fg;
          }
        }
#pragma unroll
        for (int x = 0; x < KW; ++x) {
          float pg[GC], va[PPL], vb[PPL];
          load_pairs<PPL>(vt + x * D, HALF, lane, va, vb);
          if constexpr (GC == 4) {
            const float4 v = *reinterpret_cast<const float4 *>(w_s[warp][x]);
            pg[0] = v.x, pg[1] = v.y, pg[2] = v.z, pg[3] = v.w;
          } else {
#pragma unroll
            for (int g = 0; g < GC; ++g) pg[g] = w_s[warp][x][g];
          }
#pragma unroll
          for (int g = 0; g < GC; ++g)
#pragma unroll
            for (int e = 0; e < PPL; ++e) {
              oa[y * GC + g][e] = fmaf(pg[g], va[e], oa[y * GC + g][e]);
              ob[y * GC + g][e] = fmaf(pg[g], vb[e], ob[y * GC + g][e]);
            }
        }
      }
      // (what this stage held is free: the next fetch goes to another one)
      fetch(st2, jc, row);
    }

    // merge the warps
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int y = 0; y < NC; ++y) {
#pragma unroll
      for (int x = 16; x >= 32 / KW; x >>= 1) l[y] += __shfl_xor_sync(0xffffffffu, l[y], x);
      if (lk == 0) red_ml[warp][y * GC + lg][0] = m[y], red_ml[warp][y * GC + lg][1] = l[y];
    }
#pragma unroll
    for (int g = 0; g < GP; ++g)
#pragma unroll
      for (int e = 0; e < PPL; ++e) {
        red_o[warp][g][PPL * lane + e] = oa[g][e];
        red_o[warp][g][HALF + PPL * lane + e] = ob[g][e];
      }
    __syncthreads();
    const bool whole = u0 == 0 && u1 == s.tiles;
    const size_t slot = 2 * (size_t)blockIdx.x + (u0 > 0 ? 0 : 1);
    for (int idx = threadIdx.x; idx < gh * D; idx += NT) {
      const int g = idx / D, d = idx % D;
      float M = -INFINITY, L = 0.f, acc = 0.f;
      for (int x = 0; x < NW; ++x) M = max_nan(M, red_ml[x][g][0]);
      if (M != -INFINITY)
        for (int x = 0; x < NW; ++x) {
          const float f = exp2f(red_ml[x][g][0] - M);
          L = fmaf(f, red_ml[x][g][1], L);
          acc = fmaf(f, red_o[x][g][d], acc);
        }
      if (whole) {
        const size_t bh = (size_t)b * p.Hq + h0 + g;
        ((float *)p.out)[bh * D + d] = M != -INFINITY ? acc / L : 0.f;
        if (p.lse != nullptr && d == 0) p.lse[bh] = M != -INFINITY ? (M + log2f(L)) * LN2 : -INFINITY;
      } else {
        p.part_o[(slot * PD_HEADS + g) * D + d] = acc;
        if (d == 0) {
          p.part_ml[(slot * PD_HEADS + g) * 2] = M;
          p.part_ml[(slot * PD_HEADS + g) * 2 + 1] = L;
        }
      }
    }
    __syncthreads();  // the rings are free again
  }
}

// Joins the runs' partial results of one (kv head, head block) of a sequence,
// or writes zeros and -inf where the sequence has no key.  Pairs that one run
// covered whole were finished there.  Two dependent reads of global memory: the
// plan's table, then all maxima, sums and partial outputs at once (a thread
// reads its outputs before the weights they will get are known).
template <typename T, int D>
__global__ void __launch_bounds__(NT)
paged_combine_kernel(const __grid_constant__ PagedDecodeArgs p, int ctas) {
  constexpr int VPT = PD_HEADS * D / 4 / NT;  // float4s of the pair's outputs per thread, 1 (or a half: D = 64)
  constexpr int XG = VPT > 0 ? 1 : 2;         // groups of threads that share the runs
  constexpr int AHEAD = 8;                    // partial outputs a thread reads ahead
  __shared__ float w_s[PD_MAX_CTAS][PD_HEADS];
  __shared__ float M_s[PD_HEADS], L_s[PD_HEADS];
  __shared__ float4 acc_s[XG > 1 ? NT / 2 : 1];
  const int b = blockIdx.y, pair = blockIdx.x, pairs = p.Hkv * p.HB;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kvh = pair / p.HB, hb = pair % p.HB;
  const int gh = min(PD_HEADS, p.GS - hb * PD_HEADS);
  const int h0 = kvh * p.GS + hb * PD_HEADS;
  const size_t bh0 = (size_t)b * p.Hq + h0;
  let_next_kernel_come();
  wait_for_kernel_before();
  const long long first = p.tab[b], next = p.tab[b + 1], total = p.tab[p.B];
  if (pair == 0 && b == 0 && tid < 32) {  // fold the CTAs' error words
    int e = 0;
    for (int x = tid; x < ctas; x += 32) e |= p.cta_err[x];
    e = __reduce_or_sync(0xffffffffu, e);
    if (tid == 0) *p.err = e;
  }
  if (next == first) {
    for (int idx = tid; idx < gh * D; idx += NT) ((T *)p.out)[bh0 * D + idx] = from_f<T>(0.f);
    if (p.lse != nullptr && tid < gh) p.lse[bh0 + tid] = -INFINITY;
    return;
  }
  const long long tiles = div_up(next - first, pairs), chunk = div_up(total, ctas);
  const long long p0 = first + pair * tiles, p1 = p0 + tiles;
  auto cta_of = [&](long long t) {
    return total < (1ll << 31) ? (int)((unsigned)t / (unsigned)chunk) : (int)(t / chunk);
  };
  const int c0 = cta_of(p0), c1 = cta_of(p1 - 1);
  if (c0 == c1) return;  // covered whole
  const int ns = c1 - c0 + 1;
  // the pair's first run holds it in its second slot: the run has other pairs before it, or none
  auto slot = [&](int x) { return 2 * (size_t)(c0 + x) + (x == 0 ? 1 : 0); };
  // this thread's float4 of the outputs (head vg), over runs xg, xg + XG, ...
  const int v = tid % (PD_HEADS * D / 4), xg = tid / (PD_HEADS * D / 4);
  const int vg = v / (D / 4);
  const float4 *part = reinterpret_cast<const float4 *>(p.part_o) + v;
  const bool mine = vg < gh;
  float4 buf[AHEAD];
  if (mine)
#pragma unroll
    for (int a = 0; a < AHEAD; ++a)
      if (xg + a * XG < ns) buf[a] = part[slot(xg + a * XG) * (PD_HEADS * D / 4)];
  // warp g: maximum, weights and sum of head g
  {
    const int g = warp;
    const float2 *ml = reinterpret_cast<const float2 *>(p.part_ml) + g;
    float2 y[3];
    float M = -INFINITY;
    for (int x0 = 0; x0 < ns; x0 += 96)
#pragma unroll
      for (int a = 0; a < 3; ++a) {
        const int x = x0 + 32 * a + lane;
        y[a] = g < gh && x < ns ? ml[slot(x) * PD_HEADS] : make_float2(-INFINITY, 0.f);
        M = max_nan(M, y[a].x);
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f;
    for (int x0 = 0; x0 < ns; x0 += 96)
#pragma unroll
      for (int a = 0; a < 3; ++a) {
        const int x = x0 + 32 * a + lane;
        if (ns > 96) y[a] = g < gh && x < ns ? ml[slot(x) * PD_HEADS] : make_float2(-INFINITY, 0.f);
        const float f = M == -INFINITY ? 0.f : exp2f(y[a].x - M);
        if (x < ns) w_s[x][g] = f;
        L = fmaf(f, y[a].y, L);
      }
    L = warp_sum(L);
    if (lane == 0) {
      M_s[g] = M;
      L_s[g] = L;
      if (g < gh && p.lse != nullptr) p.lse[bh0 + g] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * LN2;
    }
  }
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (mine)
    for (int x0 = xg; x0 < ns; x0 += AHEAD * XG) {
      if (x0 != xg)
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
          if (x0 + a * XG < ns) buf[a] = part[slot(x0 + a * XG) * (PD_HEADS * D / 4)];
#pragma unroll
      for (int a = 0; a < AHEAD; ++a)
        if (x0 + a * XG < ns) {
          const float f = w_s[x0 + a * XG][vg];
          acc.x = fmaf(f, buf[a].x, acc.x), acc.y = fmaf(f, buf[a].y, acc.y);
          acc.z = fmaf(f, buf[a].z, acc.z), acc.w = fmaf(f, buf[a].w, acc.w);
        }
    }
  if constexpr (XG > 1) {
    if (xg == 1) acc_s[v] = acc;
    __syncthreads();
    if (xg == 1) return;
    const float4 y = acc_s[v];
    acc.x += y.x, acc.y += y.y, acc.z += y.z, acc.w += y.w;
  }
  if (mine) {
    const float r = M_s[vg] == -INFINITY ? 0.f : 1.f / L_s[vg];
    T *to = (T *)p.out + (bh0 + vg) * D + (v % (D / 4)) * 4;
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4 *>(to) = make_float4(acc.x * r, acc.y * r, acc.z * r, acc.w * r);
    } else {
      const __nv_bfloat162 x = __floats2bfloat162_rn(acc.x * r, acc.y * r), y = __floats2bfloat162_rn(acc.z * r, acc.w * r);
      *reinterpret_cast<uint2 *>(to) =
          make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
    }
  }
}

template <typename T, int D>
cudaError_t combine(const PagedDecodeArgs &a, int ctas, cudaStream_t st) {
  return launch_overlapped(paged_combine_kernel<T, D>, dim3(a.Hkv * a.HB, a.B), NT, 0, st, a, ctas);
}

template <int D>
cudaError_t launch_fp32(const PagedDecodeArgs &a, const TurnFreq &turn, cudaStream_t st) {
  const int gp = a.GS > PD_HEADS ? PD_HEADS : a.GS;
  const int ctas = 148 * ctas_per_sm(D);
  const auto kernel = gp == 1   ? paged_decode_kernel<D, 1>
                      : gp == 2 ? paged_decode_kernel<D, 2>
                      : gp <= 4 ? paged_decode_kernel<D, 4>
                                : paged_decode_kernel<D, 8>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ring_bytes(D));
  if (e == cudaSuccess) e = launch_overlapped(kernel, ctas, NT, ring_bytes(D), st, a, turn);
  return e != cudaSuccess ? e : combine<float, D>(a, ctas, st);
}

template <int D>
cudaError_t launch_bf16(const PagedDecodeArgs &a, const TurnFreq &turn, cudaStream_t st) {
  const cudaError_t e = launch_paged_decode_tc(D, a, turn, st);
  return e != cudaSuccess ? e : combine<__nv_bfloat16, D>(a, paged_decode_tc_ctas(), st);
}

}  // namespace pgd

cudaError_t launch_paged_decode(bool bf16, int D, const PagedDecodeArgs &a, const TurnFreq &turn, cudaStream_t st) {
  if (D == 128) return bf16 ? pgd::launch_bf16<128>(a, turn, st) : pgd::launch_fp32<128>(a, turn, st);
  return bf16 ? pgd::launch_bf16<64>(a, turn, st) : pgd::launch_fp32<64>(a, turn, st);
}

}  // namespace jl
