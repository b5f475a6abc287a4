"""The paged-cache operators on the GPU against plain 64-bit forms."""
import time

import numpy as np
import pytest
import torch

import oracle
from tests import paged_util as P
from tests.gpu_util import jl, to_np

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda:0"


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


def run_decode(q, kp, vp, table, lens, w_pre, w0, theta, **kw):
    J = jl()
    B, Hq, D = q.shape
    lse = torch.full((B, Hq), float("nan"), device=DEV)
    ws = torch.full((J.jl_bifocal_decode_paged_workspace_size(B, D),), 0xA5, dtype=torch.uint8, device=DEV)
    out, lse = J.jl_bifocal_decode_paged(q.to(DEV), kp, vp, i32(table), i32(lens), w_pre, w0, theta, lse=lse,
                                         workspace=ws, **kw)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32)) == 0
    return out, lse


def on_gpu(kp, vp, interleaved):
    if not interleaved:
        return kp.to(DEV), vp.to(DEV)
    pool = torch.stack((kp, vp), 1).to(DEV)
    return pool[:, 0], pool[:, 1]


# ------------------------------------------------------------------ decode
DECODE = [
    # lens, page, Hq, Hkv, D, dtype, w_pre, w0, window
    ((1,), 16, 4, 1, 128, BF, 1, 0, 0),
    ((1,), 64, 2, 2, 64, F32, 1, 0, 0),
    ((0, 5, 0, 16, 17), 16, 8, 2, 128, BF, 4, 3, 0),
    ((100,), 64, 8, 2, 128, BF, 40, 16, 0),
    ((1000,), 32, 32, 8, 128, BF, 250, 64, 0),
    ((1001, 64, 65, 63), 64, 32, 8, 128, BF, 250, 64, 0),
    ((3333, 17, 2048, 0, 1), 16, 16, 8, 128, BF, 700, 300, 0),
    ((5000,), 128, 8, 8, 128, BF, 900, 0, 0),
    ((5000,), 256, 8, 8, 64, BF, 900, 4999, 0),
    ((600,), 64, 8, 1, 128, BF, 100, 600, 0),
    ((700, 1300), 64, 6, 2, 64, BF, 150, 50, 0),      # three query heads per kv head
    ((700, 1300), 32, 24, 2, 128, BF, 150, 50, 0),    # twelve: two blocks of heads
    ((300,), 16, 17, 1, 64, F32, 50, 10, 0),          # seventeen: three blocks, the last of one
    ((2500, 33), 64, 16, 2, 128, F32, 512, 100, 0),
    ((900, 33), 16, 4, 4, 64, F32, 200, 10, 0),
    ((4000, 70, 1), 64, 8, 2, 128, BF, 500, 64, 129),  # sliding windows that start inside blocks and tiles
    ((4000, 70, 1), 16, 8, 2, 64, F32, 500, 64, 1),
    ((4000, 4095), 32, 8, 2, 128, BF, 300, 100, 1000),
    (tuple(range(1, 300, 2)), 16, 2, 1, 64, BF, 64, 16, 0),  # more sequences than SMs
    (tuple(range(0, 600, 2)), 16, 1, 1, 64, F32, 64, 16, 0),
]


@pytest.mark.parametrize("lens,page,Hq,Hkv,D,dtype,w_pre,w0,window", DECODE)
def test_decode_matches_64_bits(lens, page, Hq, Hkv, D, dtype, w_pre, w0, window):
    # garbage (1e4, and NaN) fills every slot behind a length and every page of nobody
    g = torch.Generator().manual_seed(len(lens) * 31 + page)
    q = torch.randn(len(lens), Hq, D, generator=g).to(dtype)
    for fill, inter in ((1e4, False), (float("nan"), True)):
        kp, vp, table, keys, vals = P.make_cache(lens, page, Hkv, D, dtype, 7 + D, fill=fill)
        kd, vd = on_gpu(kp, vp, inter)
        out, lse = run_decode(q, kd, vd, table, lens, w_pre, w0, 1e4, window=window)
        ro, rl, to, tl = P.decode(q, keys, vals, w_pre, w0, 1e4, window=window)
        P.check(out, ro, to, "out")
        P.check(lse, rl, tl, "lse")
    J = jl()
    out, lse = run_decode(q, kd, vd, table, lens, w_pre, w0, 1e4, window=window, flags=J.JL_FLAG_PLAIN_CAUSAL)
    ro, rl, to, tl = P.decode(q, keys, vals, w_pre, w0, 1e4, window=window, plain=True)
    P.check(out, ro, to, "plain out")
    P.check(lse, rl, tl, "plain lse")


@pytest.mark.parametrize("page,D,dtype,Hq", [(16, 128, BF, 8), (32, 64, BF, 2), (64, 128, BF, 8), (128, 64, BF, 16),
                                             (256, 128, BF, 4), (16, 64, F32, 8), (256, 128, F32, 2)])
def test_decode_of_listed_pages(page, D, dtype, Hq):
    # lists out of order, with -1 between, pages past the length, one page
    # twice (it counts twice), another list for each kv head, an empty one
    lens, Hkv, n = (20 * page + 5, 3 * page, 1), 2, 9
    g = torch.Generator().manual_seed(page + D)
    q = torch.randn(3, Hq, D, generator=g).to(dtype)
    kp, vp, table, keys, vals = P.make_cache(lens, page, Hkv, D, dtype, 11, fill=float("nan"))
    lists = torch.full((3, Hkv, n), -1, dtype=torch.int32)
    lists[0, 0] = torch.tensor([20, 3, -1, 0, 7, 7, 12, 40, 19])
    lists[0, 1] = torch.tensor([5, -1, -1, -1, -1, -1, -1, -1, 6])
    lists[1, 0, :4] = torch.tensor([0, 1, 2, 3])
    lists[2, 1, 4] = 0
    want = [[[c for c in lists[b, h].tolist() if c >= 0] for h in range(Hkv)] for b in range(3)]
    for window in (0, 2 * page + 3):
        ro, rl, to, tl = P.decode(q, keys, vals, 4 * page, page + 1, 1e4, lists=want, page=page, window=window)
        out, lse = run_decode(q, kp.to(DEV), vp.to(DEV), table, lens, 4 * page, page + 1, 1e4, page_list=i32(lists),
                              window=window)
        P.check(out, ro, to, f"out window {window}")
        P.check(lse, rl, tl, f"lse window {window}")


def test_decode_with_an_empty_list_writes_zeros():
    q = torch.randn(2, 4, 64).to(BF)
    kp, vp, table, _, _ = P.make_cache((50, 20), 16, 2, 64, BF, 3)
    out, lse = run_decode(q, kp.to(DEV), vp.to(DEV), table, (50, 20), 16, 4, 1e4,
                          page_list=torch.empty(2, 2, 0, dtype=torch.int32, device=DEV))
    assert torch.all(out == 0) and torch.all(lse == -float("inf"))


@pytest.mark.parametrize("dtype,D", [(BF, 128), (BF, 64), (F32, 128)])
def test_decode_skips_pages_that_are_not_there(dtype, D):
    lens, page = (500, 200), 32
    q = torch.randn(2, 8, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    kp, vp, table, keys, vals = P.make_cache(lens, page, 2, D, dtype, 5, fill=float("nan"))
    table[0, 3], table[0, 15], table[1, 0] = -1, kp.shape[0], 2 ** 31 - 1
    ro, rl, to, tl = P.decode(q, keys, vals, 100, 40, 1e4, page=page, missing=[[3, 15], [0]])
    out, lse = run_decode(q, kp.to(DEV), vp.to(DEV), table, lens, 100, 40, 1e4)
    P.check(out, ro, to, "out")
    P.check(lse, rl, tl, "lse")


def test_decode_length_past_the_table_writes_zeros():
    q = torch.randn(2, 4, 128).to(BF)
    kp, vp, table, keys, vals = P.make_cache((50, 64), 16, 2, 128, BF, 9)
    out, lse = run_decode(q, kp.to(DEV), vp.to(DEV), table, (65, -3), 16, 4, 1e4)
    assert torch.all(out == 0) and torch.all(lse == -float("inf"))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_shows_a_nan_key_and_no_other(dtype):
    # a NaN in a key or value that is read reaches its own heads' outputs only
    lens, page = (300, 300), 16
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(2)).to(dtype)
    kp, vp, table, keys, vals = P.make_cache(lens, page, 2, 64, dtype, 6)
    kp[table[0, 2], 5, 1, 3] = float("nan")
    out, lse = run_decode(q, kp.to(DEV), vp.to(DEV), table, lens, 100, 40, 1e4)
    assert torch.isnan(out[0, 2:]).all() and torch.isnan(lse[0, 2:]).all()
    ro, rl, to, tl = P.decode(q, keys, vals, 100, 40, 1e4)
    P.check(out[1], ro[1], to[1], "other sequence")
    P.check(out[0, :2], ro[0, :2], to[0, :2], "other kv head")


INF = float("inf")


def _turn(j, L, w_pre, w0):
    G = P.group(L, w_pre)
    return (j // G - j) - ((L - 1) // G - (L - 1)) if j < L - w0 else 0


@pytest.mark.parametrize("dtype,D,page", [(BF, 128, 16), (BF, 128, 64), (BF, 64, 32), (F32, 64, 16)])
@pytest.mark.parametrize("j", [7, 1000, 1180, 1299])  # turned, turned, in the block with keys of both kinds, local
def test_decode_of_an_infinite_key(dtype, D, page, j):
    # one channel of a key of kv head 1 is infinite.  Queries with the sign that
    # makes its score -inf drop the key; one with the other sign has a score of
    # +inf, so its softmax is NaN, as in 64 bits
    L, w_pre, w0, theta, d = 1300, 300, 117, 1e4, 5
    assert page >= 16 and 1180 // 16 == (L - w0) // 16 and 1180 < L - w0
    q = torch.randn(2, 8, D, generator=torch.Generator().manual_seed(j)).to(dtype)
    kp, vp, table, keys, vals = P.make_cache((L, 400), page, 2, D, dtype, 6)
    kp[table[0, j // page], j % page, 1, d] = INF
    far = [k.clone() for k in keys]
    far[0][j, 1, d] = 1e30  # for the 64-bit form: a score so low that the weight is zero there too
    tame = [k.clone() for k in keys]
    tame[0][j, 1, d] = 0.0  # for the tolerances, which are those of the other keys
    turned = P.rotate(P.f64(far[0][j, 1]), _turn(j, L, w_pre, w0), theta)
    for x in np.flatnonzero(np.abs(turned) > 1e20):  # the channel, and its partner if the key is turned
        q[0, 4:, x] = q[0, 4:, x].abs() * -float(np.sign(turned[x]))
    for plus in (False, True):
        ro, rl, _, _ = P.decode(q, far, vals, w_pre, w0, theta)
        _, _, to, tl = P.decode(q, tame, vals, w_pre, w0, theta)
        if plus:
            q[0, 6] = -q[0, 6]
        out, lse = run_decode(q, kp.to(DEV), vp.to(DEV), table, (L, 400), w_pre, w0, theta)
        if plus:
            assert torch.isnan(out[0, 6]).all() and torch.isnan(lse[0, 6])
        keep = [0, 1, 2, 3, 4, 5, 7] + ([] if plus else [6])
        P.check(out[0, keep], ro[0, keep], to[0, keep], "out")
        P.check(lse[0, keep], rl[0, keep], tl[0, keep], "lse")
        P.check(out[1], ro[1], to[1], "the other sequence")


@pytest.mark.parametrize("dtype,D,page", [(BF, 128, 16), (BF, 128, 64), (BF, 64, 32), (F32, 64, 16)])
def test_decode_of_infinite_and_nan_values(dtype, D, page):
    # an infinite value makes its channel infinite for its own heads, two of
    # opposite signs or a NaN make it NaN; a key's weight may have any bits: all
    # keys are tried in turn, one channel each, turned and local ones
    L, w_pre, w0, theta = 900, 200, 333, 1e4
    q = torch.randn(1, 8, D, generator=torch.Generator().manual_seed(D)).to(dtype)
    kp, vp, table, keys, vals = P.make_cache((L,), page, 2, D, dtype, 16)
    tol = P.decode(q, keys, vals, w_pre, w0, theta)[2]
    kd = kp.to(DEV)
    for first in range(0, L, 3 * D // 4):
        v2, want = vp.clone(), vals[0].clone()
        for x in range(min(3 * D // 4, L - first)):
            j, what = first + x, (INF, -INF, float("nan"))[x % 3]
            want[j, x % 2, x] = what
            v2[table[0, j // page], j % page, x % 2, x] = what
        want[(first + 200) % L, 0, 0] = -INF  # beside the +inf of channel 0
        v2[table[0, (first + 200) % L // page], (first + 200) % L % page, 0, 0] = -INF
        with np.errstate(invalid="ignore"):
            ro = P.decode(q, keys, [want], w_pre, w0, theta)[0]
        out, lse = run_decode(q, kd, v2.to(DEV), table, (L,), w_pre, w0, theta)
        got = to_np(out)
        assert np.array_equal(np.isnan(got), np.isnan(ro)), first
        assert np.isnan(ro[0, :4, 0]).all() and (np.abs(ro[0]) == INF).any()
        there = ~np.isnan(ro)
        P.check(np.where(there, got, 0.0), np.where(there, ro, 0.0), tol, f"from key {first}")
        assert torch.isfinite(lse).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_of_infinite_values_under_small_weights(dtype):
    # scores 60 to 86 below the others', weights down to 2^-124
    D, L = 64, 64
    low = torch.linspace(-7.5, -10.75, 27)
    q = torch.zeros(1, 1, D)
    q[..., 0] = 64.0  # score = 8 k_0
    kp, vp, table, keys, vals = P.make_cache((L,), 16, 1, D, dtype, 23)
    k = torch.zeros(L, 1, D)
    k[2:2 + len(low), 0, 0] = low
    v = vals[0].clone()
    for x in range(len(low)):
        v[2 + x, 0, 2 * x], v[2 + x, 0, 2 * x + 1] = INF, -INF
    for c in range(L // 16):
        kp[table[0, c]], vp[table[0, c]] = k[c * 16:c * 16 + 16].to(dtype), v[c * 16:c * 16 + 16]
    out, lse = run_decode(q.to(dtype), kp.to(DEV), vp.to(DEV), table, (L,), 10 ** 6, 8, 1e4)
    assert out[0, 0, :2 * len(low):2].tolist() == [INF] * len(low)
    assert out[0, 0, 1:2 * len(low):2].tolist() == [-INF] * len(low)
    assert torch.isfinite(out[0, 0, 2 * len(low):]).all() and torch.isfinite(lse).all()


def test_decode_large_scores_and_one_hot():
    # a single key dominates by far (scores beyond exp's range apart)
    lens, page = (2000,), 64
    g = torch.Generator().manual_seed(4)
    q = (30 * torch.randn(1, 8, 128, generator=g)).to(BF)
    kp, vp, table, keys, vals = P.make_cache(lens, page, 2, 128, BF, 8)
    ro, rl, to, tl = P.decode(q, keys, vals, 10 ** 6, 64, 1e4)
    out, lse = run_decode(q, kp.to(DEV), vp.to(DEV), table, lens, 10 ** 6, 64, 1e4)
    P.check(out, ro, to, "out")
    P.check(lse, rl, tl, "lse")


def test_decode_128k_matches_the_contiguous_decode():
    # the long-context workload: G = 4 and 5, every output, and the contiguous
    # cache's kernel beside it
    J = jl()
    g = torch.Generator(device=DEV).manual_seed(1)
    page, Hkv, D = 64, 8, 128
    for L in (131072, 131073):
        n = -(-L // page)
        kp = torch.randn(n, page, Hkv, D, generator=g, device=DEV).to(BF)
        vp = torch.randn(n, page, Hkv, D, generator=g, device=DEV).to(BF)
        q = torch.randn(1, 32, D, generator=g, device=DEV).to(BF)
        table = torch.randperm(n, generator=g, device=DEV).to(torch.int32)[None]
        out, lse = run_decode(q, kp, vp, table, (L,), 32768, 4096, 1e6)
        order = table[0].long()
        kc, vc = kp[order].view(1, n * page, Hkv, D), vp[order].view(1, n * page, Hkv, D)
        oc, lc = J.jl_bifocal_decode(q, kc, vc, i32([L]), n * page, 32768, 4096, 1e6,
                                     lse=torch.empty(1, 32, device=DEV))
        ro, rl, to, tl = P.decode(q, [kc[0, :L].cpu()], [vc[0, :L].cpu()], 32768, 4096, 1e6)
        P.check(out, ro, to, "out")
        P.check(lse, rl, tl, "lse")
        assert np.abs(to_np(oc) - to_np(out)).max() <= 2e-2 and np.abs(to_np(lc) - to_np(lse)).max() <= 2e-2


def test_decode_repeats_bit_for_bit():
    lens, page = (5000, 300, 9000), 32
    q = torch.randn(3, 16, 128, generator=torch.Generator().manual_seed(3)).to(BF)
    kp, vp, table, _, _ = P.make_cache(lens, page, 4, 128, BF, 12)
    kd, vd = kp.to(DEV), vp.to(DEV)
    a = run_decode(q, kd, vd, table, lens, 1000, 100, 1e4)
    for _ in range(3):
        b = run_decode(q, kd, vd, table, lens, 1000, 100, 1e4)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------ append
APPEND = [
    # lengths after, new tokens, page, Hq, Hkv, D, dtype
    ((1,), (1,), 16, 4, 1, 128, BF),
    ((64, 65, 128), (1, 1, 64), 64, 8, 2, 128, BF),
    ((300, 40, 7, 1000), (300, 3, 0, 129), 32, 8, 2, 64, BF),
    ((1000, 513), (700, 500), 256, 4, 4, 128, F32),
    ((33, 100, 17), (33, 1, 2), 16, 6, 2, 64, F32),
    ((131072,), (100,), 64, 32, 8, 128, BF),
    # enough pages for all heads of one to share a CTA: 256 threads, then 128
    ((5003,), (5000,), 16, 16, 8, 128, BF),
    ((5003,), (4999,), 16, 20, 10, 64, F32),
    ((3001, 2500), (3001, 2400), 16, 2, 2, 64, BF),
]


@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("lens,new,page,Hq,Hkv,D,dtype", APPEND)
def test_append_matches_64_bits(lens, new, page, Hq, Hkv, D, dtype, rotate):
    J = jl()
    theta = 1e4
    g = torch.Generator().manual_seed(sum(lens))
    T = sum(new)
    q, k, v = (torch.randn(T, h, D, generator=g).to(dtype) for h in (Hq, Hkv, Hkv))
    kp, vp, table, _, _ = P.make_cache(lens, page, Hkv, D, dtype, 21, fill=3.0)
    kp0, vp0 = kp.clone(), vp.clone()
    sm0 = torch.randn(kp.shape[0], Hkv, 2, D, generator=g).to(dtype)
    cu = np.concatenate([[0], np.cumsum(new)])
    kd, vd = on_gpu(kp, vp, page == 32)
    sm = sm0.to(DEV)
    qo = J.jl_paged_append(k.to(DEV), v.to(DEV), kd, vd, i32(table), i32(cu), i32(lens), max(new), page_summary=sm,
                           q=q.to(DEV) if rotate else None, rope_theta=theta if rotate else None)
    torch.cuda.synchronize()
    kg, vg, smg = kd.cpu(), vd.cpu(), sm.cpu()
    wk, wv = P.f64(kp0), P.f64(vp0)
    tol = np.zeros(wk.shape)
    half = 2.0 ** -8 if dtype == BF else P.U
    written = set()
    wsm = sm0.clone().float()
    for b, (L, n) in enumerate(zip(lens, new)):
        pos = np.arange(L - n, L)
        rows = slice(cu[b], cu[b + 1])
        kk, qq = P.f64(k[rows]), P.f64(q[rows])
        kr = P.rotate(kk, pos[:, None], theta) if rotate else kk
        if rotate:
            # half a step of the type, and the angle's cosine and sine, a product and a sum in fp32
            P.check(qo[rows].cpu(), P.rotate(qq, pos[:, None], theta),
                    half * np.abs(P.rotate(qq, pos[:, None], theta)) + 6 * P.U * P.pair_len(qq), "q")
        for x, p in enumerate(pos):
            one = int(table[b, p // page])
            wk[one, p % page], wv[one, p % page] = kr[x], P.f64(v[rows])[x]
            tol[one, p % page] = (half * np.abs(kr[x]) + 6 * P.U * P.pair_len(kk[x])) if rotate else 0.0
            written.add((b, p // page))
        for c in {p // page for p in pos}:
            one, a = int(table[b, c]), max(0, (L - n) - c * page)
            mine = kg[one, a:min(page, L - c * page)].float()
            lo, hi = mine.amin(0), mine.amax(0)
            if a > 0:
                lo, hi = torch.minimum(lo, wsm[one, :, 0]), torch.maximum(hi, wsm[one, :, 1])
            wsm[one, :, 0], wsm[one, :, 1] = lo, hi
    P.check(kg, wk, tol, "k pages")
    P.check(vg, wv, np.zeros(wv.shape), "v pages")
    assert torch.equal(smg.float(), wsm)  # of the values as stored; untouched pages as they were


def test_append_in_place_query_and_no_summary():
    J = jl()
    q, k, v = (torch.randn(5, h, 64, generator=torch.Generator().manual_seed(h)).to(DEV) for h in (4, 2, 2))
    kp, vp = torch.zeros(4, 16, 2, 64, device=DEV), torch.zeros(4, 16, 2, 64, device=DEV)
    args = (k, v, kp, vp, i32([[3, 1]]), i32([0, 5]), i32([18]), 5)
    want = J.jl_paged_append(*args, q=q, rope_theta=1e4)
    got = J.jl_paged_append(*args, q=q, q_out=q, rope_theta=1e4)
    assert got is q and torch.equal(want, q)
    assert torch.equal(vp[3, 13:], v[:3]) and torch.equal(vp[1, :2], v[3:]) and torch.all(vp[3, :13] == 0)


def test_append_leaves_misfits_alone():
    # more new tokens than the length, than max_new, rows past the end,
    # decreasing prefix sums; a page that is not there
    J = jl()
    T = 10
    k = torch.randn(T, 1, 64, device=DEV)
    table = i32([[0], [1], [2], [3], [-1]])
    for cu, lens, ok in (([0, 2, 4, 6, 8, 10], [1, 2, 0, 5, 5], (1, 3)), ([0, 4, 6, 6, 8, 10], [9, 9, 9, 9, 9], (1, 3)),
                         ([0, 2, 1, 3, 12, 13], [9, 9, 9, 9, 9], (0, 2))):
        kp = torch.zeros(4, 16, 1, 64, device=DEV)
        vp, sm = torch.zeros_like(kp), torch.zeros(4, 1, 2, 64, device=DEV)
        q = torch.ones(T, 1, 64, device=DEV)
        qo = torch.full_like(q, 7.0)
        J.jl_paged_append(k, k, kp, vp, table, i32(cu), i32(lens), 2, page_summary=sm, q=q, q_out=qo, rope_theta=1e4)
        torch.cuda.synchronize()
        for b in range(4):
            assert bool((vp[b] != 0).any()) == (b in ok), (cu, b)
            assert bool((sm[b] != 0).any()) == (b in ok), (cu, b)
        rows = [cu[b + 1] - cu[b] for b in range(5)]
        for b in range(5):
            fits = b in ok or (b == 4 and cu[b + 1] <= T)
            if rows[b] > 0 and fits:
                assert (qo[cu[b]:cu[b + 1]] != 7.0).all()


def test_append_keeps_a_nan_in_the_summary():
    J = jl()
    for dtype in (BF, F32):
        k = torch.randn(20, 2, 64).to(dtype)
        k[9, 1, 5] = float("nan")
        kp = torch.zeros(2, 16, 2, 64, dtype=dtype, device=DEV)
        sm = torch.zeros(2, 2, 2, 64, dtype=dtype, device=DEV)
        J.jl_paged_append(k.to(DEV), k.to(DEV), kp, torch.zeros_like(kp), i32([[1, 0]]), i32([0, 20]), i32([20]), 20,
                          page_summary=sm)
        nan = torch.isnan(sm.cpu())
        assert nan[1, 1, :, 5].all() and nan.sum() == 2


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_at_the_last_positions(dtype):
    # lengths up to 2^31 - 1: no table reaches there, so nothing is written but
    # the rotated queries; the first row of a page, whole pages and a part of one
    J = jl()
    lens, new, D, theta = (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 65), (1, 127, 300, 70), 64, 1e4
    T = sum(new)
    g = torch.Generator().manual_seed(31)
    q, k = torch.randn(T, 4, D, generator=g).to(dtype), torch.randn(T, 2, D, generator=g).to(dtype)
    half = 2.0 ** -8 if dtype == BF else P.U
    for page in (16, 256):
        kp = torch.full((3, page, 2, D), 3.0, dtype=dtype, device=DEV)
        vp, sm = kp.clone(), torch.full((3, 2, 2, D), 3.0, dtype=dtype, device=DEV)
        cu = np.concatenate([[0], np.cumsum(new)])
        qo = J.jl_paged_append(k.to(DEV), k.to(DEV), kp, vp, i32([[0, 1, 2]] * 4), i32(cu), i32(lens), max(new),
                               page_summary=sm, q=q.to(DEV), rope_theta=theta)
        torch.cuda.synchronize()
        assert all(bool((x == 3.0).all()) for x in (kp, vp, sm))
        for b, (L, n) in enumerate(zip(lens, new)):
            rows = slice(cu[b], cu[b + 1])
            want = P.rotate(P.f64(q[rows]), np.arange(L - n, L)[:, None], theta)
            # cosine, sine, a product and a sum in fp32; the angle's frequency and product in 64 bits, on either side
            tol = half * np.abs(want) + (6 * P.U + 6 * 2.0 ** 31 * 2.0 ** -53) * P.pair_len(P.f64(q[rows]))
            P.check(qo[rows].cpu(), want, tol, f"sequence {b}")


# ------------------------------------------------------------------ select
SELECT = [
    # lens, page, Hq, Hkv, D, dtype, w_pre, w0, n_select, n_first, n_last
    ((1, 16, 17, 0), 16, 2, 1, 64, F32, 4, 2, 1, 0, 0),
    ((1000, 333, 90), 16, 8, 2, 128, BF, 200, 64, 7, 1, 1),
    ((5000,), 16, 32, 8, 128, BF, 700, 100, 24, 2, 3),
    ((5000, 4000, 77), 64, 6, 2, 64, BF, 700, 100, 5, 0, 5),
    ((9000, 2000), 32, 17, 1, 128, F32, 9999, 100, 11, 0, 0),
    ((20000,), 16, 4, 4, 64, F32, 3000, 0, 600, 10, 20),
    ((8191,), 256, 8, 1, 128, BF, 512, 9000, 3, 0, 1),
    ((150001, 40000), 16, 4, 2, 64, BF, 30000, 1000, 40, 1, 1),  # more pages than a CTA keeps in registers
    ((33000, 2000), 16, 2, 1, 64, F32, 5000, 100, 2050, 1, 1),   # a list longer than a short sequence's pages
]


@pytest.mark.parametrize("lens,page,Hq,Hkv,D,dtype,w_pre,w0,n,first,last", SELECT)
def test_select_matches_64_bits(lens, page, Hq, Hkv, D, dtype, w_pre, w0, n, first, last):
    J = jl()
    g = torch.Generator().manual_seed(n)
    q = torch.randn(len(lens), Hq, D, generator=g).to(dtype)
    _, _, table, _, _ = P.make_cache(lens, page, 1, 1, F32, 2, spare=3)
    n_pages = int(table.max()) + 4
    base = torch.randn(n_pages, Hkv, 1, D, generator=g)
    sm = torch.cat((base - 0.4, base + 0.4), 2).to(dtype)
    for flags in (0, J.JL_FLAG_PLAIN_CAUSAL):
        got = J.jl_bifocal_select_pages(q.to(DEV), sm.to(DEV), i32(table), i32(lens), page, n, w_pre, w0, 1e4,
                                        n_first=first, n_last=last, flags=flags)
        want = P.select(q, sm, table, lens, page, n, first, last, w_pre, w0, 1e4, plain=bool(flags))
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["zero", "equal", "few", "close", "nan", "inf", "huge"])
def test_select_of_scores_that_fp32_cannot_tell_apart(kind, dtype):
    # G = 1, so that equal summaries score equal: the lower page wins
    J = jl()
    page, Hkv, D, n, L = 16, 2, 64, 10, 16 * 700 - 3
    g = torch.Generator().manual_seed(5)
    pages = 700
    table = torch.randperm(pages, generator=g).to(torch.int32)[None]
    q = torch.randn(1, 4, D, generator=g).to(dtype)
    sm = torch.zeros(pages, Hkv, 2, D)
    if kind == "equal":
        sm += torch.randn(1, Hkv, 1, D, generator=g)
    elif kind == "few":  # five different pages, each many times
        sm = torch.randn(5, Hkv, 1, D, generator=g).expand(5, Hkv, 2, D)[torch.randint(5, (pages,), generator=g)]
    elif kind == "close":  # one channel, by less than the sum of the others can show in fp32
        sm = 100 * torch.randn(1, Hkv, 1, D, generator=g).expand(pages, Hkv, 2, D).clone()
        sm[:, :, :, 7] = 1e-5 * torch.rand(pages, Hkv, 1, generator=g)
    elif kind in ("nan", "inf", "huge"):
        sm = torch.randn(pages, Hkv, 1, D, generator=g).expand(pages, Hkv, 2, D).clone()
        sm[table[0, 30].item(), 0, 0, 3] = {"nan": float("nan"), "inf": -float("inf"), "huge": -3e38}[kind]
        sm[table[0, 31].item(), 0, 1, 3] = {"nan": float("nan"), "inf": float("inf"), "huge": 3e38}[kind]
        sm[table[0, 35].item(), 1, 1, 3] = {"nan": float("nan"), "inf": float("inf"), "huge": 3.1e38}[kind]
    sm = sm.to(dtype).contiguous()
    got = J.jl_bifocal_select_pages(q.to(DEV), sm.to(DEV), i32(table), i32([L]), page, n, 10 ** 6, 64, 1e4)
    want = P.select(q, sm, table, [L], page, n, 1, 1, 10 ** 6, 64, 1e4)
    assert np.array_equal(got.cpu().numpy(), want)
    if kind in ("zero", "equal"):
        assert want[0, 0].tolist() == list(range(n - 1)) + [699]


def test_select_fills_the_longest_list():
    # 2^31 - 1 entries, of which a short sequence has five
    J = jl()
    n = 2 ** 31 - 1
    q, sm = torch.ones(1, 1, 64, device=DEV), torch.zeros(5, 1, 2, 64, device=DEV)
    out = torch.full((1, 1, n), 77, dtype=torch.int32, device=DEV)
    J.jl_bifocal_select_pages(q, sm, i32([[0, 1, 2, 3, 4]]), i32([70]), 16, n, 100, 10, 1e4, out=out)
    assert out[0, 0, :5].tolist() == [0, 1, 2, 3, 4]
    for a in range(5, n, 1 << 28):
        assert bool((out[0, 0, a:a + (1 << 28)] == -1).all()), a


@pytest.mark.parametrize("dtype", [BF, F32])
def test_select_with_a_base_below_one(dtype):
    # frequencies 1, 2, 4 .. 2^31 (exact in 64 bits, and so are their angles), of
    # which the queries use the highest: angles up to 2^44, whose fractions of a
    # turn decide the scores
    J = jl()
    page, Hkv, D, L, n = 16, 32, 64, 8192, 256
    g = torch.Generator().manual_seed(12)
    q = torch.zeros(2, Hkv, D)
    q[..., [31, 63]] = torch.randn(2, Hkv, 2, generator=g)
    q = q.to(dtype)
    table = torch.randperm(L // page, generator=g).to(torch.int32)[None].repeat(2, 1)
    base = torch.randn(L // page, Hkv, 1, D, generator=g)
    sm = torch.cat((base - 0.1, base + 0.1), 2).to(dtype)
    lens = (L, L - 777)
    got = J.jl_bifocal_select_pages(q.to(DEV), sm.to(DEV), i32(table), i32(lens), page, n, 64, 16, 2.0 ** -32)
    want = P.select(q, sm, table, lens, page, n, 1, 1, 64, 16, 2.0 ** -32)
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("n_near", [2, 3, 17, 64, 65, 130])
@pytest.mark.parametrize("kind,dtype,Hq,D", [("local", BF, 2, 64), ("local", F32, 8, 128), ("slow", BF, 8, 128),
                                             ("slow", F32, 2, 64), ("turned", F32, 8, 128), ("turned", F32, 2, 64)])
def test_select_among_a_few_near_ties(kind, dtype, Hq, D, n_near):
    # n_near pages whose scores differ by less than fp32 can show, in an order
    # that is not that of the pages, half of them chosen; all others far above or
    # below.  "local": no turn, differences in one channel, some exactly equal;
    # "slow": turned, by frequencies that hardly matter; "turned": each page's
    # keys turned so that the query meets the same ones, and rounded
    J = jl()
    page, Hkv, pages, n_high = 16, 2, 300, 9
    L, w0, half = page * pages - 5, 40, D // 2
    w_pre = 10 ** 6 if kind == "local" else 1000
    theta = 1e12 if kind == "slow" else 1e4
    g = torch.Generator().manual_seed(n_near + D)
    q = torch.randn(1, Hq, D, generator=g).to(dtype)
    first = q[0, ::Hq // Hkv].double()  # the query head that all keys favour
    base = 100 * (1 + torch.rand(Hkv, D, generator=g).double()) * first.sign()
    if kind == "slow":
        base[:, :half - 4], base[:, half:D - 4] = 0.0, 0.0
    order = torch.randperm(pages - 50, generator=g) + 10  # (the last pages are local: no near ties there)
    near, high = order[:n_near], order[n_near:n_near + n_high]
    size = torch.full((pages,), 0.3, dtype=torch.float64) - 0.2 * torch.rand(pages, generator=g).double()
    size[near], size[high] = 1.0, 1.5
    m = size[:, None, None] * base
    fine = torch.randint(0, max(2, n_near // 2), (pages, Hkv), generator=g)
    if kind == "turned":
        G = P.group(L, w_pre)
        mid = np.arange(pages) * page + page // 2
        turn = np.where(mid < L - w0, (mid - mid // G) - ((L - 1) - (L - 1) // G), 0)
        m = torch.from_numpy(P.rotate(m.numpy(), np.broadcast_to(turn[:, None], (pages, Hkv)), theta))
    else:
        m[near, :, D - 1] = 1e-5 * (1 + fine[near].double())
    sm = torch.zeros(pages, Hkv, 2, D, dtype=dtype)
    table = torch.randperm(pages, generator=g).to(torch.int32)[None]
    sm[table[0].long()] = m[:, :, None].to(dtype).expand(-1, -1, 2, -1)
    n = 2 + n_high + (n_near + 1) // 2
    want = P.select(q, sm, table, [L], page, n, 1, 1, w_pre, w0, theta)
    for h in range(Hkv):  # the case is what it says
        assert set(high.tolist()) <= set(want[0, h]) <= set(high.tolist() + near.tolist() + [0, pages - 1])
    got = J.jl_bifocal_select_pages(q.to(DEV), sm.to(DEV), i32(table), i32([L]), page, n, w_pre, w0, theta)
    assert np.array_equal(got.cpu().numpy(), want)


def test_select_passes_over_pages_that_are_not_there():
    J = jl()
    g = torch.Generator().manual_seed(6)
    sm = torch.randn(40, 2, 2, 64, generator=g).sort(dim=2).values
    table = torch.arange(40, dtype=torch.int32)[None].clone()
    table[0, 5:30] = -1
    table[0, 30] = 40
    q = torch.randn(1, 4, 64, generator=g)
    for n in (6, 20):
        got = J.jl_bifocal_select_pages(q.to(DEV), sm.to(DEV), i32(table), i32([640]), 16, n, 100, 64, 1e4)
        assert np.array_equal(got.cpu().numpy(), P.select(q, sm, table, [640], 16, n, 1, 1, 100, 64, 1e4))


def test_select_scores_bound_the_keys():
    # what the score is for: with G = 1 no key of an unlisted page outscores
    # the bound of the weakest listed one; the best key's page is always found
    J = jl()
    lens, page, D = (4000,), 32, 128
    kp, vp, table, keys, _ = P.make_cache(lens, page, 1, D, BF, 14)
    q = torch.randn(1, 1, D, generator=torch.Generator().manual_seed(8)).to(BF)
    sm = torch.zeros(kp.shape[0], 1, 2, D, dtype=BF)
    for c in range(125):
        mine = keys[0][c * page:(c + 1) * page]
        sm[table[0, c]] = torch.stack((mine.amin(0), mine.amax(0)), 1)
    got = J.jl_bifocal_select_pages(q.to(DEV), sm.to(DEV), i32(table), i32(lens), page, 124, 10 ** 6, 64, 1e4, n_first=0,
                                    n_last=0)
    out = sorted(set(range(125)) - set(got[0, 0].tolist()))
    assert len(out) == 1
    s = P.f64(keys[0][:, 0]) @ P.f64(q[0, 0])
    assert s.argmax() // page not in out


# -------------------------------------------------------------- all of them
def test_generation_over_a_paged_cache():
    """Prompt through the prefill, its keys into pages, then steps of append,
    select and decode; against the oracle on the same (rotated) keys."""
    J = jl()
    g = torch.Generator().manual_seed(77)
    Hq, Hkv, D, page, w_pre, w0, theta = 8, 2, 128, 16, 100, 40, 1e4
    lens = [130, 61]
    T = sum(lens)
    raw = [torch.randn(T, h, D, generator=g).to(BF).to(DEV) for h in (Hq, Hkv, Hkv)]
    pool = torch.full((40, 2, page, Hkv, D), float("nan"), dtype=BF, device=DEV)
    kp, vp = pool[:, 0], pool[:, 1]
    sm = torch.zeros(40, Hkv, 2, D, dtype=BF, device=DEV)
    table = torch.randperm(40, generator=g).to(torch.int32)[:40].view(2, 20).to(DEV)
    cu = i32([0, 130, 191])
    q = J.jl_paged_append(raw[1], raw[2], kp, vp, table, cu, i32(lens), 130, page_summary=sm, q=raw[0], rope_theta=theta)

    def cached(b, n):
        at = table[b].long()
        return [x[at].reshape(-1, Hkv, D)[:n] for x in (kp, vp)]

    kv = [torch.cat([cached(b, lens[b])[x] for b in range(2)]) for x in range(2)]
    out, _ = J.jl_bifocal_prefill(q, kv[0], kv[1], cu, 130, w_pre, w0, theta)
    ro, _ = oracle.bifocal_attention(q.cpu(), kv[0].cpu(), kv[1].cpu(), cu.cpu(), w_pre, w0, theta)
    assert np.abs(to_np(out) - ro).max() <= 2e-2
    for step in range(20):
        lens = [n + 1 for n in lens]
        raw = [torch.randn(2, h, D, generator=g).to(BF).to(DEV) for h in (Hq, Hkv, Hkv)]
        q = J.jl_paged_append(raw[1], raw[2], kp, vp, table, i32([0, 1, 2]), i32(lens), 1, page_summary=sm, q=raw[0],
                              rope_theta=theta)
        keys, vals = zip(*[[x.cpu() for x in cached(b, lens[b])] for b in range(2)])
        listed = J.jl_bifocal_select_pages(q, sm, table, i32(lens), page, 4, w_pre, w0, theta)
        assert np.array_equal(listed.cpu().numpy(), P.select(q.cpu(), sm.cpu(), table.cpu(), lens, page, 4, 1, 1, w_pre,
                                                             w0, theta))
        full, _ = run_decode(q, kp, vp, table, lens, w_pre, w0, theta)
        some, _ = run_decode(q, kp, vp, table, lens, w_pre, w0, theta, page_list=listed)
        every = J.jl_bifocal_select_pages(q, sm, table, i32(lens), page, 20, w_pre, w0, theta)
        same, _ = run_decode(q, kp, vp, table, lens, w_pre, w0, theta, page_list=every)
        ro, _, to, _ = P.decode(q.cpu(), keys, vals, w_pre, w0, theta)
        P.check(full, ro, to, f"step {step}")
        P.check(same, ro, to, f"every page listed, step {step}")
        pages = [[[c for c in listed[b, h].tolist() if c >= 0] for h in range(Hkv)] for b in range(2)]
        ro, _, to, _ = P.decode(q.cpu(), keys, vals, w_pre, w0, theta, lists=pages, page=page)
        P.check(some, ro, to, f"listed, step {step}")
        for b in range(2):  # the summary is the range of the page's keys so far
            for c in range(-(-lens[b] // page)):
                mine = keys[b][c * page:(c + 1) * page]
                assert torch.equal(sm[table[b, c]].cpu(), torch.stack((mine.amin(0), mine.amax(0)), 1))


def test_step_replays_from_a_graph_on_another_stream():
    # append, select and decode captured together; lengths, tokens and table
    # change between replays
    J = jl()
    g = torch.Generator().manual_seed(5)
    B, Hq, Hkv, D, page, w_pre, w0, theta = 3, 8, 2, 128, 32, 500, 64, 1e4
    lens0 = (2000, 31, 700)
    kp, vp, table, keys, vals = P.make_cache([2064] * B, page, Hkv, D, BF, 4)
    kd, vd, td = kp.to(DEV), vp.to(DEV), table.to(DEV)
    sm = torch.stack((kd.amin(1), kd.amax(1)), 2).contiguous()
    q, k, v = (torch.zeros(B, h, D, dtype=BF, device=DEV) for h in (Hq, Hkv, Hkv))
    lens, cu = i32(lens0), i32([0, 1, 2, 3])
    ws1 = torch.empty(J.jl_bifocal_select_pages_workspace_size(B, Hkv, table.shape[1], 8), dtype=torch.uint8, device=DEV)
    ws2 = torch.empty(J.jl_bifocal_decode_paged_workspace_size(B, D), dtype=torch.uint8, device=DEV)
    res = {}

    def step(stream=None):
        qr = J.jl_paged_append(k, v, kd, vd, td, cu, lens, 1, page_summary=sm, q=q, rope_theta=theta, stream=stream)
        res["list"] = J.jl_bifocal_select_pages(qr, sm, td, lens, page, 8, w_pre, w0, theta, workspace=ws1,
                                                stream=stream)
        res["q"] = qr
        res["out"], _ = J.jl_bifocal_decode_paged(qr, kd, vd, td, lens, w_pre, w0, theta, page_list=res["list"],
                                                  workspace=ws2, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)  # on a stream that is not the current one
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r in range(3):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g).to(BF))
        lens.copy_(torch.tensor([n + 1 + r for n in lens0], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        n = [a + 1 + r for a in lens0]
        ks = [kd[td[b].long()].reshape(-1, Hkv, D)[:n[b]].cpu() for b in range(B)]
        vs = [vd[td[b].long()].reshape(-1, Hkv, D)[:n[b]].cpu() for b in range(B)]
        want = P.select(res["q"], sm, table, n, page, 8, 1, 1, w_pre, w0, theta)
        assert np.array_equal(res["list"].cpu().numpy(), want)
        pages = [[[c for c in want[b, h] if c >= 0] for h in range(Hkv)] for b in range(B)]
        ro, _, to, _ = P.decode(res["q"], ks, vs, w_pre, w0, theta, lists=pages, page=page)
        P.check(res["out"], ro, to, f"replay {r}")


def test_two_decodes_at_once_on_two_streams():
    # each call allocates its own workspace
    J = jl()
    lens, page = (9000, 4000), 64
    q = torch.randn(2, 32, 128, generator=torch.Generator().manual_seed(3)).to(BF).to(DEV)
    kp, vp, table, _, _ = P.make_cache(lens, page, 8, 128, BF, 2)
    kd, vd, td, ld = kp.to(DEV), vp.to(DEV), table.to(DEV), i32(lens)
    want, _ = J.jl_bifocal_decode_paged(q, kd, vd, td, ld, 1000, 100, 1e4)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        outs = [J.jl_bifocal_decode_paged(q, kd, vd, td, ld, 1000, 100, 1e4, stream=s)[0] for s in streams]
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)


def test_a_strided_block_table():
    lens, page = (500, 300), 16
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(3)).to(BF)
    kp, vp, table, keys, vals = P.make_cache(lens, page, 2, 64, BF, 2)
    wide = torch.full((2, 100), -1, dtype=torch.int32)
    wide[:, 10:10 + table.shape[1]] = table
    J = jl()
    out, lse = J.jl_bifocal_decode_paged(q.to(DEV), kp.to(DEV), vp.to(DEV), wide.to(DEV)[:, 10:10 + table.shape[1]],
                                         i32(lens), 100, 40, 1e4, lse=torch.empty(2, 4, device=DEV))
    ro, rl, to, tl = P.decode(q, keys, vals, 100, 40, 1e4)
    P.check(out, ro, to, "out")
    P.check(lse, rl, tl, "lse")


@pytest.mark.parametrize("D", [128, 64])
def test_decode_returns_whatever_the_wait_limit(D):
    # With the limit at 1 ns a wait that outlasts its first probes gives up.
    # mbarrier.try_wait itself suspends for a time that the hardware sets, so
    # whether one does is not for the test to say: the call must return, report
    # 64 if one did and be right if none did, and leave the next call sound.
    J = jl()
    lens, page = (30000, 9000), 64
    q = torch.randn(2, 8, D, generator=torch.Generator().manual_seed(1)).to(BF)
    kp, vp, table, keys, vals = P.make_cache(lens, page, 2, D, BF, 5)
    kd, vd = kp.to(DEV), vp.to(DEV)
    ws = torch.zeros(J.jl_bifocal_decode_paged_workspace_size(2, D), dtype=torch.uint8, device=DEV)
    assert J.lib().jl_debug_set_wait_limit(1) == 0
    try:
        first, _ = J.jl_bifocal_decode_paged(q.to(DEV), kd, vd, i32(table), i32(lens), 8000, 100, 1e4, workspace=ws)
        torch.cuda.synchronize()
        code = int(ws[:4].view(torch.int32))
        assert code in (0, 64)
    finally:
        assert J.lib().jl_debug_set_wait_limit(0) == 0
    out, lse = run_decode(q, kd, vd, table, lens, 8000, 100, 1e4)
    ro, rl, to, tl = P.decode(q, keys, vals, 8000, 100, 1e4)
    if code == 0:
        P.check(first, ro, to, "out under the short limit")
    P.check(out, ro, to, "out")
    P.check(lse, rl, tl, "lse")


@pytest.mark.parametrize("D,page", [(128, 64), (128, 16), (64, 64)])
def test_decode_reports_a_wait_that_ran_out(D, page):
    # With the limit at 1 ns the first wait for a tile, whose load takes a
    # thousand times that, gives up: every role stops, the loads in flight are
    # let land (which takes no further time-out), the error word says so, and
    # the next call is right.
    J = jl()
    lens = (30000, 9000)
    q = torch.randn(2, 8, D, generator=torch.Generator().manual_seed(1)).to(BF)
    kp, vp, table, keys, vals = P.make_cache(lens, page, 2, D, BF, 5)
    kd, vd, qd, td, ld = kp.to(DEV), vp.to(DEV), q.to(DEV), i32(table), i32(lens)
    want, _ = run_decode(q, kd, vd, table, lens, 8000, 100, 1e4)
    ws = torch.zeros(J.jl_bifocal_decode_paged_workspace_size(2, D), dtype=torch.uint8, device=DEV)
    for _ in range(5):
        try:
            assert J.lib().jl_debug_set_wait_limit(1) == 0
            began = time.perf_counter()
            J.jl_bifocal_decode_paged(qd, kd, vd, td, ld, 8000, 100, 1e4, workspace=ws)
            torch.cuda.synchronize()
            took = time.perf_counter() - began
        finally:
            assert J.lib().jl_debug_set_wait_limit(0) == 0
        assert int(ws[:4].view(torch.int32)) == 64
        assert took < 1.0  # a time-out while the loads land would be 2 s
        out, _ = run_decode(q, kd, vd, table, lens, 8000, 100, 1e4)
        assert torch.equal(out, want)
    ro, _, to, _ = P.decode(q, keys, vals, 8000, 100, 1e4)
    P.check(out, ro, to, "out")


@pytest.mark.parametrize("D,page", [(128, 64), (64, 16)])
def test_decode_at_full_pace_repeats(D, page):
    # no key is turned (G = 1), so the tiles pass at the memory's pace and their
    # loads land out of order: many calls, all alike and right
    J = jl()
    lens = (65536, 31000)
    g = torch.Generator(device=DEV).manual_seed(9)
    n = [-(-x // page) for x in lens]
    kp = torch.randn(sum(n), page, 2, D, generator=g, device=DEV).to(BF)
    vp = torch.randn(sum(n), page, 2, D, generator=g, device=DEV).to(BF)
    order = torch.randperm(sum(n), generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(2, max(n), dtype=torch.int32, device=DEV)
    table[0, :n[0]], table[1, :n[1]] = order[:n[0]], order[n[0]:]
    q = torch.randn(2, 8, D, generator=g, device=DEV).to(BF)
    out, lse = run_decode(q, kp, vp, table, lens, 1 << 20, 64, 1e4)
    keys, vals = [[x[table[b, :n[b]].long()].reshape(-1, 2, D)[:lens[b]].cpu() for b in range(2)] for x in (kp, vp)]
    ro, rl, to, tl = P.decode(q, keys, vals, 1 << 20, 64, 1e4)
    P.check(out, ro, to, "out")
    P.check(lse, rl, tl, "lse")
    ld = i32(lens)
    for _ in range(200):
        again, _ = J.jl_bifocal_decode_paged(q, kp, vp, table, ld, 1 << 20, 64, 1e4)
    assert torch.equal(again, out)


@pytest.mark.parametrize("D,page", [(128, 64), (128, 16), (64, 16)])
def test_every_decode_at_full_pace_is_the_same(D, page):
    # as the test above, but every call's outputs and error word are looked at
    # (on the GPU, so that the calls stay back to back)
    J = jl()
    lens = (65536, 31000)
    g = torch.Generator(device=DEV).manual_seed(10)
    n = [-(-x // page) for x in lens]
    kp = torch.randn(sum(n), page, 2, D, generator=g, device=DEV).to(BF)
    vp = torch.randn(sum(n), page, 2, D, generator=g, device=DEV).to(BF)
    order = torch.randperm(sum(n), generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(2, max(n), dtype=torch.int32, device=DEV)
    table[0, :n[0]], table[1, :n[1]] = order[:n[0]], order[n[0]:]
    q = torch.randn(2, 8, D, generator=g, device=DEV).to(BF)
    want = run_decode(q, kp, vp, table, lens, 1 << 20, 64, 1e4)
    ld = i32(lens)
    calls = 300
    outs = torch.full((calls, 2, 8, D), float("nan"), dtype=BF, device=DEV)
    lses = torch.full((calls, 2, 8), float("nan"), device=DEV)
    ws = torch.full((calls, J.jl_bifocal_decode_paged_workspace_size(2, D)), 0xA5, dtype=torch.uint8, device=DEV)
    for x in range(calls):
        J.jl_bifocal_decode_paged(q, kp, vp, table, ld, 1 << 20, 64, 1e4, out=outs[x], lse=lses[x], workspace=ws[x])
    torch.cuda.synchronize()
    assert torch.equal(ws[:, :4].contiguous().view(torch.int32), torch.zeros(calls, 1, dtype=torch.int32, device=DEV))
    assert torch.equal(outs, want[0].expand_as(outs)) and torch.equal(lses, want[1].expand_as(lses))


@pytest.mark.parametrize("dtype,page", [(BF, 64), (F32, 32)])
def test_pools_past_32_bit_offsets(dtype, page):
    # pages whose first element lies past 2^31, with the largest w_pretrained and
    # w0: everything is local; then turned keys at far positions of a wide table
    J = jl()
    Hkv, D = 8, 128
    n = (1 << 31) // (page * Hkv * D) + 40
    pool = torch.empty(n, 2, page, Hkv, D, dtype=dtype, device=DEV)
    kp, vp = pool[:, 0], pool[:, 1]
    L = 5 * page + 3
    pages = torch.tensor([n - 1, n - 7, n // 2 + 5, n - 2, 0, n - 30], dtype=torch.int32)
    g = torch.Generator().manual_seed(1)
    k, v, q = (torch.randn(L if h == Hkv else 1, h, D, generator=g).to(dtype) for h in (Hkv, Hkv, 16))
    sm = torch.zeros(n, Hkv, 2, D, dtype=dtype, device=DEV)
    J.jl_paged_append(k.to(DEV), v.to(DEV), kp, vp, i32(pages[None]), i32([0, L]), i32([L]), L, page_summary=sm)
    for w_pre, w0 in ((2 ** 63 - 1, 2 ** 31 - 1), (100, 40)):
        out, lse = run_decode(q, kp, vp, pages[None], (L,), w_pre, w0, 1e4)
        ro, rl, to, tl = P.decode(q, [k], [v], w_pre, w0, 1e4)
        P.check(out, ro, to, "out")
        P.check(lse, rl, tl, "lse")
        got = J.jl_bifocal_select_pages(q.to(DEV), sm, i32(pages[None]), i32([L]), page, 3, w_pre, w0, 1e4)
        assert np.array_equal(got.cpu().numpy(), P.select(q, sm.cpu(), pages[None], [L], page, 3, 1, 1, w_pre, w0, 1e4))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_keys_at_far_positions(dtype):
    # a table of 2^30 / 256 pages, most of them one and the same, listed pages at
    # its far end: positions near 2^30, G in the thousands
    J = jl()
    page, Hkv, D, w_pre, w0 = 256, 1, 128, 40000, 300
    cols = (1 << 30) // page
    L = (1 << 30) - 77
    g = torch.Generator().manual_seed(2)
    kp, vp = (torch.randn(6, page, Hkv, D, generator=g).to(dtype) for _ in range(2))
    q = torch.randn(1, 4, D, generator=g).to(dtype)
    table = torch.zeros(1, cols, dtype=torch.int32)
    want = [3, 70000, cols // 2 + 1, cols - 3, cols - 2, cols - 1]
    for x, c in enumerate(want):
        table[0, c] = x
    lists = torch.tensor(want, dtype=torch.int32).view(1, 1, -1)
    out, lse = run_decode(q, kp.to(DEV), vp.to(DEV), table, (L,), w_pre, w0, 1e4, page_list=i32(lists))
    # the plain form, on the listed keys alone
    pos = np.concatenate([np.arange(c * page, (c + 1) * page) for c in want])
    seen = pos < L
    G = P.group(L, w_pre)
    shift = np.where(pos < L - w0, (pos // G - pos) - ((L - 1) // G - (L - 1)), 0)[seen]
    raw, vv = P.f64(kp).reshape(-1, D)[seen], P.f64(vp).reshape(-1, D)[seen]
    kk = P.rotate(raw, shift, 1e4)
    for h in range(4):
        s = kk @ P.f64(q)[0, h] / np.sqrt(D)
        e = np.exp(s - s.max())
        size = (P.pair_len(raw) @ np.abs(P.f64(q)[0, h])).max() / np.sqrt(D)
        # the angle itself, n w, is known to n w 2^-53 and the turn to 2^-32
        ds, dw = P.slack(size * (1 + (2.0 ** 30 * 2.0 ** -52 + 2 * np.pi * 2.0 ** -32) / (160 * P.U)), abs(s).max(),
                         len(s), dtype == BF)
        ref = e @ vv / e.sum()
        P.check(out[0, h], ref, dw * np.abs(vv).max() + (2.0 ** -8 if dtype == BF else P.U) * np.abs(ref), f"head {h}")
