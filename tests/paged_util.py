"""Plain 64-bit forms of the paged-cache operators, for the tests: written from
the formulas, key by key positions, no page arithmetic shared with the
library.  Inputs are CPU tensors."""
import math

import numpy as np
import torch

U = 2.0 ** -24  # half a step of fp32


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def rotate(x, n, theta):
    """x [..., D] rotated by n positions (n broadcast over the leading axes)."""
    d = x.shape[-1]
    ang = np.asarray(n, dtype=np.float64)[..., None] * theta ** (-2.0 * np.arange(d // 2) / d)
    a, b = x[..., : d // 2], x[..., d // 2:]
    c, s = np.cos(ang), np.sin(ang)
    return np.concatenate([a * c - b * s, b * c + a * s], axis=-1)


def group(L, w_pre):
    return max(1, -(-L // w_pre))


def pair_len(x):
    """Length of each rotation pair, at both of its places: what a rotation can
    make of an element."""
    a, b = np.split(np.abs(x), 2, axis=-1)
    r = np.hypot(a, b)
    return np.concatenate([r, r], axis=-1)


def make_cache(lens, page, hkv, d, dtype, seed, spare=2, interleaved=False, fill=None):
    """A pool whose pages are dealt out in random order, with garbage (or
    ``fill``) in every slot that no key of ``lens`` owns.  Returns (k_pages,
    v_pages, table, keys, values) with keys[b] [L_b, Hkv, D]."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    total, cols = sum(need) + spare, max(1, max(need, default=1))
    pool = torch.full((total, 2, page, hkv, d), 1e4 if fill is None else fill, dtype=torch.float32)
    table = torch.full((len(lens), cols), -7, dtype=torch.int32)
    order = torch.randperm(total, generator=g)
    keys, vals, at = [], [], 0
    for b, n in enumerate(lens):
        k = torch.randn(n, hkv, d, generator=g).to(dtype)
        v = torch.randn(n, hkv, d, generator=g).to(dtype)
        keys.append(k)
        vals.append(v)
        for c in range(need[b]):
            one = int(order[at])
            at += 1
            table[b, c] = one
            m = min(page, n - c * page)
            pool[one, 0, :m] = k[c * page:c * page + m].float()
            pool[one, 1, :m] = v[c * page:c * page + m].float()
    pool = pool.to(dtype)
    if interleaved:
        return pool[:, 0], pool[:, 1], table, keys, vals
    return pool[:, 0].contiguous(), pool[:, 1].contiguous(), table, keys, vals


def decode(q, keys, vals, w_pre, w0, theta, window=0, lists=None, page=0, missing=None, plain=False):
    """(out [B, Hq, D], lse [B, Hq], bound of |out| errors, bound of |lse|
    errors).  lists[b][h]: logical pages read (None: all); missing[b]: logical
    pages that are not there.  The bounds count roundings: see ``slack``."""
    q = f64(q)
    B, Hq, D = q.shape
    hkv = keys[0].shape[1]
    gs = Hq // hkv
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    tol_o, tol_l = np.zeros((B, Hq, 1)), np.zeros((B, Hq))
    bf16 = keys[0].dtype == torch.bfloat16
    for b in range(B):
        k, v = f64(keys[b]), f64(vals[b])
        L = k.shape[0]
        G = 1 if plain else group(L, w_pre)
        for h in range(hkv):
            if lists is None:
                pos = np.arange(L)
            else:
                pos = np.concatenate([np.arange(c * page, (c + 1) * page) for c in lists[b][h]] or [np.zeros(0)])
                pos = pos.astype(np.int64)
            pos = pos[pos < L]
            if window:
                pos = pos[pos >= L - window]
            if missing is not None:
                pos = pos[~np.isin(pos // page, missing[b])]
            if pos.size == 0:
                continue
            far = pos < L - w0
            shift = np.where(far, (pos // G - pos) - ((L - 1) // G - (L - 1)), 0)
            kk = rotate(k[pos, h], shift, theta)
            vv = v[pos, h]
            for x in range(h * gs, (h + 1) * gs):
                s = kk @ q[b, x] / math.sqrt(D)
                m = s.max()
                e = np.exp(s - m)
                out[b, x] = e @ vv / e.sum()
                lse[b, x] = m + np.log(e.sum())
                size = (pair_len(k[pos, h]) @ np.abs(q[b, x])).max() / math.sqrt(D)
                ds, dw = slack(size, abs(s).max(), pos.size, bf16)
                tol_o[b, x] = dw * np.abs(vv).max()
                tol_l[b, x] = ds + dw + 4 * U * max(1.0, abs(lse[b, x]))
    half_step = 2.0 ** -8 if bf16 else U
    return out, lse, tol_o + half_step * np.abs(out), tol_l


def slack(size, top, n, bf16):
    """(error of a score, relative error that the weighted sum can add up to).

    A score is a sum of D products whose sizes add up to at most ``size``: 128
    roundings of a chain, 30 of the turned key (its angle, at most 8 steps of 3
    roundings, its products), each U relative to it.  In bf16 a turned key is
    the sum of two bf16: the first is off by 2^-8, the second by 2^-8 of that.
    A weight e^(s - m) moves by the errors of s and m, by the exponential's own
    error (4 U, and 2 U |s - m| for the scaled argument); in bf16 it too is a
    sum of two bf16.  Sums of n weights: a chain of n / 8 + 64 roundings.  The
    numerator and the sum below it both move: twice."""
    ds = size * (160 * U + (2.0 ** -16 if bf16 else 0.0))
    dw = 2 * (2 * ds + (8 + 4 * top) * U + (n / 8 + 64) * U + (2.0 ** -16 if bf16 else 0.0))
    return ds, dw


def check(got, want, tol, what=""):
    got = got if isinstance(got, np.ndarray) else f64(got)
    fine = np.isfinite(want)
    assert np.array_equal(fine, np.isfinite(got)), f"{what}: not finite elsewhere"
    assert np.array_equal(want[~fine], got[~fine]), what
    err = np.abs(np.where(fine, got, 0.0) - np.where(fine, want, 0.0))
    worst = (err / np.maximum(np.broadcast_to(tol, err.shape), 1e-300))[fine]
    assert worst.size == 0 or worst.max() <= 1.0, f"{what}: {worst.max():.2f} of the tolerance, error {err.max():.3e}"


def select(q, summary, table, lens, page, n_select, n_first, n_last, w_pre, w0, theta, plain=False):
    """page_list [B, Hkv, n_select] from the definition, in 64 bits."""
    q, sm = f64(q), f64(summary)
    B, Hq, D = q.shape
    n_pages, hkv = sm.shape[:2]
    gs = Hq // hkv
    out = np.full((B, hkv, n_select), -1, dtype=np.int64)
    for b, L in enumerate(lens):
        n = -(-L // page)
        if L > table.shape[1] * page:
            continue
        if n <= n_select:
            out[b, :, :n] = np.arange(n)
            continue
        G = 1 if plain else group(L, w_pre)
        i = L - 1
        for h in range(hkv):
            score = np.empty(n)
            for c in range(n):
                one = int(table[b, c])
                if not 0 <= one < n_pages:
                    score[c] = -np.inf
                    continue
                m = c * page + page // 2
                turn = (m - m // G) - (i - i // G) if m < L - w0 else 0
                t = rotate(q[b, h * gs:(h + 1) * gs], np.full(gs, turn), theta)
                with np.errstate(invalid="ignore", over="ignore"):
                    x = np.maximum(t * sm[one, h, 0], t * sm[one, h, 1]).sum(-1)
                score[c] = x.max() if np.isfinite(x).all() else np.inf
            forced = [c for c in range(n) if c < n_first or c >= n - n_last]
            rest = [c for c in range(n) if n_first <= c < n - n_last]
            rest.sort(key=lambda c: (-score[c], c))
            out[b, h] = sorted(forced + rest[:n_select - len(forced)])
    return out
