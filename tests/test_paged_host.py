"""Refusals of the paged-cache calls that need no GPU: the C ABI on raw
arguments, and the binding's checks of shapes, types, strides and devices."""
import ctypes

import numpy as np
import pytest
import torch

from tests import paged_util as P


def _lib():
    from zero_shot_rope_b200 import build, jetlong
    build.build()
    return jetlong


A = 1 << 12  # an aligned address that is never read


def _append_raw(jl, **kw):
    a = dict(k=A, v=A, kp=A, vp=A, sm=A, table=A, ts=4, cols=4, cu=A, sl=A, B=2, T=8, new=4, Hq=4, Hkv=2, D=128, page=16,
             n=10, ps=16 * 2 * 128, q=A, qo=A, theta=1e4, dtype=jl.JL_BF16, flags=jl.JL_FLAG_ROTATE)
    a.update(kw)
    return jl.lib().jl_paged_append(a["k"], a["v"], a["kp"], a["vp"], a["sm"], a["table"], a["ts"], a["cols"], a["cu"],
                                    a["sl"], a["B"], a["T"], a["new"], a["Hq"], a["Hkv"], a["D"], a["page"], a["n"],
                                    a["ps"], a["q"], a["qo"], a["theta"], a["dtype"], a["flags"], None)


def _select_raw(jl, **kw):
    a = dict(q=A, sm=A, table=A, ts=40, cols=40, sl=A, B=2, Hq=4, Hkv=2, D=128, page=16, n=10, sel=8, first=1, last=1,
             w_pre=100, w0=10, theta=1e4, out=A, ws=1 << 20, wsb=1 << 30, dtype=jl.JL_BF16, flags=0)
    a.update(kw)
    return jl.lib().jl_bifocal_select_pages(a["q"], a["sm"], a["table"], a["ts"], a["cols"], a["sl"], a["B"], a["Hq"],
                                            a["Hkv"], a["D"], a["page"], a["n"], a["sel"], a["first"], a["last"],
                                            a["w_pre"], a["w0"], a["theta"], a["out"], a["ws"], a["wsb"], a["dtype"],
                                            a["flags"], None)


def _decode_raw(jl, **kw):
    a = dict(q=A, kp=A, vp=A, table=A, ts=40, cols=40, sl=A, list=None, nl=0, B=2, Hq=4, Hkv=2, D=128, page=16, n=10,
             ps=16 * 2 * 128, w_pre=100, w0=10, window=0, theta=1e4, out=A, lse=None, ws=1 << 20, wsb=1 << 30,
             dtype=jl.JL_BF16, flags=0)
    a.update(kw)
    return jl.lib().jl_bifocal_decode_paged(a["q"], a["kp"], a["vp"], a["table"], a["ts"], a["cols"], a["sl"], a["list"],
                                            a["nl"], a["B"], a["Hq"], a["Hkv"], a["D"], a["page"], a["n"], a["ps"],
                                            a["w_pre"], a["w0"], a["window"], a["theta"], a["out"], a["lse"], a["ws"],
                                            a["wsb"], a["dtype"], a["flags"], None)


COMMON = [
    (dict(Hq=3), "JL_ERR_INVALID_ARG"),
    (dict(Hkv=0), "JL_ERR_INVALID_ARG"),
    (dict(D=96), "JL_ERR_UNSUPPORTED"),
    (dict(theta=0.0), "JL_ERR_INVALID_ARG"),
    (dict(theta=float("inf")), "JL_ERR_INVALID_ARG"),
    (dict(dtype=5), "JL_ERR_INVALID_ARG"),
    (dict(page=24), "JL_ERR_INVALID_ARG"),
    (dict(page=0), "JL_ERR_INVALID_ARG"),
    (dict(page=8), "JL_ERR_UNSUPPORTED"),
    (dict(page=512, ps=512 * 256), "JL_ERR_UNSUPPORTED"),
    (dict(n=0), "JL_ERR_INVALID_ARG"),
    (dict(cols=0), "JL_ERR_INVALID_ARG"),
    (dict(ts=3), "JL_ERR_INVALID_ARG"),
    (dict(cols=1 << 27, ts=1 << 27), "JL_ERR_UNSUPPORTED"),
    (dict(B=-1), "JL_ERR_INVALID_ARG"),
    (dict(B=65536), "JL_ERR_UNSUPPORTED"),
    (dict(flags=0x40), "JL_ERR_INVALID_ARG"),
    (dict(q=A + 8), "JL_ERR_INVALID_ARG"),
    (dict(table=None), "JL_ERR_INVALID_ARG"),
    (dict(sl=None), "JL_ERR_INVALID_ARG"),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(k=None), "JL_ERR_INVALID_ARG"),
    (dict(vp=None), "JL_ERR_INVALID_ARG"),
    (dict(cu=None), "JL_ERR_INVALID_ARG"),
    (dict(sm=A + 4), "JL_ERR_INVALID_ARG"),
    (dict(q=None), "JL_ERR_INVALID_ARG"),          # q_out without q
    (dict(qo=None), "JL_ERR_INVALID_ARG"),
    (dict(flags=0), "JL_ERR_INVALID_ARG"),         # q without rotation
    (dict(flags=1), "JL_ERR_INVALID_ARG"),
    (dict(new=9), "JL_ERR_INVALID_ARG"),
    (dict(new=0), "JL_ERR_INVALID_ARG"),
    (dict(T=-1), "JL_ERR_INVALID_ARG"),
    (dict(ps=16 * 2 * 128 - 8), "JL_ERR_INVALID_ARG"),
    (dict(ps=16 * 2 * 128 + 4), "JL_ERR_INVALID_ARG"),
    (dict(Hkv=70000, Hq=70000, ps=16 * 70000 * 128), "JL_ERR_UNSUPPORTED"),
])
def test_append_refuses(kw, status):
    jl = _lib()
    assert jl.status_string(_append_raw(jl, **kw)) == status, jl.last_error()
    assert jl.last_error()


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(sm=None), "JL_ERR_INVALID_ARG"),
    (dict(out=None), "JL_ERR_INVALID_ARG"),
    (dict(sel=0), "JL_ERR_INVALID_ARG"),
    (dict(first=-1), "JL_ERR_INVALID_ARG"),
    (dict(first=5, last=4), "JL_ERR_INVALID_ARG"),
    (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), "JL_ERR_INVALID_ARG"),
    (dict(w_pre=0), "JL_ERR_INVALID_ARG"),
    (dict(w0=-1), "JL_ERR_INVALID_ARG"),
    (dict(ws=None), "JL_ERR_WORKSPACE"),
    (dict(wsb=100), "JL_ERR_WORKSPACE"),
    (dict(ws=(1 << 20) + 16), "JL_ERR_WORKSPACE"),
])
def test_select_refuses(kw, status):
    jl = _lib()
    assert jl.status_string(_select_raw(jl, **kw)) == status, jl.last_error()


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(kp=None), "JL_ERR_INVALID_ARG"),
    (dict(out=None), "JL_ERR_INVALID_ARG"),
    (dict(w_pre=0), "JL_ERR_INVALID_ARG"),
    (dict(w0=-1), "JL_ERR_INVALID_ARG"),
    (dict(window=-1), "JL_ERR_INVALID_ARG"),
    (dict(nl=3), "JL_ERR_INVALID_ARG"),            # a count without a list
    (dict(list=A, nl=-1), "JL_ERR_INVALID_ARG"),
    (dict(list=A, nl=(1 << 20) + 1), "JL_ERR_INVALID_ARG"),
    (dict(ps=0), "JL_ERR_INVALID_ARG"),
    (dict(ws=None), "JL_ERR_WORKSPACE"),
    (dict(wsb=100), "JL_ERR_WORKSPACE"),
    (dict(ws=(1 << 20) + 16), "JL_ERR_WORKSPACE"),
    (dict(flags=0x8), "JL_ERR_INVALID_ARG"),
])
def test_decode_refuses(kw, status):
    jl = _lib()
    assert jl.status_string(_decode_raw(jl, **kw)) == status, jl.last_error()


@pytest.mark.parametrize("Hq,Hkv", [(65536, 2), (1 << 20, 1 << 20), (1 << 30, 1)])
def test_more_heads_than_a_call_takes(Hq, Hkv):
    jl = _lib()
    for call in (_append_raw, _select_raw, _decode_raw):
        kw = {} if call is _select_raw else dict(ps=16 * Hkv * 128)
        assert jl.status_string(call(jl, Hq=Hq, Hkv=Hkv, **kw)) == "JL_ERR_UNSUPPORTED" and "heads" in jl.last_error()


def test_empty_calls_are_no_ops():
    jl = _lib()
    assert _append_raw(jl, B=0) == jl.JL_OK and _append_raw(jl, T=0, new=0) == jl.JL_OK
    assert _select_raw(jl, B=0) == jl.JL_OK and _decode_raw(jl, B=0) == jl.JL_OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the behaviour without a GPU")
def test_calls_fail_loudly_without_a_gpu():
    jl = _lib()
    for call in (_append_raw, _select_raw, _decode_raw):
        assert jl.status_string(call(jl)) == "JL_ERR_CUDA" and jl.last_error()


def test_workspace_sizes():
    jl = _lib()
    assert jl.jl_bifocal_decode_paged_workspace_size(0, 128) == 0
    sizes = [jl.jl_bifocal_decode_paged_workspace_size(b, 128) for b in (1, 64, 65535)]
    assert 0 < sizes[0] <= sizes[1] < sizes[2] < 8 << 20
    assert jl.jl_bifocal_select_pages_workspace_size(4, 8, 64, 64) == 0  # every page is listed: nothing is scored
    assert jl.jl_bifocal_select_pages_workspace_size(4, 8, 65, 64) >= 4 * 8 * 65 * 20
    assert jl.jl_bifocal_select_pages_workspace_size(65535, 8, 1 << 20, 64) >= 65535 * 8 * (1 << 20) * 20


def _tensors(dtype=torch.bfloat16):
    t = dict(k=torch.zeros(3, 2, 64, dtype=dtype), kp=torch.zeros(5, 16, 2, 64, dtype=dtype),
             table=torch.zeros(2, 4, dtype=torch.int32), cu=torch.zeros(3, dtype=torch.int32),
             lens=torch.zeros(2, dtype=torch.int32), sm=torch.zeros(5, 2, 2, 64, dtype=dtype),
             q=torch.zeros(2, 4, 64, dtype=dtype), list=torch.zeros(2, 2, 3, dtype=torch.int32))
    t["v"], t["vp"] = t["k"].clone(), t["kp"].clone()
    return t


def _calls(jl, t):
    return {
        "append": lambda: jl.jl_paged_append(t["k"], t["v"], t["kp"], t["vp"], t["table"], t["cu"], t["lens"], 2,
                                             page_summary=t["sm"]),
        "select": lambda: jl.jl_bifocal_select_pages(t["q"], t["sm"], t["table"], t["lens"], 16, 2, 10, 1, 1e4),
        "decode": lambda: jl.jl_bifocal_decode_paged(t["q"], t["kp"], t["vp"], t["table"], t["lens"], 10, 1, 1e4,
                                                     page_list=t["list"]),
    }


BAD = [
    ("append", dict(v=torch.zeros(3, 2, 128, dtype=torch.bfloat16)), ValueError),
    ("append", dict(v=torch.zeros(3, 2, 64)), TypeError),
    ("append", dict(k=torch.zeros(3, 64, 2, dtype=torch.bfloat16).transpose(1, 2)), ValueError),
    ("append", dict(k=torch.zeros(3, 2, 64, dtype=torch.float16)), TypeError),
    ("append", dict(k=torch.zeros(6, 64, dtype=torch.bfloat16)), ValueError),
    ("append", dict(cu=torch.zeros(2, dtype=torch.int32)), ValueError),
    ("append", dict(cu=torch.zeros(3, dtype=torch.int64)), TypeError),
    ("append", dict(sm=torch.zeros(5, 2, 64, 2, dtype=torch.bfloat16)), ValueError),
    ("append", dict(sm=torch.zeros(5, 2, 2, 64)), TypeError),
    ("append", dict(kp=torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16)), ValueError),
    ("append", dict(kp=torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16).transpose(1, 2)), ValueError),
    ("append", dict(kp=torch.zeros(5, 2, 16, 2, 64, dtype=torch.bfloat16)[:, 0]), ValueError),  # strides differ from v's
    ("append", dict(kp=torch.zeros(0, 16, 2, 64, dtype=torch.bfloat16), vp=torch.zeros(0, 16, 2, 64, dtype=torch.bfloat16)),
     ValueError),
    ("append", dict(table=torch.zeros(3, 4, dtype=torch.int32)), ValueError),
    ("append", dict(table=torch.zeros(4, 2, dtype=torch.int32).t()), ValueError),
    ("append", dict(table=torch.zeros(2, 4, dtype=torch.int64)), TypeError),
    ("select", dict(sm=torch.zeros(5, 2, 64, dtype=torch.bfloat16)), ValueError),
    ("select", dict(sm=torch.zeros(5, 2, 2, 64)), TypeError),
    ("select", dict(lens=torch.zeros(3, dtype=torch.int32)), ValueError),
    ("select", dict(q=torch.zeros(2, 256, dtype=torch.bfloat16)), ValueError),
    ("decode", dict(list=torch.zeros(2, 4, 3, dtype=torch.int32)), ValueError),
    ("decode", dict(list=torch.zeros(2, 2, 3, dtype=torch.int64)), TypeError),
    ("decode", dict(list=torch.zeros(2, 2, 6, dtype=torch.int32)[:, :, ::2]), ValueError),
    ("decode", dict(q=torch.zeros(2, 4, 128, dtype=torch.bfloat16)), ValueError),
    ("decode", dict(kp=torch.zeros(5, 16, 128, dtype=torch.bfloat16)), ValueError),
    ("decode", dict(vp=torch.zeros(5, 16, 2, 64)), TypeError),
]


@pytest.mark.parametrize("call,kw,error", BAD)
def test_binding_refuses(call, kw, error):
    jl = _lib()
    t = _tensors()
    t.update(kw)
    with pytest.raises(error):
        _calls(jl, t)[call]()


def test_binding_refuses_host_tensors_and_lone_queries():
    jl = _lib()
    t = _tensors()
    for call in _calls(jl, t).values():
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="rope_theta"):
        jl.jl_paged_append(t["k"], t["v"], t["kp"], t["vp"], t["table"], t["cu"], t["lens"], 2, q=t["k"])


def test_plain_forms_agree_with_the_oracle():
    # the 64-bit forms that the GPU tests compare against, against the oracle
    import oracle

    g = torch.Generator().manual_seed(3)
    lens = (300, 41)
    kp, vp, table, keys, vals = P.make_cache(lens, 16, 2, 64, torch.float32, 5)
    q = torch.randn(2, 4, 64, generator=g)
    kc, vc = torch.zeros(2, 300, 2, 64), torch.zeros(2, 300, 2, 64)
    for b, n in enumerate(lens):
        kc[b, :n], vc[b, :n] = keys[b], vals[b]
        got = kp[table[b, : -(-n // 16)].long()].reshape(-1, 2, 64)[:n]
        assert torch.equal(got, keys[b])
    for kw in ({}, {"plain": True}, {"window": 77}):
        out, lse, _, _ = P.decode(q, keys, vals, 70, 30, 1e4, **kw)
        ro, rl = oracle.bifocal_decode(q, kc, vc, list(lens), 70, 30, 1e4, **kw)
        assert np.abs(out - ro).max() < 1e-12 and np.abs(lse - rl).max() < 1e-12
    every = [[list(range(19))] * 2, [list(range(3))] * 2]
    a, b = P.decode(q, keys, vals, 70, 30, 1e4)[0], P.decode(q, keys, vals, 70, 30, 1e4, lists=every, page=16)[0]
    assert np.abs(a - b).max() == 0.0
    x = np.random.default_rng(0).normal(size=(5, 64))
    assert np.abs(P.rotate(P.rotate(x, np.full(5, 9), 1e4), np.full(5, -9), 1e4) - x).max() < 1e-14


def test_turns_match_64_bit_angles():
    # cos and sin within 3 steps of 2^-24 for every position and frequency, the
    # frequencies of a base below 1 and the largest positions among them; the
    # angle itself is known to n w 2^-53 (the frequency is a double)
    jl = _lib()
    L = jl.lib()
    L.jl_debug_turn_cs.argtypes = [ctypes.c_int32, ctypes.c_double, ctypes.POINTER(ctypes.c_float),
                                   ctypes.POINTER(ctypes.c_float)]
    c, s = ctypes.c_float(), ctypes.c_float()
    rng = np.random.default_rng(1)
    worst = 0.0
    for theta in (1e4, 1e6, 0.5):
        for k in range(64):
            w = theta ** (-2.0 * k / 128)
            for n in [0, 1, -1, 2, 16, -131071, 131071, 2 ** 30] + rng.integers(-2 ** 20, 2 ** 20, 60).tolist():
                L.jl_debug_turn_cs(int(n), w, ctypes.byref(c), ctypes.byref(s))
                slack = 3 * 2.0 ** -24 + 4 * abs(n) * w * 2.0 ** -53
                err = max(abs(c.value - np.cos(n * w)), abs(s.value - np.sin(n * w)))
                worst = max(worst, err / slack)
    assert worst <= 1.0, worst
    L.jl_debug_turn_cs(0, 1.0, ctypes.byref(c), ctypes.byref(s))
    assert c.value == 1.0 and s.value == 0.0


def test_turns_of_high_frequencies():
    # bases below 1 have frequencies above 1: cos and sin within 3 steps of 2^-24
    # of those of the exact product, at every position (worked out in whole numbers)
    from decimal import Decimal, getcontext

    getcontext().prec = 140
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534"
                         "211706798214808651328230664709384460955058223172535940812848111745")
    per_turn = int((1 / two_pi) * (1 << 400))  # 1 / (2 pi), in 2^-400
    jl = _lib()
    L = jl.lib()
    L.jl_debug_turn_cs.argtypes = [ctypes.c_int32, ctypes.c_double, ctypes.POINTER(ctypes.c_float),
                                   ctypes.POINTER(ctypes.c_float)]
    c, s = ctypes.c_float(), ctypes.c_float()
    rng = np.random.default_rng(2)
    worst = 0.0
    for theta in (1e6, 0.5, 1e-3, 1e-12, 2.0 ** -32):
        for k in range(0, 64, 3):
            w = theta ** (-2.0 * k / 128)
            num, den = w.as_integer_ratio()
            for n in [1, -3, 2 ** 30, -(2 ** 30) + 1, 2 ** 31 - 1] + rng.integers(-2 ** 30, 2 ** 30, 25).tolist():
                turns = (n * num * per_turn // den) & ((1 << 400) - 1)
                a = float(Decimal(turns) / (1 << 400) * two_pi)
                L.jl_debug_turn_cs(int(n), w, ctypes.byref(c), ctypes.byref(s))
                worst = max(worst, abs(c.value - np.cos(a)), abs(s.value - np.sin(a)))
    assert worst <= 3 * 2.0 ** -24, worst * 2.0 ** 24


def test_packed_call_checks_its_words():
    import struct

    jl = _lib()
    L = jl.lib()

    def call(which, words, n=None):
        data = struct.pack(f"={len(words)}q", *words)
        return jl.status_string(L.jl_paged_call(which, data, len(words) if n is None else n))

    theta = struct.unpack("=q", struct.pack("=d", 1e4))[0]
    append = [A, A, A, A, 0, A, 4, 4, A, A, 0, 8, 4, 4, 2, 128, 16, 10, 16 * 256, 0, 0, theta, 0, 0, 0]
    select = [A, A, A, 40, 40, A, 0, 4, 2, 128, 16, 10, 8, 1, 1, 100, 10, theta, A, 1 << 20, 1 << 30, 0, 0, 0]
    decode = [A, A, A, A, 40, 40, A, 0, 0, 0, 4, 2, 128, 16, 10, 16 * 256, 100, 10, 0, theta, A, 0, 1 << 20, 1 << 30, 0,
              0, 0]
    for which, words in enumerate((append, select, decode)):
        assert call(which, words) == "JL_OK"          # an empty batch
        assert call(which, words[:-1]) == "JL_ERR_INVALID_ARG"
        assert call(which, words + [0]) == "JL_ERR_INVALID_ARG"
        at = words.index(128)
        assert call(which, words[:at] + [128 + (1 << 32)] + words[at + 1:]) == "JL_ERR_INVALID_ARG"
        assert call(which, words[:at] + [96] + words[at + 1:]) == "JL_ERR_UNSUPPORTED"
        assert call(which, words[:-2] + [-1, 0]) == "JL_ERR_INVALID_ARG"   # flags
    assert call(3, append) == "JL_ERR_INVALID_ARG" and call(-1, append) == "JL_ERR_INVALID_ARG"
    assert jl.status_string(L.jl_paged_call(0, None, 25)) == "JL_ERR_INVALID_ARG"
