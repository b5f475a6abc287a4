"""Timed cases of the paged-cache operators, with their plain forms.

Three operators make up one generation step over a paged key-value cache:
``append`` rotates new tokens and writes them into their pages, ``select``
scores the pages by their key ranges and lists the ones worth reading, and
``decode`` attends one new token per sequence to the pages (all of them, a
sliding window, or the listed ones).

``run`` computes the plain form in elementary torch operations while ``own``
is false, and makes the library's calls when it is true.
"""
import math

import torch

own = False

BF16, FP32 = "bf16", "fp32"
_TORCH = {BF16: torch.bfloat16, FP32: torch.float32}


def _case(name, op, batch, lo, hi, hq, hkv, dim, page, dtype, w_pre, w0, theta=1.0e6, new=0, select=0, window=0):
    """One case.  Sequence lengths run evenly from ``lo`` to ``hi``; ``new``:
    longest number of appended tokens; ``select``: pages in a list (0: no
    list); ``window``: sliding window (0: none)."""
    return dict(name=name, op=op, batch=batch, lo=lo, hi=hi, hq=hq, hkv=hkv, dim=dim, page=page, dtype=dtype,
                w_pre=w_pre, w0=w0, theta=theta, new=new, select=select, window=window)


def listed():
    return [
        # one sequence of the 32/8-head model generates: its token enters the cache (latency)
        _case("append 1 token", "append", 1, 5001, 5001, 32, 8, 128, 64, BF16, 32768, 4096, new=1),
        # a serving batch generates: 64 tokens enter ragged sequences in small pages
        _case("append 64x1", "append", 64, 33, 8190, 32, 8, 128, 16, BF16, 32768, 4096, new=1),
        # a whole 32K prompt of the 16/8-head model is written behind its prefill
        _case("append 32K prompt", "append", 1, 32768, 32768, 16, 8, 128, 64, BF16, 32768, 4096, new=32768),
        # ragged chunks that start and end inside pages, in fp32 at head_dim 64
        _case("append chunks fp32", "append", 7, 700, 2900, 4, 2, 64, 32, FP32, 256, 64, 1.0e4, new=611),
        # which 64 of the 2048 pages of a 128K context the next token reads
        _case("select 128K", "select", 1, 131072, 131072, 32, 8, 128, 64, BF16, 32768, 4096, select=64),
        # the same for a ragged batch of 32
        _case("select 32x32K", "select", 32, 4100, 32767, 32, 8, 128, 64, BF16, 4096, 1024, select=64),
        # small pages, head_dim 64, fp32: a short-context model
        _case("select small fp32", "select", 3, 900, 2500, 8, 2, 64, 16, FP32, 256, 64, 1.0e4, select=24),
        # the smallest decode: one 1024-token sequence, 2/1 heads, fp32
        _case("decode 1K fp32", "decode", 1, 1024, 1024, 2, 1, 64, 16, FP32, 256, 64, 1.0e4),
        # one token over a 128K context, every key read
        _case("decode 128K", "decode", 1, 131072, 131072, 32, 8, 128, 64, BF16, 32768, 4096),
        # a ragged serving batch in small pages
        _case("decode 16x32K", "decode", 16, 4097, 32768, 32, 8, 128, 16, BF16, 4096, 1024),
        # the sparse step: 16 long sequences, 64 listed pages of each kv head
        _case("decode 16x64K listed", "decode", 16, 20011, 65536, 32, 8, 128, 64, BF16, 32768, 4096, select=64),
        # a sliding-window layer in fp32, odd lengths
        _case("decode window fp32", "decode", 5, 3001, 17777, 8, 2, 128, 32, FP32, 2048, 512, window=8200),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("append", "select", "decode", "decode"))
    dtype = rng.choice((BF16, BF16, FP32))
    hq, hkv = rng.choice(((32, 8), (16, 8), (8, 8), (16, 2), (8, 1), (12, 4), (2, 1)))
    dim = rng.choice((64, 128))
    page = rng.choice((16, 32, 64, 128))
    size = 2 if dtype == BF16 else 4
    row = hkv * dim * size
    w_pre = rng.choice((256, 4096, 32768))
    w0 = _spread(rng, 1, w_pre // 2)
    theta = rng.choice((1.0e4, 1.0e6))
    new = select = window = 0
    if op == "append":
        new = _spread(rng, 1, max(1, (1 << 27) // (row + hq * dim * size // 2)))
        new = min(new, 32768)
        batch = _spread(rng, 1, max(1, min(64, 32768 // new)))
        hi = new + _spread(rng, 1, 4096)
        lo = max(new, hi // 3)
    elif op == "select":
        hi = _spread(rng, 2 * page, 131072)
        batch = _spread(rng, 1, max(1, min(64, (1 << 25) // (2 * (hi // page) * row), (1 << 26) // ((hi // page) * hq * dim))))
        lo = max(1, hi // rng.choice((1, 2, 8)))
        select = _spread(rng, 2, 96)
    else:
        hi = _spread(rng, 1, 131072)
        batch = _spread(rng, 1, max(1, min(64, (1 << 30) // (2 * hi * row))))
        lo = max(1, hi // rng.choice((1, 2, 8)))
        kind = rng.choice(("all", "all", "list", "window"))
        if kind == "list":
            select = _spread(rng, 1, 96)
        if kind == "window":
            window = _spread(rng, 1, 8192)
    c = _case("", op, batch, lo, hi, hq, hkv, dim, page, dtype, w_pre, w0, theta, new, select, window)
    del c["name"]
    return c


# ------------------------------------------------------------------- sizes
def _lengths(c):
    """Lengths of the sequences, the new tokens included."""
    b = c["batch"]
    return [c["hi"]] if b == 1 else [c["lo"] + (c["hi"] - c["lo"]) * k // (b - 1) for k in range(b)]


def _news(c):
    """Appended tokens of each sequence: ``new`` for the first, fewer for some
    of the others, at least one."""
    return [max(1, c["new"] - (c["new"] * (k % 5)) // 7) for k in range(c["batch"])]


def _pages_of(c, length):
    return -(-length // c["page"])


def work(case):
    c = case
    size = 2 if c["dtype"] == BF16 else 4
    row = c["dim"] * size  # one head of one token
    lens = _lengths(c)
    if c["op"] == "append":
        t = sum(_news(c))
        touched = sum((n - 1) // c["page"] + 1 for n in _news(c))
        moved = 2 * t * (c["hq"] + 2 * c["hkv"]) * row + touched * c["hkv"] * 2 * row
        return {"bytes": moved, "flops": 3 * t * (c["hq"] + c["hkv"]) * c["dim"]}
    if c["op"] == "select":
        pages = sum(_pages_of(c, n) for n in lens)
        moved = pages * (c["hkv"] * 2 * row + 4) + c["batch"] * (c["hq"] * row + c["hkv"] * c["select"] * 4)
        return {"bytes": moved, "flops": pages * c["hq"] * c["dim"] * 5}
    keys = 0
    for n in lens:
        if c["select"]:
            n = min(n, c["select"] * c["page"])
        keys += min(n, c["window"]) if c["window"] else n
    moved = keys * c["hkv"] * 2 * row + c["batch"] * c["hq"] * (2 * row + 4)
    return {"bytes": moved, "flops": keys * (4 * c["hq"] + 3 * c["hkv"]) * c["dim"]}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    dt = _TORCH[c["dtype"]]
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    lens, p, b = _lengths(c), c["page"], c["batch"]
    cols = max(_pages_of(c, n) for n in lens)
    need = [_pages_of(c, n) for n in lens]
    total = sum(need) + 3  # a few pages of the pool belong to nobody
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(b, cols, dtype=torch.int32, device=dev)
    at = 0
    for k, n in enumerate(need):
        table[k, :n] = order[at:at + n]
        at += n

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    s = dict(case=dict(c), table=table, lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    if c["op"] == "select":
        # keys of one page resemble one another: a direction of the page's own, and noise
        parts = []
        for a in range(0, total, 512):
            n = min(512, total - a)
            k = normal(n, 1, c["hkv"], c["dim"]) + 0.7 * normal(n, p, c["hkv"], c["dim"])
            parts.append(torch.stack((k.amin(1), k.amax(1)), 2).to(dt))
        s["summary"] = torch.cat(parts)
    else:
        pool = (total, p, c["hkv"], c["dim"])
        s["k_pages"], s["v_pages"] = normal(*pool).to(dt), normal(*pool).to(dt)
    if c["op"] == "append":
        news = _news(c)
        t = sum(news)
        s["summary"] = torch.stack((s["k_pages"].amin(1), s["k_pages"].amax(1)), 2).contiguous()
        s["q"], s["k"], s["v"] = (normal(t, h, c["dim"]).to(dt) for h in (c["hq"], c["hkv"], c["hkv"]))
        cu = [0]
        for n in news:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["q_out"] = torch.empty_like(s["q"])
    else:
        s["q"] = normal(b, c["hq"], c["dim"]).to(dt)
    if c["op"] == "decode":
        s["lse"] = torch.empty(b, c["hq"], dtype=torch.float32, device=dev)
        if c["select"]:
            # as a selection gives them: ascending, the last page among them, -1 behind
            n = c["select"]
            pages = torch.full((b, c["hkv"], n), -1, dtype=torch.int32, device=dev)
            for k, m in enumerate(need):
                if m <= n:
                    pages[k, :, :m] = torch.arange(m, dtype=torch.int32, device=dev)
                else:
                    r = torch.rand(c["hkv"], m, generator=g, device=dev)
                    r[:, m - 1] = 2.0
                    pages[k] = r.topk(n, dim=1).indices.sort(dim=1).values.to(torch.int32)
            s["pages"] = pages
    return s


# -------------------------------------------------------------- plain form
def _turned(x, angle):
    """Half-split rotation of x by angle (64 bits): pairs (x_k, x_{k + D/2})."""
    co, si = angle.cos().float(), angle.sin().float()
    a, b = x.chunk(2, dim=-1)
    return torch.cat((a * co - b * si, b * co + a * si), dim=-1)


def _freq(c, device):
    k = torch.arange(c["dim"] // 2, dtype=torch.float64, device=device)
    return torch.pow(torch.tensor(c["theta"], dtype=torch.float64, device=device), -2.0 * k / c["dim"])


def _group(c, lens):
    return ((lens.long() + c["w_pre"] - 1) // c["w_pre"]).clamp(min=1)


def _plain_append(s):
    c = s["case"]
    cu, lens, p = s["cu"].long(), s["lens"].long(), c["page"]
    t = torch.arange(s["k"].shape[0], device=cu.device)
    b = (t[:, None] >= cu[None, 1:]).sum(1)
    pos = lens[b] - (cu[b + 1] - cu[b]) + t - cu[b]
    angle = (pos.double()[:, None] * _freq(c, cu.device))[:, None, :]
    dt = s["k"].dtype
    k = _turned(s["k"].float(), angle).to(dt)
    s["q_out"].copy_(_turned(s["q"].float(), angle))
    page = s["table"][b, pos // p].long()
    s["k_pages"][page, pos % p] = k
    s["v_pages"][page, pos % p] = s["v"]
    n = s["k_pages"].shape[0]
    inf = float("inf")
    lo = torch.full((n,) + k.shape[1:], inf, device=k.device).index_reduce_(0, page, k.float(), "amin")
    hi = torch.full((n,) + k.shape[1:], -inf, device=k.device).index_reduce_(0, page, k.float(), "amax")
    # a page whose first token is among the new ones starts afresh, any other keeps what it had
    fresh = torch.zeros(n, dtype=torch.bool, device=k.device)
    fresh[page[pos % p == 0]] = True
    hit = torch.zeros(n, dtype=torch.bool, device=k.device)
    hit[page] = True
    old = s["summary"].float()
    keep = ~fresh[:, None, None]
    lo = torch.where(keep, torch.minimum(lo, old[:, :, 0]), lo)
    hi = torch.where(keep, torch.maximum(hi, old[:, :, 1]), hi)
    new = torch.where(hit[:, None, None, None], torch.stack((lo, hi), 2), old)
    s["summary"].copy_(new)
    return [s["k_pages"], s["v_pages"], s["summary"], s["q_out"]]


def _plain_select(s):
    c = s["case"]
    p, gs = c["page"], c["hq"] // c["hkv"]
    lens = s["lens"].long()
    table = s["table"].long()
    b, cols = table.shape
    idx = torch.arange(cols, device=lens.device)
    mid = idx * p + p // 2
    grp = _group(c, lens)[:, None]
    i = (lens - 1)[:, None]
    turn = torch.where(mid[None] < (lens - c["w0"])[:, None], (mid // grp - mid) - (i // grp - i), 0)
    angle = -turn.double()[:, :, None] * _freq(c, lens.device)                # [B, pages, D/2]
    co, si = angle.cos()[:, None, None], angle.sin()[:, None, None]
    qa, qb = s["q"].double().view(b, c["hkv"], gs, 1, c["dim"]).chunk(2, dim=-1)
    turned = torch.cat((qa * co - qb * si, qb * co + qa * si), dim=-1)        # [B, Hkv, GS, pages, D]
    key = s["summary"][table].double().permute(0, 2, 3, 1, 4)                 # [B, Hkv, 2, pages, D]
    score = torch.maximum(turned * key[:, :, 0:1], turned * key[:, :, 1:2]).sum(-1).amax(2)
    n = ((lens + p - 1) // p)[:, None]
    first, last = _forced(c)
    inf = float("inf")
    forced = (idx[None] < first) | (idx[None] >= n - last)
    score = torch.where(forced[:, None], inf, score)
    score = torch.where((idx[None] < n)[:, None], score, -inf)
    want = min(c["select"], cols)
    best = score.sort(dim=-1, descending=True, stable=True).indices[..., :want]
    best = torch.where(best < n[:, None], best, cols).sort(dim=-1).values
    out = torch.full((b, c["hkv"], c["select"]), -1, dtype=torch.int32, device=lens.device)
    out[..., :want] = torch.where(best < cols, best, -1)
    return out


def _plain_decode(s):
    c = s["case"]
    p, gs = c["page"], c["hq"] // c["hkv"]
    lens = s["lens"].long()
    table = s["table"].long()
    b, cols = table.shape
    dev = lens.device
    inside = torch.arange(p, device=dev)
    if c["select"]:
        pages = s["pages"].long()
        listed_ = (pages >= 0)[..., None]
        pos = (pages.clamp(min=0)[..., None] * p + inside).flatten(2)         # [B, Hkv, N]
        there = listed_.expand(-1, -1, -1, p).flatten(2)
    else:
        pos = torch.arange(cols * p, device=dev)[None, None]
        there = pos >= 0
    length = lens[:, None, None]
    there = there & (pos < length)
    if c["window"]:
        there = there & (pos >= length - c["window"])
    pos = pos.expand(b, pos.shape[1], pos.shape[2])
    row = table.gather(1, (pos // p).flatten(1)).view_as(pos) * p + pos % p
    head = torch.arange(c["hkv"], device=dev)[None, :, None]
    k = s["k_pages"].view(-1, c["hkv"], c["dim"])[row, head].float()          # [B, Hkv, N, D]
    v = s["v_pages"].view(-1, c["hkv"], c["dim"])[row, head].float()
    grp = _group(c, lens)[:, None, None]
    i = length - 1
    turn = torch.where(pos < length - c["w0"], (pos // grp - pos) - (i // grp - i), 0)
    k = _turned(k, turn.double()[..., None] * _freq(c, dev))
    q = s["q"].float().view(b, c["hkv"], gs, c["dim"])
    score = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(c["dim"])
    score = torch.where(there[:, :, None], score, float("-inf"))
    top = score.amax(-1, keepdim=True).clamp(min=-3.0e38)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    v = torch.where(there[..., None], v, 0.0)
    out = torch.matmul(e, v) / torch.where(total > 0, total, 1.0)
    s["lse"].copy_((top + torch.log(total)).view(b, c["hq"]))
    return [out.view(b, c["hq"], c["dim"]).to(s["q"].dtype), s["lse"]]


def _forced(c):
    """Pages that a list always holds: the first, and the newest."""
    return (1, 1) if c["select"] >= 2 else (0, 1)


# ---------------------------------------------------------------- the call
def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"append": _plain_append, "select": _plain_select, "decode": _plain_decode}[c["op"]](s)
    from zero_shot_rope_b200 import jetlong as jl

    if c["op"] == "append":
        jl.jl_paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["cu"], s["lens"], c["new"],
                           page_summary=s["summary"], q=s["q"], q_out=s["q_out"], rope_theta=c["theta"])
        return [s["k_pages"], s["v_pages"], s["summary"], s["q_out"]]
    if c["op"] == "select":
        first, last = _forced(c)
        return jl.jl_bifocal_select_pages(s["q"], s["summary"], s["table"], s["lens"], c["page"], c["select"],
                                          c["w_pre"], c["w0"], c["theta"], n_first=first, n_last=last)
    out, lse = jl.jl_bifocal_decode_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], c["w_pre"],
                                          c["w0"], c["theta"], page_list=s.get("pages"), window=c["window"],
                                          lse=s["lse"])
    return [out, lse]


# ------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """From the definitions, sequence by sequence, rotations as products of
    complex numbers."""
    s = prepare(case, seed)
    c = case
    p, half = c["page"], c["dim"] // 2
    dev = s["q"].device
    freq = float(c["theta"]) ** (-2.0 * torch.arange(half, dtype=torch.float64, device=dev) / c["dim"])

    def whirl(x, by):  # x [..., D], by: positions, broadcast over x's leading dimensions
        z = torch.complex(x[..., :half], x[..., half:]) * torch.polar(torch.ones_like(by * freq), by * freq)
        return torch.cat((z.real, z.imag), dim=-1)

    lens = _lengths(c)
    if c["op"] == "append":
        kp, vp, sm = s["k_pages"].double(), s["v_pages"].double(), s["summary"].double()
        qo = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
        at = 0
        for b, (length, n) in enumerate(zip(lens, _news(c))):
            pos = torch.arange(length - n, length, device=dev)
            by = pos.double()[:, None, None]
            k = whirl(s["k"][at:at + n].double(), by)
            qo[at:at + n] = whirl(s["q"][at:at + n].double(), by)
            page = s["table"][b, pos // p].long()
            kp[page, pos % p] = k
            vp[page, pos % p] = s["v"][at:at + n].double()
            for a in range((length - n) // p, (length - 1) // p + 1):
                lo, hi = max(a * p, length - n) - (length - n), min((a + 1) * p, length) - (length - n)
                ends = torch.stack((k[lo:hi].amin(0), k[lo:hi].amax(0)), 1)
                one = int(s["table"][b, a])
                if a * p < length - n:
                    ends = torch.stack((torch.minimum(ends[:, 0], sm[one, :, 0]), torch.maximum(ends[:, 1], sm[one, :, 1])), 1)
                sm[one] = ends
            at += n
        return [kp, vp, sm, qo]
    gs = c["hq"] // c["hkv"]
    if c["op"] == "select":
        out = torch.full((c["batch"], c["hkv"], c["select"]), -1, dtype=torch.int32, device=dev)
        first, last = _forced(c)
        for b, length in enumerate(lens):
            n = _pages_of(c, length)
            if n <= c["select"]:
                out[b, :, :n] = torch.arange(n, dtype=torch.int32, device=dev)
                continue
            g = max(1, -(-length // c["w_pre"]))
            mid = torch.arange(n, device=dev) * p + p // 2
            by = ((length - 1) // g - (length - 1)) - (mid // g - mid)
            by = torch.where(mid < length - c["w0"], by, 0).double()
            ends = s["summary"][s["table"][b, :n].long()].double()            # [n, Hkv, 2, D]
            q = whirl(s["q"][b].double()[None], by[:, None, None]).view(n, c["hkv"], gs, c["dim"])
            side = torch.where(q > 0, ends[:, :, 1:2], ends[:, :, 0:1])
            score = (q * side).sum(-1).amax(-1)                               # [n, Hkv]
            score[:first] = float("inf")
            score[n - last:] = float("inf")
            best = torch.argsort(-score, dim=0, stable=True)[:c["select"]]
            out[b] = best.sort(dim=0).values.t().to(torch.int32)
        return out
    outs, lses = [], []
    for b, length in enumerate(lens):
        g = max(1, -(-length // c["w_pre"]))
        i = length - 1
        for h in range(c["hkv"]):
            if c["select"]:
                pages = s["pages"][b, h]
                pages = pages[pages >= 0].long()
                pos = (pages[:, None] * p + torch.arange(p, device=dev)).flatten()
            else:
                pos = torch.arange(length, device=dev)
            pos = pos[(pos < length) & ((pos >= length - c["window"]) | (c["window"] == 0))]
            page = s["table"][b, pos // p].long()
            k = s["k_pages"][page, pos % p, h].double()
            v = s["v_pages"][page, pos % p, h].double()
            q = s["q"][b, h * gs:(h + 1) * gs].double()
            near = q @ k.t()
            far = whirl(q, torch.tensor(float(i // g - i), device=dev)) @ whirl(k, (pos // g - pos).double()[:, None]).t()
            score = torch.where(pos < length - c["w0"], far, near) / math.sqrt(c["dim"])
            lses.append(torch.logsumexp(score, dim=1))
            outs.append(torch.softmax(score, dim=1) @ v)
    return [torch.cat(outs).view(c["batch"], c["hq"], c["dim"]), torch.cat(lses).view(c["batch"], c["hq"])]
