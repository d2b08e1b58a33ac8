"""Operators measured on the GPU: the normed and rotated append into a paged
cache, and the attention of new tokens over that cache (full or sliding window
with sinks; chunks, prompts and single tokens).

`run` computes them in a plain torch form, or through the package's calls when
`own` is set; `exact` computes them in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
THETA = 1.0e7


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One decode step's new tokens of 8 requests, 24 query / 4 KV heads of 256,
        # a quarter of the head rotated, appended as int8 rows: a latency call.
        dict(name="append 8 int8", op="append", n=8, Hq=24, Hkv=4, d=256, rot=64, inter=False, kv="int8",
             far=250000, fused=True, pad=0),
        # A prefill chunk of 2048 tokens, 16 / 2 heads of 256, whole head rotated, bf16 rows.
        dict(name="append 2048 bf16", op="append", n=2048, Hq=16, Hkv=2, d=256, rot=256, inter=False, kv="bf16",
             far=1048576, fused=True, pad=0),
        # An odd chunk of head dimension 128 with neighbouring pairs rotated, separate
        # projections, some padding tokens that own no cache row.
        dict(name="append 5237 odd bf16", op="append", n=5237, Hq=32, Hkv=8, d=128, rot=96, inter=True, kv="bf16",
             far=131072, fused=False, pad=37),
        # A long prompt appended at once, int8 rows.
        dict(name="append 32768 int8", op="append", n=32768, Hq=24, Hkv=4, d=256, rot=64, inter=False, kv="int8",
             far=250000, fused=True, pad=0),
        # Decode, one token of each of 8 requests in a layer with a window of 1024 and
        # 64 sinks, contexts of 250K: the smallest attention call.
        dict(name="decode window int8", op="attend", B=8, n=1, T=250000, ragged=False, Hq=24, Hkv=4, d=256, kv="int8",
             page=64, S=64, W=1024, lens=1),
        # Decode of 4 requests over a full 128K cache: the bandwidth case.
        dict(name="decode 4x131072 bf16", op="attend", B=4, n=1, T=131072, ragged=False, Hq=16, Hkv=2, d=256,
             kv="bf16", page=64, S=0, W=0, lens=2),
        # Decode of a serving batch whose contexts run from a token to 20K, int8 rows.
        dict(name="decode 64 ragged int8", op="attend", B=64, n=1, T=20000, ragged=True, Hq=24, Hkv=4, d=256,
             kv="int8", page=16, S=0, W=0, lens=3),
        # Checking a handful of drafted tokens for each of 16 requests, head dimension 128.
        dict(name="verify 16x5 ragged bf16", op="attend", B=16, n=5, T=30011, ragged=True, Hq=32, Hkv=8, d=128,
             kv="bf16", page=32, S=0, W=0, lens=4),
        # Prompts from one token to 4096, each from its start, head dimension 128.
        dict(name="prompts 6x4096 ragged bf16", op="attend", B=6, n=4096, T=4096, ragged=True, Hq=32, Hkv=8, d=128,
             kv="bf16", page=16, S=0, W=0, lens=5),
        # A prefill chunk in a window layer, int8 rows, odd sizes.
        dict(name="chunk 4001 window int8", op="attend", B=1, n=4001, T=20011, ragged=False, Hq=24, Hkv=4, d=256,
             kv="int8", page=64, S=64, W=1024, lens=6),
        # A short chunk late in a long context.
        dict(name="chunk 256 at 262144 bf16", op="attend", B=1, n=256, T=262144, ragged=False, Hq=16, Hkv=2, d=256,
             kv="bf16", page=64, S=0, W=0, lens=7),
        # A full prefill chunk: the largest call, tensor-core bound.
        dict(name="chunk 2048 at 65536 bf16", op="attend", B=1, n=2048, T=65536, ragged=False, Hq=16, Hkv=2, d=256,
             kv="bf16", page=64, S=0, W=0, lens=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 3, 4, 6, 8])
    d = rng.choice([128, 256])
    kv = rng.choice(["bf16", "int8"])
    if rng.random() < 0.4:
        n = _log(rng, 1, 30000)
        return dict(op="append", n=n, Hq=Hq, Hkv=Hkv, d=d, rot=16 * rng.randint(1, d // 16), inter=rng.random() < 0.5,
                    kv=kv, far=_log(rng, 64, 1 << 20) + n, fused=rng.random() < 0.5,
                    pad=rng.randint(0, n // 8) if rng.random() < 0.5 else 0)
    window = rng.random() < 0.5
    S, W = (rng.choice([0, 4, 64, 100]), _log(rng, 16, 4096)) if window else (0, 0)
    form = rng.choice(["decode", "few", "chunk"])
    B = _log(rng, 1, 64) if form == "decode" else _log(rng, 1, 16) if form == "few" else rng.choice([1, 1, 2, 4])
    n = 1 if form == "decode" else rng.randint(2, 16) if form == "few" else _log(rng, 17, 4096)
    # The plain form's score matrix stays below 2^30 values, and the cache below 2^30.
    top = min(262144, (1 << 30) // (B * n * Hq), (1 << 30) // (B * Hkv * d))
    T = _log(rng, n, max(n, top))
    return dict(op="attend", B=B, n=n, T=T, ragged=rng.random() < 0.5, Hq=Hq, Hkv=Hkv, d=d, kv=kv,
                page=rng.choice([8, 16, 32, 48, 64, 128, 256]), S=S, W=W, lens=rng.randint(10, 1 << 20))


def _lengths(case):
    """(tokens in the cache, new tokens among them) of each request."""
    B, n, T = case["B"], case["n"], case["T"]
    if not case["ragged"]:
        return [T] * B, [min(n, T)] * B
    rng = random.Random(case["lens"])
    lens = [T] + [max(1, _log(rng, 1, T)) for _ in range(B - 1)]
    new = [min(n, t) for t in lens]
    both = list(zip(lens, new))
    rng.shuffle(both)
    return [t for t, _ in both], [m for _, m in both]


def _visible(T, n, S, W):
    """How many (query, key) pairs the mask leaves, and how many keys some query sees."""
    p = np.arange(T - n, T, dtype=np.int64)
    if W == 0:
        return int((p + 1).sum()), T
    first = np.maximum(p - W + 1, 0)
    pairs = (p + 1 - first) + np.minimum(first, S)
    lo = int(first[0])
    return int(pairs.sum()), T - lo + min(lo, S)


def work(case):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    row = 2 * d if case["kv"] == "bf16" else d + 2
    if case["op"] == "append":
        n, m = case["n"], case["n"] - case["pad"]
        rd = n * (Hq * d * 2 + 4 + 8) + m * 2 * Hkv * d * 2 + 2 * d * 4 + case["rot"] * 2
        return {"bytes": rd + n * Hq * d * 2 + m * 2 * Hkv * row, "flops": 10 * n * (Hq + Hkv) * d}
    lens, new = _lengths(case)
    pairs = keys = 0
    for t, m in zip(lens, new):
        a, b = _visible(t, m, case["S"], case["W"])
        pairs, keys = pairs + a, keys + b
    return {"bytes": 2 * sum(new) * Hq * d * 2 + keys * 2 * Hkv * row, "flops": 4 * pairs * Hq * d}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _int8_pool(g, rows, Hkv, d):
    codes = torch.randint(-127, 128, (rows, Hkv, d), generator=g, device="cuda", dtype=torch.int8)
    # codes uniform in +-127 have a standard deviation of 73.3: scales near 1/73 make unit rows
    scale = (torch.rand((rows, Hkv), generator=g, device="cuda") + 0.5) / 73.3
    return codes, scale.to(torch.float16)


def prepare(case, seed):
    return _prepare_append(case, seed) if case["op"] == "append" else _prepare_attend(case, seed)


def _prepare_append(c, seed):
    g = _gen(seed)
    n, Hq, Hkv, d = c["n"], c["Hq"], c["Hkv"], c["d"]
    if c["fused"]:  # views of one projection's output
        x = _randn(g, (n, Hq + 2 * Hkv, d), 1.7)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    else:
        q, k, v = _randn(g, (n, Hq, d), 1.7), _randn(g, (n, Hkv, d), 0.6), _randn(g, (n, Hkv, d))
    rows = n + 64
    out_rows = torch.randperm(rows, generator=g, device="cuda")[:n]
    if c["pad"]:
        out_rows[torch.randperm(n, generator=g, device="cuda")[:c["pad"]]] = -1
    int8 = c["kv"] == "int8"
    dt = torch.int8 if int8 else torch.bfloat16
    return dict(
        c=c, q=q, k=k, v=v, out_rows=out_rows,
        qw=1 + 0.3 * torch.randn((d,), generator=g, device="cuda"),
        kw=1 + 0.3 * torch.randn((d,), generator=g, device="cuda"),
        pos=torch.randint(0, c["far"], (n,), generator=g, device="cuda", dtype=torch.int32),
        inv_freq=(THETA ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])).float().cuda(),
        q_out=torch.zeros((n, Hq, d), dtype=torch.bfloat16, device="cuda"),
        pool=torch.zeros((2, rows, Hkv, d), dtype=dt, device="cuda"),  # K rows, V rows
        scale=torch.zeros((2, rows, Hkv), dtype=torch.float16, device="cuda") if int8 else [None, None],
        status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _prepare_attend(c, seed):
    g = _gen(seed)
    Hq, Hkv, d, page = c["Hq"], c["Hkv"], c["d"], c["page"]
    lens, new = _lengths(c)
    n_pages = -(-max(lens) // page)
    blocks = sum(-(-t // page) for t in lens)
    perm = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.full((c["B"], n_pages), -1, dtype=torch.int32)
    at = 0
    for b, t in enumerate(lens):
        m = -(-t // page)
        table[b, :m] = perm[at:at + m]
        at += m
    rows = blocks * page
    if c["kv"] == "int8":
        (k, ks), (v, vs) = _int8_pool(g, rows, Hkv, d), _int8_pool(g, rows, Hkv, d)
    else:
        k, v, ks, vs = _randn(g, (rows, Hkv, d)), _randn(g, (rows, Hkv, d)), None, None
    starts = [0]
    for m in new:
        starts.append(starts[-1] + m)
    n = starts[-1]
    st = dict(
        c=c, q=_randn(g, (n, Hq, d), 1.5), k=k, v=v, ks=ks, vs=vs, table=table.cuda(), lens=lens, new=new,
        lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"),
        q_start=None if c["n"] == 1 else torch.tensor(starts, dtype=torch.int32, device="cuda"),
        starts=torch.tensor(starts, dtype=torch.int64, device="cuda"),
        out=torch.zeros((n, Hq, d), dtype=torch.bfloat16, device="cuda"),
        status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    if s["c"]["op"] == "append":
        return _append_own(s) if own else _append_plain(s)
    return _attend_own(s) if own else _attend_plain(s)


def _append_out(s):
    """q and the K and V rows of the pool; int8 rows as the values they stand for."""
    if s["c"]["kv"] == "bf16":
        return {"q": s["q_out"], "kv": s["pool"]}
    return {"q": s["q_out"], "kv": s["pool"] * s["scale"][..., None]}


def _append_own(s):
    import sparse_kv_long_gb300 as skv
    c, (k_pool, v_pool), (k_scale, v_scale) = s["c"], s["pool"], s["scale"]
    skv.norm_rope_append(s["q"], s["k"], s["v"], s["pos"], s["inv_freq"], s["q_out"], k_pool, v_pool,
                         q_weight=s["qw"], k_weight=s["kw"], eps=EPS, interleaved=c["inter"],
                         kv_kind=skv.KV_INT8 if c["kv"] == "int8" else skv.KV_BF16, k_scale=k_scale,
                         v_scale=v_scale, out_rows=s["out_rows"], status=s["status"])
    return _append_out(s)


def _rotate(x, ang, inter):
    """x [n][H][rot] fp32, ang [n][rot/2] in 64 bits."""
    co, si = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    if inter:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * co - b * si, b * co + a * si), -1).flatten(-2)
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    return torch.cat((a * co - b * si, b * co + a * si), -1)


def _int8_rows(x):
    """bf16 rows -> codes and one fp16 scale per (row, head)."""
    x = x.float()
    scale = (x.abs().amax(-1) / 127).to(torch.float16)
    inv = scale.float()[..., None]
    codes = torch.where(inv > 0, torch.round(x / inv).clamp(-127, 127), torch.zeros_like(x))
    return codes.to(torch.int8), scale


def _append_plain(s):
    c = s["c"]
    rot = c["rot"]
    ang = s["pos"].double()[:, None] * s["inv_freq"].double()
    q, k = s["q"].float(), s["k"].float()
    q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + EPS) * s["qw"]
    k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + EPS) * s["kw"]
    q = torch.cat((_rotate(q[..., :rot], ang, c["inter"]), q[..., rot:]), -1)
    k = torch.cat((_rotate(k[..., :rot], ang, c["inter"]), k[..., rot:]), -1)
    s["q_out"].copy_(q)
    keep = s["out_rows"] >= 0
    rows = s["out_rows"][keep]
    kv = torch.stack((k.to(torch.bfloat16)[keep], s["v"][keep]))
    if c["kv"] == "bf16":
        s["pool"][:, rows] = kv
    else:
        s["pool"][:, rows], s["scale"][:, rows] = _int8_rows(kv)
    return _append_out(s)


_workspace = None  # one for all calls, as a user's program keeps it: it grows to the largest need


def _attend_own(s):
    global _workspace
    import sparse_kv_long_gb300 as skv
    c = s["c"]
    need = skv.paged_attend_workspace_size(c["B"], s["q"].shape[0], c["Hq"], c["Hkv"], c["d"])
    if _workspace is None or _workspace.numel() < need:
        _workspace = torch.zeros((need,), dtype=torch.uint8, device="cuda")
    skv.paged_attend(skv.KV_INT8 if c["kv"] == "int8" else skv.KV_BF16, s["q"], s["k"], s["v"], s["table"], c["page"],
                     s["lengths"], c["d"] ** -0.5, s["out"], _workspace, q_start=s["q_start"], S=c["S"], W=c["W"],
                     k_scale=s["ks"], v_scale=s["vs"], status=s["status"])
    return s["out"]


def _attend_plain(s):
    """The batch padded to its longest request: [B][Hkv][n * G][T] scores."""
    c = s["c"]
    B, Hq, Hkv, d, page = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"]
    G, T, n = Hq // Hkv, max(s["lens"]), max(s["new"])
    t = torch.arange(T, device="cuda")
    L = s["lengths"].long()
    rows = s["table"].long().clamp(min=0)[:, t // page] * page + t % page           # [B][T]
    k, v = s["k"][rows].float(), s["v"][rows].float()                               # [B][T][Hkv][d]
    if s["ks"] is not None:
        k, v = k * s["ks"][rows].float()[..., None], v * s["vs"][rows].float()[..., None]
    i = torch.arange(n, device="cuda")
    m = s["starts"][1:] - s["starts"][:-1]                                          # new tokens [B]
    own_q = i[None] < m[:, None]                                                    # [B][n]
    at = (s["starts"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][at].float().view(B, n, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, d)
    logit = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(d ** -0.5).view(B, Hkv, n, G, T)
    p = (L - m)[:, None] + i                                                        # position of each query
    see = (t <= p[..., None]) & own_q[..., None]
    if c["W"]:
        see &= (t > p[..., None] - c["W"]) | (t < c["S"])
    logit.masked_fill_(~see[:, None, :, None], -math.inf)
    top = logit.amax(-1, keepdim=True).clamp_(min=-3e38)
    w = logit.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.view(B, Hkv, n * G, T), v.transpose(1, 2)).view(B, Hkv, n, G, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.permute(0, 2, 1, 3, 4).reshape(B, n, Hq, d)
    s["out"].copy_(o[own_q])
    return s["out"]


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return _append_exact(s) if case["op"] == "append" else _attend_exact(s)


def _append_exact(s):
    c = s["c"]
    rot, pos, f = c["rot"], s["pos"].double(), s["inv_freq"].double()

    def normed(x, w):
        y = x.double()
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + EPS) * w.double()
        z = y[..., :rot]
        z = z.unflatten(-1, (rot // 2, 2)) if c["inter"] else z.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        z = torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones_like(f), pos[:, None] * f)[:, None]
        z = torch.view_as_real(z)
        z = z.flatten(-2) if c["inter"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat((z, y[..., rot:]), -1)

    def pool(*parts):  # the rows as the cache holds them
        full = torch.zeros(s["pool"].shape, dtype=torch.float64, device="cuda")
        keep = s["out_rows"] >= 0
        for half, x in zip(full, parts):
            half[s["out_rows"][keep]] = x[keep]
        return full

    q, k, v = normed(s["q"], s["qw"]), normed(s["k"], s["kw"]), s["v"].double()
    if c["kv"] == "bf16":
        return {"q": q, "kv": pool(k, v)}

    def int8(x):  # int8 rows hold the bf16 value's nearest multiple of the row's fp16 scale
        x = x.to(torch.bfloat16).double()
        scale = (x.abs().amax(-1, keepdim=True) / 127).to(torch.float16).double()
        return torch.where(scale > 0, torch.round(x / scale.clamp(min=1e-30)).clamp(-127, 127) * scale, 0.0)

    return {"q": q, "kv": pool(int8(k), int8(v))}


def _attend_exact(s):
    c = s["c"]
    Hq, Hkv, d, page = c["Hq"], c["Hkv"], c["d"], c["page"]
    G = Hq // Hkv
    if sum(t * m for t, m in zip(s["lens"], s["new"])) * Hq * d * 4 > 1.0e13:
        return None
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (T, m) in enumerate(zip(s["lens"], s["new"])):
        t = torch.arange(T, device="cuda")
        rows = s["table"][b].long()[t // page] * page + t % page
        pos = torch.arange(T - m, T, device="cuda")
        hidden = t[None] > pos[:, None]
        if c["W"]:
            hidden |= (t[None] <= pos[:, None] - c["W"]) & (t[None] >= c["S"])
        for h in range(Hkv):
            k, v = s["k"][rows, h].double(), s["v"][rows, h].double()
            if s["ks"] is not None:
                k, v = k * s["ks"][rows, h].double()[:, None], v * s["vs"][rows, h].double()[:, None]
            for g in range(h * G, h * G + G):
                z = s["q"][at:at + m, g].double() @ k.T / math.sqrt(d)
                out[at:at + m, g] = torch.softmax(z.masked_fill_(hidden, -math.inf), -1) @ v
        at += m
    return out
