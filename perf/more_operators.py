"""Operators measured on the GPU: the attention of a batch whose requests share
long prefixes, each prefix read once for all of them, and the moving of cached
rows between places, positions and encodings, of which such a prefix is made.

`run` computes them in a plain torch form, or through the package's calls when
`own` is set; `exact` computes them in 64 bits.
"""
import math
import random

import torch

own = False

THETA = 1.0e7


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # A decode step of 8 agents behind a short system prompt, a few turns of their own: a latency call.
        dict(name="agents 8 at 2000 int8", op="attend", B=8, groups=1, alone=0, n=1, P=2000, T=100, ragged=True,
             Hq=24, Hkv=4, d=256, kv="int8", page=64, lens=1),
        # The same agents over a source tree of 250K tokens: the bandwidth case.
        dict(name="agents 8 at 250000 int8", op="attend", B=8, groups=1, alone=0, n=1, P=250000, T=2000, ragged=True,
             Hq=24, Hkv=4, d=256, kv="int8", page=64, lens=2),
        # 64 samples drawn from one long prompt.
        dict(name="samples 64 at 131072 bf16", op="attend", B=64, groups=1, alone=0, n=1, P=131072, T=1000,
             ragged=True, Hq=16, Hkv=2, d=256, kv="bf16", page=64, lens=3),
        # A serving batch: five prompts of odd lengths shared by a few requests each, three requests that share
        # none, head dimension 128.
        dict(name="groups 5 of 40 ragged bf16", op="attend", B=40, groups=5, alone=3, n=1, P=30011, T=5000, ragged=True,
             Hq=32, Hkv=8, d=128, kv="bf16", page=16, lens=4),
        # Checking five drafted tokens of each of 16 requests behind one prompt.
        dict(name="drafts 16x5 at 60000 int8", op="attend", B=16, groups=1, alone=0, n=5, P=60000, T=400, ragged=True,
             Hq=32, Hkv=8, d=128, kv="int8", page=32, lens=5),
        # Questions of odd lengths about two documents, read for the first time.
        dict(name="questions 5x333 at 20011 int8", op="attend", B=5, groups=2, alone=0, n=333, P=20011, T=333,
             ragged=True, Hq=24, Hkv=4, d=256, kv="int8", page=64, lens=6),
        # 16 prompts that differ in their last 256 tokens: the largest call, tensor-core bound.
        dict(name="prompts 16x256 at 32768 bf16", op="attend", B=16, groups=1, alone=0, n=256, P=32768, T=256,
             ragged=False, Hq=16, Hkv=2, d=256, kv="bf16", page=64, lens=7),
        # One page's keys at other positions: a latency call.
        dict(name="move 64 keys int8", op="move", n=64, Hkv=4, d=256, rot=64, inter=False, src="int8", dst="int8",
             values=False, far=250000, pad=0, scaled=False),
        # Rows of an odd prompt moved behind another one, neighbouring pairs rotated, some tokens left out.
        dict(name="move 5237 odd bf16", op="move", n=5237, Hkv=2, d=256, rot=96, inter=True, src="bf16", dst="bf16",
             values=True, far=131072, pad=37, scaled=False),
        # A document cached as bf16 rows made part of an int8 prefix, head dimension 128.
        dict(name="move 8192 bf16 to int8", op="move", n=8192, Hkv=8, d=128, rot=128, inter=False, src="bf16",
             dst="int8", values=True, far=1048576, pad=0, scaled=False),
        # A long int8 document at another position.
        dict(name="move 32768 int8", op="move", n=32768, Hkv=4, d=256, rot=64, inter=False, src="int8", dst="int8",
             values=True, far=250000, pad=0, scaled=False),
        # A prefix kept as int4 rows brought back as int8, its keys at the frequencies of a longer context.
        dict(name="move 65536 int4 to int8", op="move", n=65536, Hkv=4, d=256, rot=64, inter=False, src="int4",
             dst="int8", values=True, far=250000, pad=0, scaled=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    Hkv = rng.choice([1, 2, 4, 8])
    if rng.random() < 0.4:
        src, dst = rng.choice(["bf16", "int8", "int4"]), rng.choice(["bf16", "int8", "int4"])
        d = 256 if "int4" in (src, dst) else rng.choice([64, 128, 256])
        n = _log(rng, 1, 65536 // Hkv * 2)
        return dict(op="move", n=n, Hkv=Hkv, d=d, rot=16 * rng.randint(0, d // 16), inter=rng.random() < 0.5, src=src,
                    dst=dst, values=rng.random() < 0.7, far=_log(rng, 64, 1 << 20) + n,
                    pad=rng.randint(0, n // 8) if rng.random() < 0.5 else 0, scaled=rng.random() < 0.5)
    Hq = Hkv * rng.choice([1, 3, 4, 6, 8])
    d = rng.choice([128, 256])
    form = rng.choice(["decode", "decode", "few", "chunk"])
    B = _log(rng, 2, 64) if form == "decode" else rng.randint(2, 16)
    n = 1 if form == "decode" else rng.randint(2, 8) if form == "few" else _log(rng, 9, 333)
    groups = rng.choice([1, 1, 2, 3, 5])
    groups = min(groups, B)
    alone = rng.randint(0, B - groups) if rng.random() < 0.3 else 0
    # The plain form's score matrix stays below 2^30 values, and the cache below 2^30.
    top = min(262144, (1 << 30) // (B * n * Hq), (1 << 29) // (groups * Hkv * d))
    return dict(op="attend", B=B, groups=groups, alone=alone, n=n, P=_log(rng, 1, top),
                T=_log(rng, n, max(n, min(8192, top))), ragged=rng.random() < 0.7, Hq=Hq, Hkv=Hkv, d=d,
                kv=rng.choice(["bf16", "int8"]), page=rng.choice([8, 16, 32, 48, 64, 128]), lens=rng.randint(10, 1 << 20))


def _batch(case):
    """(first request of each group and the end of the last, prefix length of each group, own cached tokens of each
    request, new ones among them); the last `alone` requests are in no group."""
    B, groups, n, T, P = case["B"], case["groups"], case["n"], case["T"], case["P"]
    m = B - case["alone"]
    if not case["ragged"]:
        return [m * g // groups for g in range(groups + 1)], [P] * groups, [T] * B, [min(n, T)] * B
    rng = random.Random(case["lens"])
    start = [0] + sorted(rng.sample(range(1, m), groups - 1)) + [m]
    prefix = [P] + [_log(rng, 1, P) for _ in range(groups - 1)]
    rng.shuffle(prefix)
    lens = [T] + [_log(rng, 1, T) for _ in range(B - 1)]
    rng.shuffle(lens)
    return start, prefix, lens, [min(n, t) for t in lens]


def _row_bytes(kv, d):
    return {"bf16": 2 * d, "int8": d + 2, "int4": d // 2 + d // 32}[kv]


def work(case):
    Hkv, d = case["Hkv"], case["d"]
    if case["op"] == "move":
        m, kinds = case["n"] - case["pad"], 2 if case["values"] else 1
        rows = m * kinds * Hkv * (_row_bytes(case["src"], d) + _row_bytes(case["dst"], d))
        if case["dst"] == "int4":  # and read back as bf16
            rows += m * kinds * Hkv * (_row_bytes("int4", d) + 2 * d)
        return {"bytes": rows + case["n"] * 24 + 4 * case["rot"], "flops": 6 * m * kinds * Hkv * d}
    Hq = case["Hq"]
    start, prefix, lens, new = _batch(case)
    pairs = sum(t * m - m * (m - 1) // 2 for t, m in zip(lens, new))
    pairs += sum(p * sum(new[a:b]) for p, a, b in zip(prefix, start, start[1:]))
    rows = sum(prefix) + sum(lens)
    return {"bytes": 4 * sum(new) * Hq * d + rows * 2 * Hkv * _row_bytes(case["kv"], d), "flops": 4 * pairs * Hq * d}


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


def _int4_tier(g, rows, Hkv, d):
    """Host-tier rows [rows][Hkv][K, V][d / 2 bytes of codes, d / 64 fp16 scales]."""
    codes = torch.randint(-7, 8, (rows, Hkv, 2, d // 2, 2), generator=g, device="cuda", dtype=torch.int8)
    codes = ((codes[..., 0] & 15) | (codes[..., 1] << 4)).view(torch.uint8)
    scale = ((torch.rand((rows, Hkv, 2, d // 64), generator=g, device="cuda") + 0.5) / 4.3).to(torch.float16)
    return torch.cat((codes, scale.view(torch.uint8)), -1)


def prepare(case, seed):
    return _prepare_move(case, seed) if case["op"] == "move" else _prepare_attend(case, seed)


def _pages(lens, page, perm, at):
    """A block table [len(lens)][pages of the longest]; unused entries -1."""
    table = torch.full((len(lens), max(1, -(-max(lens) // page))), -1, dtype=torch.int32)
    for b, t in enumerate(lens):
        m = -(-t // page)
        table[b, :m] = perm[at:at + m]
        at += m
    return table.cuda(), at


def _prepare_attend(c, seed):
    g = _gen(seed)
    Hq, Hkv, d, page = c["Hq"], c["Hkv"], c["d"], c["page"]
    start, prefix, lens, new = _batch(c)
    blocks = sum(-(-t // page) for t in prefix + lens)
    perm = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32).cpu()
    prefix_table, at = _pages(prefix, page, perm, 0)
    table, _ = _pages(lens, page, perm, at)
    rows = blocks * page
    if c["kv"] == "int8":
        (k, ks), (v, vs) = _int8_pool(g, rows, Hkv, d), _int8_pool(g, rows, Hkv, d)
    else:
        k, v, ks, vs = _randn(g, (rows, Hkv, d)), _randn(g, (rows, Hkv, d)), None, None
    starts = [0]
    for m in new:
        starts.append(starts[-1] + m)
    n = starts[-1]

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    return dict(c=c, q=_randn(g, (n, Hq, d), 1.5), k=k, v=v, ks=ks, vs=vs, start=start, prefix=prefix, lens=lens,
                new=new, starts=starts, prefix_table=prefix_table, table=table, group_start=i32(start),
                prefix_lengths=i32(prefix), lengths=i32(lens), q_start=None if c["n"] == 1 else i32(starts),
                out=torch.zeros((n, Hq, d), dtype=torch.bfloat16, device="cuda"),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _empty(kv, rows, Hkv, d):
    """(K rows, V rows, K scales, V scales), or the int4 tier that holds them all."""
    if kv == "int4":
        return torch.zeros((rows, Hkv, 2, d // 2 + d // 32), dtype=torch.uint8, device="cuda")
    pool = torch.zeros((2, rows, Hkv, d), dtype=torch.int8 if kv == "int8" else torch.bfloat16, device="cuda")
    scale = torch.zeros((2, rows, Hkv), dtype=torch.float16, device="cuda") if kv == "int8" else (None, None)
    return pool, scale


def _prepare_move(c, seed):
    g = _gen(seed)
    n, Hkv, d, rot = c["n"], c["Hkv"], c["d"], c["rot"]
    rows = n + 64
    if c["src"] == "int4":
        src = _int4_tier(g, rows, Hkv, d)
    elif c["src"] == "int8":
        both = _int8_pool(g, 2 * rows, Hkv, d)
        src = both[0].view(2, rows, Hkv, d), both[1].view(2, rows, Hkv)
    else:
        src = _randn(g, (2, rows, Hkv, d)), (None, None)
    dst_rows = torch.randperm(rows, generator=g, device="cuda")[:n]
    if c["pad"]:
        dst_rows[torch.randperm(n, generator=g, device="cuda")[:c["pad"]]] = -1
    old = torch.arange(n, device="cuda", dtype=torch.int32)
    shift = int(torch.randint(1, c["far"] - n + 2, (1,), generator=g, device="cuda"))
    freq = THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    # frequencies of a context four times as long: the slowest a quarter, the fastest as they were
    slow = freq / (1 + 3 * torch.linspace(0, 1, rot // 2, dtype=torch.float64)) if c["scaled"] else freq
    return dict(c=c, src=src, dst=_empty(c["dst"], rows, Hkv, d),
                back=_empty("bf16", rows, Hkv, d) if c["dst"] == "int4" else None,
                src_rows=torch.randperm(rows, generator=g, device="cuda")[:n], dst_rows=dst_rows, old=old,
                new=old + shift, old_freq=freq.float().cuda(), new_freq=slow.float().cuda(),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    if s["c"]["op"] == "move":
        return _move_own(s) if own else _move_plain(s)
    return _attend_own(s) if own else _attend_plain(s)


_workspace = None  # one for all calls, as a user's program keeps it: it grows to the largest need


def _attend_own(s):
    global _workspace
    import sparse_kv_long_gb300 as skv
    c = s["c"]
    need = skv.shared_attend_workspace_size(c["B"], c["groups"], s["q"].shape[0], c["Hq"], c["Hkv"], c["d"])
    if _workspace is None or _workspace.numel() < need:
        _workspace = torch.zeros((need,), dtype=torch.uint8, device="cuda")
    skv.shared_attend(skv.KV_INT8 if c["kv"] == "int8" else skv.KV_BF16, s["q"], s["k"], s["v"], s["group_start"],
                      s["prefix_table"], s["prefix_lengths"], s["table"], c["page"], s["lengths"], c["d"] ** -0.5,
                      s["out"], _workspace, q_start=s["q_start"], k_scale=s["ks"], v_scale=s["vs"], status=s["status"])
    return s["out"]


def _keys(s, table, n, dtype):
    """K and V of the first n tokens of a table's row (or of all its rows)."""
    t = torch.arange(n, device="cuda")
    rows = table.long().clamp(min=0)[..., t // s["c"]["page"]] * s["c"]["page"] + t % s["c"]["page"]
    k, v = s["k"][rows].to(dtype), s["v"][rows].to(dtype)
    if s["ks"] is not None:
        k, v = k * s["ks"][rows].to(dtype)[..., None], v * s["vs"][rows].to(dtype)[..., None]
    return k, v


def _attend_plain(s):
    """Both parts in 32 bits with their maxima and sums: the prefixes group by group, the requests' own keys as a batch
    padded to its longest request."""
    c = s["c"]
    Hq, Hkv, d, B = c["Hq"], c["Hkv"], c["d"], c["B"]
    G, N = Hq // Hkv, s["q"].shape[0]
    q = s["q"].float().view(N, Hkv, G, d) * d ** -0.5
    n, T = max(s["new"]), max(s["lens"])
    k, v = _keys(s, s["table"], T, torch.float32)                                   # [B][T][Hkv][d]
    starts = torch.tensor(s["starts"], device="cuda")
    m = (starts[1:] - starts[:-1])[:, None]
    i, t = torch.arange(n, device="cuda"), torch.arange(T, device="cuda")
    mine = i < m                                                                    # [B][n]
    qb = q[(starts[:-1, None] + i).clamp(max=N - 1)].permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, d)
    logit = torch.matmul(qb, k.permute(0, 2, 3, 1)).view(B, Hkv, n, G, T)
    see = (t <= (s["lengths"].long()[:, None] - m + i)[..., None]) & mine[..., None]
    logit.masked_fill_(~see[:, None, :, None], -math.inf)
    top = logit.amax(-1, keepdim=True).clamp_(min=-3e38)
    w = logit.sub_(top).exp_()
    o = torch.matmul(w.view(B, Hkv, n * G, T), v.transpose(1, 2)).view(B, Hkv, n, G, d)

    def by_token(x):
        return x.permute(0, 2, 1, 3, 4)[mine]                                       # [N][Hkv][G][..]

    top, total, o = by_token(top), by_token(w.sum(-1, keepdim=True)), by_token(o)
    del logit, w
    for g, P in enumerate(s["prefix"]):
        a, b = s["starts"][s["start"][g]], s["starts"][s["start"][g + 1]]
        k, v = _keys(s, s["prefix_table"][g], P, torch.float32)                     # [P][Hkv][d]
        qg = q[a:b].permute(1, 0, 2, 3).reshape(Hkv, (b - a) * G, d)
        w = torch.matmul(qg, k.permute(1, 2, 0))
        ptop = w.amax(-1, keepdim=True)
        w.sub_(ptop).exp_()

        def rows(x):
            return x.view(Hkv, b - a, G, -1).permute(1, 0, 2, 3)

        po, psum, ptop = rows(torch.matmul(w, v.transpose(0, 1))), rows(w.sum(-1, keepdim=True)), rows(ptop)
        both = torch.maximum(ptop, top[a:b])
        fp, fo = (ptop - both).exp(), (top[a:b] - both).exp()
        o[a:b], total[a:b] = po * fp + o[a:b] * fo, psum * fp + total[a:b] * fo
    s["out"].copy_((o / total).view(N, Hq, d))
    return s["out"]


def _move_own(s):
    import sparse_kv_long_gb300 as skv
    c = s["c"]
    kinds = {"bf16": skv.KV_BF16, "int8": skv.KV_INT8}

    def rows(kv, x):
        if kv == "int4":
            return skv.tier_rows(x, values=c["values"])
        (k, v), (ks, vs) = x
        return skv.row_set(kinds[kv], k, v if c["values"] else None, ks, vs if c["values"] else None)

    dst = rows(c["dst"], s["dst"])
    skv.move_rows(rows(c["src"], s["src"]), dst, c["n"], src_rows=s["src_rows"], dst_rows=s["dst_rows"],
                  old_positions=s["old"], old_inv_freq=s["old_freq"], new_positions=s["new"],
                  new_inv_freq=s["new_freq"], interleaved=c["inter"], status=s["status"])
    if c["dst"] == "int4":
        skv.move_rows(dst, rows("bf16", s["back"]), c["n"], src_rows=s["dst_rows"], dst_rows=s["dst_rows"],
                      status=s["status"])
    return _move_out(s)


def _move_out(s):
    """The destination's rows; int8 rows as the values they stand for, int4 rows as read back."""
    c = s["c"]
    pool, scale = s["back"] if c["dst"] == "int4" else s["dst"]
    m = 2 if c["values"] else 1
    return pool[:m] if c["dst"] != "int8" else pool[:m] * scale[:m, ..., None]


def _decode(c, src, rows, dtype):
    """K and V of some rows, [2][n][Hkv][d]."""
    if c["src"] == "int4":
        x, half = src[rows].permute(2, 0, 1, 3), c["d"] // 2
        b = x[..., :half].view(torch.int8)
        codes = torch.stack(((b << 4) >> 4, b >> 4), -1).flatten(-2).to(dtype)
        scale = x[..., half:].contiguous().view(torch.float16).to(dtype)
        return (codes.unflatten(-1, (-1, 64)) * scale[..., None]).flatten(-2)
    x, scale = src
    x = x[:, rows].to(dtype)
    return x if c["src"] == "bf16" else x * scale[:, rows].to(dtype)[..., None]


def _codes(x, top):
    """x [..][values of one scale] -> rounded codes (as x's type) and fp16 scales."""
    scale = (x.abs().amax(-1, keepdim=True) / top).to(torch.float16)
    s = scale.to(x.dtype)
    lowest = -8 if top == 7 else -top
    return torch.where(s > 0, torch.round(x / s.clamp(min=1e-30)).clamp(lowest, top), torch.zeros_like(x)), scale


def _as_they_are(c):
    """Which of K and V are copied, codes and scales: those whose encoding does not change, keys if none turns."""
    return [c["src"] == c["dst"] and (kv == 1 or c["rot"] == 0) for kv in range(2 if c["values"] else 1)]


def _move_plain(s):
    c = s["c"]
    rot = c["rot"]
    keep = s["dst_rows"] >= 0
    at, frm = s["dst_rows"][keep], s["src_rows"][keep]
    kv = _decode(c, s["src"], s["src_rows"][keep], torch.float32)
    if rot:
        ang = s["new"][keep].double()[:, None] * s["new_freq"].double() - s["old"][keep].double()[:, None] * \
            s["old_freq"].double()
        co, si = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
        x = kv[0][..., :rot]
        if c["inter"]:
            a, b = x[..., 0::2], x[..., 1::2]
            x = torch.stack((a * co - b * si, b * co + a * si), -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:]
            x = torch.cat((a * co - b * si, b * co + a * si), -1)
        kv = torch.stack((torch.cat((x, kv[0][..., rot:]), -1), kv[1]))
    for i, same in enumerate(_as_they_are(c)):
        if c["dst"] == "bf16":
            s["dst"][0][i, at] = kv[i].to(torch.bfloat16)
        elif c["dst"] == "int8":
            if same:
                s["dst"][0][i, at], s["dst"][1][i, at] = s["src"][0][i, frm], s["src"][1][i, frm]
            else:
                codes, scale = _codes(kv[i], 127)
                s["dst"][0][i, at], s["dst"][1][i, at] = codes.to(torch.int8), scale[..., 0]
        elif same:
            s["dst"][at, :, i] = s["src"][frm, :, i]
            s["back"][0][i, at] = kv[i].to(torch.bfloat16)
        else:
            codes, scale = _codes(kv[i].unflatten(-1, (-1, 64)), 7)
            s["back"][0][i, at] = (codes * scale.float()).flatten(-2).to(torch.bfloat16)
            codes = codes.flatten(-2).to(torch.int8)
            codes = ((codes[..., 0::2] & 15) | (codes[..., 1::2] << 4)).view(torch.uint8)
            s["dst"][at, :, i] = torch.cat((codes, scale[..., 0].contiguous().view(torch.uint8)), -1)
    return _move_out(s)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] != "move" and work(case)["flops"] > 1.0e13:
        return None
    s = prepare(case, seed)
    return _move_exact(s) if case["op"] == "move" else _attend_exact(s)


def _attend_exact(s):
    """Request by request: one softmax over the prefix's keys and the request's own."""
    c = s["c"]
    Hq, d = c["Hq"], c["d"]
    G = Hq // c["Hkv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    group = -1
    for b, (T, m) in enumerate(zip(s["lens"], s["new"])):
        at = s["starts"][b]
        g = max(i for i in range(len(s["start"])) if s["start"][i] <= b)
        P = s["prefix"][g] if g < len(s["prefix"]) else 0
        if P and g != group:
            group, (pk, pv) = g, _keys(s, s["prefix_table"][g], P, torch.float64)
        k, v = _keys(s, s["table"][b], T, torch.float64)
        hidden = torch.arange(T, device="cuda")[None] > torch.arange(T - m, T, device="cuda")[:, None]
        for h in range(c["Hkv"]):
            q = s["q"][at:at + m, h * G:(h + 1) * G].double() / math.sqrt(d)        # [m][G][d]
            z = (q @ k[:, h].T).masked_fill_(hidden[:, None], -math.inf)
            if P:
                z = torch.cat((q @ pk[:, h].T, z), -1)
            w = torch.softmax(z, -1)
            o = w[..., P:] @ v[:, h]
            if P:
                o = o + w[..., :P] @ pv[:, h]
            out[at:at + m, h * G:(h + 1) * G] = o
    return out


def _move_exact(s):
    c = s["c"]
    rot, d, m = c["rot"], c["d"], 2 if c["values"] else 1
    x = _decode(c, s["src"], s["src_rows"], torch.float64)
    if rot:
        z = x[0][..., :rot]
        z = z.unflatten(-1, (rot // 2, 2)) if c["inter"] else z.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        turn = s["new"].double()[:, None] * s["new_freq"].double() - s["old"].double()[:, None] * s["old_freq"].double()
        z = torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones_like(turn), turn)[:, None]
        z = torch.view_as_real(z)
        z = z.flatten(-2) if c["inter"] else z.transpose(-1, -2).flatten(-2)
        x = torch.stack((torch.cat((z, x[0][..., rot:]), -1), x[1]))
    x = x[:m]
    if c["dst"] != "bf16":  # the nearest multiples of the row's, or of each 64 values', fp16 scale
        codes, scale = _codes(x.unflatten(-1, (-1, d if c["dst"] == "int8" else 64)), 127 if c["dst"] == "int8" else 7)
        new = (codes * scale.double()).flatten(-2)
        x = torch.stack([a if same else b for a, b, same in zip(x, new, _as_they_are(c))])
    full = torch.zeros((m, c["n"] + 64, c["Hkv"], d), dtype=torch.float64, device="cuda")
    keep = s["dst_rows"] >= 0
    full[:, s["dst_rows"][keep]] = x[:, keep]
    return full
