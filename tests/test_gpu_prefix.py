"""A prefix put together and attended, as a serving program does it: documents
appended once, at positions of their own, are moved behind a prompt and a batch
asks about them.

Tolerances, from the arithmetic: what the rows hold against the fp64 keys at
their last positions, a rounding at a time -- appended (bf16, 2^-8 of a value, then
int8, half a code of the row's largest value), kept as int4 (half a code of it),
turned (at most sqrt(2) of what the pair was off by, and 2^-20 of its values) and
encoded again; the attention against its plain form on what the rows hold.
"""
import numpy as np
import pytest
import torch

from oracle import newtokens as append
from oracle import shared as plain
from test_gpu_shared import f64, skv, tolerance  # noqa: F401  (skv is a fixture)

pytestmark = pytest.mark.gpu


def rows_of(table, page, n):
    t = np.arange(n)
    return torch.from_numpy(np.asarray(table)[t // page].astype(np.int64) * page + t % page).cuda()


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("through", ["bf16", "int8", "int4"])
def test_documents_behind_a_prompt(skv, through, graph):  # noqa: F811
    d, Hq, Hkv, page, rot = 256, 8, 2, 16, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    inv = (1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
    weight = 1 + 0.1 * torch.randn((d,), generator=g, device="cuda")
    docs, asks = [130, 75], [3, 1, 5, 2]                   # tokens of the documents, of the questions
    P, n = sum(docs), sum(asks)
    x = [(randn(m, Hkv, d), randn(m, Hkv, d)) for m in docs]
    q, k, v = randn(n, Hq, d), randn(n, Hkv, d), randn(n, Hkv, d)

    int8 = through != "bf16"
    kind = skv.KV_INT8 if int8 else skv.KV_BF16
    blocks = -(-P // page) + sum(-(-m // page) for m in asks) + 2
    perm = np.random.default_rng(0).permutation(blocks).astype(np.int32)
    prefix_table = perm[None, :-(-P // page)].copy()
    table = np.array([[perm[prefix_table.shape[1] + b]] for b in range(len(asks))], np.int32)

    def pool(rows):
        if int8:
            return ([torch.zeros((rows, Hkv, d), dtype=torch.int8, device="cuda") for _ in range(2)],
                    [torch.zeros((rows, Hkv), dtype=torch.float16, device="cuda") for _ in range(2)])
        return [torch.zeros((rows, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)], [None, None]

    (kp, vp), (ks, vs) = pool(blocks * page)
    stores = []
    for m in docs:  # where the documents wait: rows as appended, or an int4 tier
        rows, scales = pool(m)
        tier = torch.zeros((m, Hkv, 2, d // 2 + d // 32), dtype=torch.uint8, device="cuda") if through == "int4" else None
        stores.append((rows, scales, tier))
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    starts = np.concatenate([[0], np.cumsum(asks)])
    dev = dict(group_start=i32([0, len(asks)]), prefix_table=i32(prefix_table.tolist()), prefix_lengths=i32([P]),
               block_table=i32(table.tolist()), lengths=i32(asks), q_start=i32(starts.tolist()))
    own_rows = torch.cat([rows_of(t, page, m) for t, m in zip(table, asks)])
    own_pos = torch.cat([torch.arange(P, P + m, device="cuda", dtype=torch.int32) for m in asks])
    prefix_rows = rows_of(prefix_table[0], page, P)
    at = [torch.arange(m, device="cuda", dtype=torch.int32) for m in docs]
    first = np.concatenate([[0], np.cumsum(docs)])
    q_out, out = torch.zeros_like(q), torch.full_like(q, 9.0)
    ws = torch.zeros((skv.shared_attend_workspace_size(len(asks), 1, n, Hq, Hkv, d),), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        for i, ((dk, dv), (rows, scales, tier)) in enumerate(zip(x, stores)):
            m = docs[i]
            skv.norm_rope_append(None, dk, dv, at[i], inv, None, *rows, k_weight=weight, kv_kind=kind, k_scale=scales[0],
                                 v_scale=scales[1], status=st)
            src = skv.row_set(kind, *rows, *scales)
            if tier is not None:
                skv.move_rows(src, skv.tier_rows(tier), m, status=st)
                src = skv.tier_rows(tier)
            to = int(first[i])
            skv.move_rows(src, skv.row_set(kind, kp, vp, ks, vs), m, dst_rows=prefix_rows[to:to + m], old_positions=at[i],
                          old_inv_freq=inv, new_positions=at[i] + to, new_inv_freq=inv, status=st)
        skv.norm_rope_append(q, k, v, own_pos, inv, q_out, kp, vp, q_weight=weight, k_weight=weight, kv_kind=kind,
                             k_scale=ks, v_scale=vs, out_rows=own_rows, status=st)
        skv.shared_attend(kind, q_out, kp, vp, page=page, softmax_scale=d ** -0.5, out=out, workspace=ws, k_scale=ks,
                          v_scale=vs, status=st, **dev)

    step()
    if graph:
        torch.cuda.synchronize()
        once = out.clone()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            step()
        for t in (kp, vp, out, q_out):
            t.zero_()
        cg.replay()
        assert torch.equal(out, once)
    assert int(st.item()) == 0

    norm = lambda t, pos: append.norm_rope(f64(t), f64(weight), 1e-6, pos.cpu().numpy(), f64(inv), False)  # noqa: E731
    held = [f64(p) * (1 if s is None else f64(s)[..., None]) for p, s in ((kp, ks), (vp, vs))]
    want = [np.concatenate([norm(dk, a + int(o))[0] for (dk, _), a, o in zip(x, at, first)]), np.concatenate([f64(dv) for _, dv in x])]
    for turned, got, z in ((True, held[0], want[0]), (False, held[1], want[1])):
        largest = np.abs(z).max(-1, keepdims=True)
        off = 2.0 ** -8 * np.abs(z) + 2.0 ** -19 * largest if turned else 0 * z  # values are appended as they are
        if turned:  # a pair's lengths, and with them its values, change by the turn: the row's largest value bounds them
            off = off.max(-1, keepdims=True) * 2 ** 0.5 + 0 * z
        code = lambda top, e: (largest * 2 ** 0.5 + e) / (2 * top) * (1 + 2.0 ** -10)  # noqa: E731
        if int8:
            off = off + code(127, off)
        if through == "int4":
            off = off + code(7, off)
        if turned:
            off = 2 ** 0.5 * off + 2.0 ** -19 * largest
        if int8:
            off = off + code(127, off) if turned or through == "int4" else off
        elif turned:
            off = off + 2.0 ** -8 * (np.abs(z) + off)
        assert (np.abs(got[prefix_rows.cpu().numpy()] - z) <= off).all()
    z, mag = norm(q, own_pos)
    assert (np.abs(f64(q_out) - z) <= 2.0 ** -8 * np.abs(z) + 2.0 ** -19 * mag).all()
    ref, spread = plain.shared_attend(f64(q_out), *held, [0, len(asks)], prefix_table, [P], table, page, asks, d ** -0.5, starts)
    assert (np.abs(f64(out) - ref) <= tolerance(ref, spread)).all()
