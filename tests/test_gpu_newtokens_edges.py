"""skv_norm_rope_append and skv_paged_attend where they could go wrong without
an ordinary call showing it: waits that give up, offsets out of order, values
and scales at the ends of their ranges."""
import ctypes
import os
import subprocess
import types

import numpy as np
import pytest
import torch

from oracle import newtokens as plain
from test_gpu_newtokens import KINDS, Case, f64, gen, kind_of, skv, status  # noqa: F401  (skv is a fixture)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# waits that give up
# ---------------------------------------------------------------------------

@pytest.fixture(scope="module")
def hasty(skv, tmp_path_factory):  # noqa: F811
    """The attention built so that a wait gives up after its first look, in place of the library's."""
    from sparse_kv_long_gb300 import _build
    so = str(tmp_path_factory.mktemp("hasty") / "libhasty.so")
    cmd = [_build.nvcc(), *_build.ARCH, *_build.FLAGS, "-DSKV_PAGED_LOOKS=0", "-shared",
           os.path.join(_build.CSRC, "paged.cu"), "-o", so]
    subprocess.run(cmd, check=True, capture_output=True)
    lib, usual = ctypes.CDLL(so), skv.lib()
    for name in ("skv_paged_attend", "skv_paged_attend_workspace_size"):
        f, u = getattr(lib, name), getattr(usual, name)
        f.argtypes, f.restype = u.argtypes, u.restype
    return types.SimpleNamespace(skv_paged_attend=lib.skv_paged_attend,
                                 skv_paged_attend_workspace_size=lib.skv_paged_attend_workspace_size)


def gives_up(skv, hasty, monkeypatch, c, single):  # noqa: F811
    """A call whose waits give up sets SKV_DEV_TIMEOUT and touches nothing but its tokens' output and its workspace,
    whatever that held; the next call on the same buffers is right."""
    want = c.run(single=single).clone()
    n, need = c.q.shape[0], c.ws.numel()
    ws = torch.full((need + 4096,), 0x7F, dtype=torch.uint8, device="cuda")
    with monkeypatch.context() as m:
        m.setattr(skv, "_lib", hasty)
        got = c.run(single=single, ws=ws[:need])
        torch.cuda.synchronize()
    assert int(c.st.item()) == skv.DEV_TIMEOUT
    tokens = int(c.starts[-1])
    assert (got[tokens:] == 123).all() and n >= tokens
    assert (ws[need:] == 0x7F).all()
    assert torch.equal(c.run(single=single, ws=ws[:need]), want) and int(c.st.item()) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,lens,new,single", [
    (256, [9000, 20, 3000], [1, 1, 1], True), (128, [20000], [3], False), (256, [3000] * 9, [8] * 9, False),
])
def test_single_ctas_that_give_up(skv, hasty, monkeypatch, kind, d, lens, new, single):  # noqa: F811
    c = Case(skv, kind_of(skv, kind), d, 8, 2, 16, lens, new, seed=50, pad=0 if single else 3)
    gives_up(skv, hasty, monkeypatch, c, single)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,lens,new", [(256, [30000], [700]), (128, [9000, 12000], [300, 300]), (256, [5000, 300], [2000, 250])])
def test_pairs_that_give_up(skv, hasty, monkeypatch, kind, d, lens, new):  # noqa: F811
    """Requests cut into pieces whose descriptors other pairs write: given up on, they are this call's all the same."""
    c = Case(skv, kind_of(skv, kind), d, 8, 2, 64, lens, new, seed=51, pad=3)
    gives_up(skv, hasty, monkeypatch, c, False)


# ---------------------------------------------------------------------------
# the merge
# ---------------------------------------------------------------------------

def test_changing_calls_queued_on_one_workspace(skv):  # noqa: F811
    """Calls whose lists of split items and partials differ, one behind the other on a workspace without a wait: the
    merge, launched while the attention runs, reads this call's."""
    cases = [Case(skv, kind_of(skv, k), d, 8, 2, 16, lens, new, seed=60 + i) for i, (k, d, lens, new) in enumerate([
        ("bf16", 256, [9000], [1]), ("int8", 256, [700, 5000, 3], [2, 3, 1]), ("bf16", 128, [6000], [400]),
        ("bf16", 256, [4000, 100, 2500], [1, 1, 1]), ("int8", 128, [8000], [200])])]
    need = max(skv.paged_attend_workspace_size(len(c.lens), c.q.shape[0], 8, 2, c.d) for c in cases)
    ws = torch.zeros((need,), dtype=torch.uint8, device="cuda")
    want = []
    for c in cases:
        want.append(c.run(ws=ws).clone())
        torch.cuda.synchronize()
    for _ in range(20):
        for c in cases:
            c.out.zero_()
        for c in cases + cases[::-1]:
            c.call()
        torch.cuda.synchronize()
        assert all(torch.equal(c.out, w) for c, w in zip(cases, want))
    assert all(int(c.st.item()) == 0 for c in cases)


# ---------------------------------------------------------------------------
# offsets out of order
# ---------------------------------------------------------------------------

def kept(starts, n):
    """Requests that remain: offsets in order and within [0, n], and no token that such a request before them has."""
    good = [0 <= s <= e <= n for s, e in zip(starts, starts[1:])]
    return [b for b in range(len(good)) if good[b] and not any(
        good[i] and starts[i + 1] > starts[i] and starts[i + 1] > starts[b] for i in range(b))]


def bad_offsets(skv, kind, d, page, lens, starts, n):  # noqa: F811
    c = Case(skv, kind, d, 8, 2, page, lens, [0] * len(lens), seed=70, pad=n)
    c.starts = np.array(starts, np.int32)
    c.run()  # lays the device tensors out; once more into the middle of a larger output
    wide = torch.full((n + 64, 8, d), 123.0, dtype=torch.bfloat16, device="cuda")
    c.out = wide[32:32 + n]
    c.st.zero_()
    c.call()
    keep, owned = kept(starts, n), torch.zeros(n + 64, dtype=torch.bool, device="cuda")
    assert int(c.st.item()) == (0 if len(keep) == len(lens) else skv.DEV_RANGE)
    k, v = c.values()
    for b in keep:
        s, e = starts[b], starts[b + 1]
        owned[32 + s:32 + e] = True
        ref, spread = plain.paged_attend(f64(c.q)[s:e], k, v, c.table[b:b + 1], page, [lens[b]], c.scale, [0, e - s], 0, 0)
        tol = 2.0 ** -8 * np.abs(ref) + 2 * (2.0 ** -8 + 2.0 ** -10) * (spread + np.abs(ref))
        assert (np.abs(f64(c.out[s:e]) - ref) <= tol).all()
    assert (wide[~owned] == 123).all()  # nobody's rows, and those around the output


@pytest.mark.parametrize("starts", [[0, 5, 3, 9], [0, 5, 9, 400], [-3, 2, 4, 9], [2, 4, 6, 9], [0, 9, 0, 9], [7, 7, 3, 9],
                                    [0, 400, 5, 9], [4, 2, 6, 5], [9, 9, 9, 9], [10, 9, 0, 4]])
@pytest.mark.parametrize("kind", KINDS)
def test_offsets_out_of_order(skv, kind, starts):  # noqa: F811
    """Single CTAs: only the requests that remain are written, and these are right."""
    bad_offsets(skv, kind_of(skv, kind), 128, 16, [64, 700, 64], starts, 9)


@pytest.mark.parametrize("starts", [[0, 300, 0, 300], [0, 250, 100, 300], [5, 2, 290, 280], [0, 1000, 120, 300], [30, 40, 40, 200]])
@pytest.mark.parametrize("kind", KINDS)
def test_offsets_out_of_order_in_chunks(skv, kind, starts):  # noqa: F811
    """The same for CTA pairs."""
    bad_offsets(skv, kind_of(skv, kind), 256, 16, [400, 300, 900], starts, 300)


@pytest.mark.parametrize("d,n,T", [(128, 1 << 20, 40000), (256, 1 << 19, 20100)])
def test_offsets_that_repeat_the_largest_request(skv, d, n, T):  # noqa: F811
    """2048 times the same tokens: taken as they are, the work list's counts would pass 32 bits.  The first has them."""
    B, page = 4096, 64
    g = gen(71)
    k = torch.randn((T // page + 1) * page, 1, d, generator=g, device="cuda").bfloat16()
    q = torch.randn(n, 1, d, generator=g, device="cuda").bfloat16()
    table = torch.arange(T // page + 1, device="cuda", dtype=torch.int32).repeat(B, 1)
    lens = torch.full((B,), T, device="cuda", dtype=torch.int32)
    ws = torch.zeros((skv.paged_attend_workspace_size(B, n, 1, 1, d),), dtype=torch.uint8, device="cuda")
    out = []
    for starts in ([0] + [n] * B, [0, n] * (B // 2) + [0]):
        st, o = status(), torch.zeros_like(q)
        skv.paged_attend(skv.KV_BF16, q, k, k, table, page, lens, d ** -0.5, o, ws,
                         q_start=torch.tensor(starts, device="cuda", dtype=torch.int32), status=st)
        out.append((o, int(st.item())))
    assert torch.equal(out[0][0], out[1][0]) and (out[0][0] != 0).any()
    assert [x[1] for x in out] == [0, skv.DEV_RANGE]


# ---------------------------------------------------------------------------
# values at the ends of their ranges
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("d,T,n", [(256, 20000, 1), (128, 20000, 3), (256, 20000, 200)])
def test_a_value_under_a_vanishing_weight_reaches_the_output(skv, d, T, n, value):  # noqa: F811
    """A value that is not finite, seen under a weight below fp32's range (another key's logit is hundreds larger):
    whatever piece of the keys it falls into, its column is not finite, and the others are as without it."""
    c = Case(skv, skv.KV_BF16, d, 2, 2, 64, [T], [n], seed=80)
    row = lambda t: int(c.table[0][t // 64]) * 64 + t % 64  # noqa: E731
    c.q[:] = c.q[:1]
    c.k[row(T - 300)] = 8 * c.q[0]  # every token sees it, with a logit of 8 |q|^2 / sqrt(d)
    clean, col = c.run().clone(), 77
    for t in (0, 100, T // 2, T - 700):
        kept = c.v[row(t), 0, col].clone()
        c.v[row(t), 0, col] = value
        got = c.run()
        c.v[row(t), 0, col] = kept
        assert not torch.isfinite(got[:, 0, col]).any(), t
        same = torch.ones_like(got, dtype=torch.bool)
        same[:, 0, col] = False
        assert torch.equal(got[same], clean[same])


FORMS = [  # single tokens, drafts, pairs
    (256, [700, 64, 1, 3000], [1, 1, 1, 1], True), (128, [700, 64, 1, 3000], [1, 1, 1, 1], True),
    (256, [2000, 90], [3, 5], False), (128, [2000, 90], [7, 2], False),
    (256, [2000, 300], [400, 300], False), (128, [2000, 300], [400, 300], False),
]


@pytest.mark.parametrize("d,lens,new,single", FORMS)
def test_value_rows_of_zeros(skv, d, lens, new, single):  # noqa: F811
    """An all-zero value row has a zero scale: its weight counts in the sum.  Half the rows, every row of the first
    request (exact zeros come out), and none elsewhere in turn."""
    for seed, share in ((90, 0.5), (91, 0.9), (92, 1.0)):
        c = Case(skv, skv.KV_INT8, d, 8, 2, 16, lens, new, seed=seed)
        zero = (torch.rand(c.vs.shape, generator=gen(seed), device="cuda") < share) & c.owned[:, None]
        t = np.arange(lens[0])
        zero[torch.from_numpy(c.table[0][t // 16].astype(np.int64) * 16 + t % 16).cuda()] = True
        c.vs[zero], c.v[zero] = 0, 0
        c.check(single=single)
        assert (c.out[:new[0]] == 0).all()


@pytest.mark.parametrize("d,lens,new,single", FORMS)
def test_value_scales_of_every_size(skv, d, lens, new, single):  # noqa: F811
    """Scales from the smallest fp16 subnormal to the largest number within a tile, a tenth of the rows zero: the sum
    takes every weight through the reciprocal of its scale.  Keys' scales from zero to large ones, too."""
    for seed, lo, hi in ((93, -24.0, 15.9), (94, -24.0, -20.0), (95, -12.0, 4.0), (96, 10.0, 15.9)):
        c = Case(skv, skv.KV_INT8, d, 8, 2, 16, lens, new, seed=seed)
        g = gen(seed)
        scale = torch.exp2(lo + (hi - lo) * torch.rand(c.vs.shape, generator=g, device="cuda")).half()
        scale[torch.rand(c.vs.shape, generator=g, device="cuda") < 0.1] = 0
        scale = torch.where(torch.rand(c.vs.shape, generator=g, device="cuda") < 0.2, -scale, scale)
        c.v[(scale == 0) & c.owned[:, None]] = 0
        c.vs = torch.where(c.owned[:, None], scale, c.vs)
        ks = torch.exp2(-24.0 + 18.0 * torch.rand(c.ks.shape, generator=g, device="cuda")).half()
        ks[torch.rand(c.ks.shape, generator=g, device="cuda") < 0.1] = 0
        c.ks = torch.where(c.owned[:, None], ks, c.ks)
        c.check(single=single)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_append_encodes_rows_of_any_value(skv, d):  # noqa: F811
    """Zeros, subnormals, numbers too small or too large for the scale, infinities, NaN: int8 rows are what
    skv_quantize_int8_rows makes of the bf16 rows."""
    g, n, H = gen(100), 400, 3
    size = torch.exp2(torch.randint(-130, 127, (n, H, 1), generator=g, device="cuda").float())
    x = (torch.randn((n, H, d), generator=g, device="cuda") * size).bfloat16()
    x[:8] = 0
    pick = lambda: torch.rand(x.shape, generator=g, device="cuda") < 0.01  # noqa: E731
    for i, value in enumerate([float("inf"), float("-inf"), float("nan"), 1e-40, 3.38e38, 127 * 2.0 ** -25,
                               127 * 1.5 * 2.0 ** -24]):
        m = pick()
        m[:40 + 40 * i] = False
        x[m] = value
    pos = torch.arange(n, device="cuda", dtype=torch.int32)
    rows = [torch.zeros_like(x) for _ in range(2)]
    skv.norm_rope_append(None, x, x, pos, None, None, *rows)
    codes = [torch.full(x.shape, 99, dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.full((n, H), 9.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    skv.norm_rope_append(None, x, x, pos, None, None, *codes, kv_kind=skv.KV_INT8, k_scale=scales[0], v_scale=scales[1])
    for r, c, s in zip(rows, codes, scales):
        rc, rs = torch.zeros_like(c), torch.zeros_like(s)
        skv.quantize_int8_rows(r, rc, rs)
        assert torch.equal(rc, c) and torch.equal(rs.view(torch.int16), s.view(torch.int16))
    assert torch.equal(rows[1].view(torch.int16), x.view(torch.int16))  # values as they are, bit for bit


def test_outputs_may_take_the_queries_place(skv):  # noqa: F811
    """Attention whose output is its queries' tensor: a query is read before its row is written, also where the keys are
    cut and joined."""
    for kind, d, lens, new in [("bf16", 256, [5000, 30], [1, 1]), ("int8", 128, [2000, 900], [300, 5])]:
        c = Case(skv, kind_of(skv, kind), d, 8, 2, 16, lens, new, seed=101)
        want = c.run().clone()
        q = c.q.clone()
        c.run(q=q)
        skv.paged_attend(c.kind, q, c.k, c.v, c.dev[0], 16, c.dev[1], c.scale, q, c.ws, q_start=c.dev[2], k_scale=c.ks,
                         v_scale=c.vs, status=c.st)
        assert torch.equal(q, want)


@pytest.mark.parametrize("kind", KINDS)
def test_values_alone_read_no_frequencies(skv, kind):  # noqa: F811
    """With q and k left out nothing is rotated, whatever rot says: inv_freq may be NULL."""
    n, H, d = 5, 2, 128
    v = torch.randn((n, H, d), device="cuda").bfloat16()
    pos = torch.arange(n, device="cuda", dtype=torch.int32)
    pool = torch.zeros((n, H, d), dtype=torch.int8 if kind == "int8" else torch.bfloat16, device="cuda")
    scale = torch.zeros((n, H), dtype=torch.float16, device="cuda")
    at = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    assert skv.lib().skv_norm_rope_append(
        n, 0, H, d, 64, 0, None, 0, None, 0, at(v), H * d, None, None, 1e-6, at(pos), None, None, kind_of(skv, kind), None, n,
        None, at(pool), None, at(scale), None, None) == 0
    torch.cuda.synchronize()
    want, ws = torch.zeros_like(pool), torch.zeros_like(scale)
    if kind == "int8":
        skv.quantize_int8_rows(v, want, ws)
    assert torch.equal(pool, want if kind == "int8" else v) and torch.equal(scale, ws)
