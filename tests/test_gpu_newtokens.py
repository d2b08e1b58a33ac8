"""skv_norm_rope_append and skv_paged_attend against their plain fp64 forms.

Tolerances, from the arithmetic.  Half a step of bf16 is 2^-8 of the value.
  norm + rotation: 2^-8 |z| for the output's rounding, and fp32 errors of the
    chain (a sum of d squares, rsqrt, three products, the sine and cosine, the
    rotation) below 2^-19 of |y_a| + |y_b|.
  attention: weights rounded to bf16 and divided by their rounded sum change
    the mean by at most 2 * 2^-8 of sum w |v| + |out|; a logit's fp32 error
    below 2^-10 (d products of a few units, 2^-24 each) the same way; and
    2^-8 |out| for the output's rounding.
"""
import math

import numpy as np
import pytest
import torch

import skvtest as T
from oracle import newtokens as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def skv():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from sparse_kv_long_gb300 import _build
    _build.build()
    import sparse_kv_long_gb300 as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def f64(t):
    return t.detach().double().cpu().numpy()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# norm + rotation + append
# ---------------------------------------------------------------------------

def freqs(rot, theta=1e6):
    return (theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()


def check_norm(got, x, weight, pos, inv, inter, eps=1e-6):
    z, mag = plain.norm_rope(f64(x), None if weight is None else f64(weight), eps, pos.cpu().numpy(), f64(inv), inter)
    err = np.abs(f64(got) - z)
    tol = 2.0 ** -8 * np.abs(z) + 2.0 ** -19 * mag
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,Hq,Hkv,rot,n", [
    (256, 24, 4, 64, 8), (256, 16, 2, 256, 33), (256, 1, 1, 16, 1), (128, 32, 8, 128, 5), (128, 3, 1, 96, 700),
    (128, 5, 3, 48, 65), (64, 7, 3, 32, 19), (64, 1, 1, 64, 1), (256, 24, 4, 0, 9), (128, 8, 8, 112, 9000),
])
def test_norm_rope_bf16(skv, d, Hq, Hkv, rot, n, inter):
    g = gen(d + n + rot)
    x = randn(g, n, Hq + 2 * Hkv, d, scale=1.7)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]  # views of one projection
    qw = 1 + 0.3 * torch.randn((d,), generator=g, device="cuda")
    kw = 1 + 0.3 * torch.randn((d,), generator=g, device="cuda")
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = 0
    inv = freqs(rot)
    rows = torch.randperm(n + 7, generator=g, device="cuda")[:n]
    if n > 4:
        rows[n // 2] = -1
    q_out = torch.full((n, Hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    kp = torch.full((n + 7, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    vp, st = kp.clone(), status()
    skv.norm_rope_append(q, k, v, pos, inv, q_out, kp, vp, q_weight=qw, k_weight=kw, interleaved=inter, out_rows=rows,
                         status=st)
    assert int(st.item()) == 0
    check_norm(q_out, q, qw, pos, inv, inter)
    keep = rows >= 0
    check_norm(kp[rows[keep]], k[keep], kw, pos[keep], inv, inter)
    assert torch.equal(vp[rows[keep]], v[keep])
    other = torch.ones(n + 7, dtype=torch.bool, device="cuda")
    other[rows[keep]] = False
    assert (kp[other] == 7).all() and (vp[other] == 7).all()  # rows of nobody are left as they were


@pytest.mark.parametrize("d,Hq,Hkv,rot,inter", [(256, 24, 4, 64, False), (128, 4, 3, 128, True), (64, 2, 5, 16, False)])
def test_norm_rope_int8_rows_are_the_encoding_of_the_bf16_rows(skv, d, Hq, Hkv, rot, inter):
    """Bit-exact: int8 mode stores what skv_quantize_int8_rows makes of the bf16 mode's rows."""
    g, n = gen(5), 301
    q, k, v = randn(g, n, Hq, d), randn(g, n, Hkv, d, scale=0.4), randn(g, n, Hkv, d)
    v[3] = 0  # a zero row has a zero scale and zero codes
    pos = torch.randint(0, 1 << 18, (n,), generator=g, device="cuda", dtype=torch.int32)
    inv, w = freqs(rot), torch.rand((d,), generator=g, device="cuda") + 0.5
    kb, vb = torch.zeros_like(k), torch.zeros_like(v)
    q1, q2 = torch.zeros_like(q), torch.zeros_like(q)
    skv.norm_rope_append(q, k, v, pos, inv, q1, kb, vb, q_weight=w, k_weight=w, interleaved=inter)
    k8, v8 = (torch.full((n, Hkv, d), 99, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((n, Hkv), 9.0, dtype=torch.float16, device="cuda") for _ in range(2))
    skv.norm_rope_append(q, k, v, pos, inv, q2, k8, v8, q_weight=w, k_weight=w, interleaved=inter,
                         kv_kind=skv.KV_INT8, k_scale=ks, v_scale=vs)
    assert torch.equal(q1, q2)
    for rows, codes, scale in [(kb, k8, ks), (vb, v8, vs)]:
        rc, rs = torch.zeros_like(codes), torch.zeros_like(scale)
        skv.quantize_int8_rows(rows, rc, rs)
        assert torch.equal(rc, codes) and torch.equal(rs, scale)


def test_norm_rope_parts_may_be_left_out(skv):
    g, n, d = gen(6), 40, 128
    q, k, v = randn(g, n, 4, d), randn(g, n, 2, d), randn(g, n, 2, d)
    pos, inv = torch.arange(n, device="cuda", dtype=torch.int32) * 977, freqs(64)
    w = torch.rand((d,), generator=g, device="cuda") + 0.5
    full = [torch.zeros_like(t) for t in (q, k, v)]
    skv.norm_rope_append(q, k, v, pos, inv, *full, q_weight=w, k_weight=w)
    part = [torch.zeros_like(t) for t in (q, k, v)]
    skv.norm_rope_append(q, k, None, pos, inv, part[0], part[1], None, q_weight=w, k_weight=w)
    skv.norm_rope_append(None, None, v, pos, None, None, None, part[2])
    assert all(torch.equal(a, b) for a, b in zip(full, part))
    only = torch.zeros_like(k)
    skv.norm_rope_append(None, k, None, pos, inv, None, only, None, k_weight=w)
    assert torch.equal(only, full[1])
    # no weight: rotated, not normed
    skv.norm_rope_append(q, None, None, pos, inv, part[0], None, None)
    check_norm(part[0], q, None, pos, inv, False)


@pytest.mark.parametrize("n_of", [1, 3])
def test_norm_rope_far_positions(skv, n_of):
    """Positions up to 2^31 - 1 and negative ones: the angle keeps 1e-6 of a turn there (up to 2^24 below 1e-7)."""
    d = 128
    pos = torch.tensor(([1 << 20, (1 << 24) - 1, (1 << 24) + 1, 1 << 30, (1 << 31) - 1, -5, 0] * n_of),
                       dtype=torch.int32, device="cuda")
    q, inv = randn(gen(8), len(pos), 2, d), freqs(d)
    out = torch.zeros_like(q)
    skv.norm_rope_append(q, None, None, pos, inv, out, None, None)
    check_norm(out, q, None, pos, inv, False)


def test_norm_rope_bad_row_is_skipped_and_flagged(skv):
    n, d = 6, 256
    q, k = randn(gen(9), n, 4, d), randn(gen(10), n, 2, d)
    pos, inv = torch.arange(n, device="cuda", dtype=torch.int32), freqs(64)
    rows = torch.tensor([0, 1, 9, 3, -4, 5], device="cuda")
    big = torch.zeros((12, 2, d), dtype=torch.bfloat16, device="cuda")
    st, out = status(), torch.zeros_like(q)
    skv.norm_rope_append(q, k, None, pos, inv, out, big[:6], None, out_rows=rows, status=st)
    assert int(st.item()) == skv.DEV_RANGE
    check_norm(out, q, None, pos, inv, False)
    assert (big[6:] == 0).all() and (big[2] == 0).all() and (big[4] == 0).all()
    check_norm(big[[0, 1, 3, 5]], k[[0, 1, 3, 5]], None, pos[[0, 1, 3, 5]], inv, False)


# ---------------------------------------------------------------------------
# attention of new tokens
# ---------------------------------------------------------------------------

class Case:
    """A paged batch with shuffled blocks; every pool row that no request owns holds NaN (int8: NaN scales)."""

    def __init__(self, skv, kind, d, Hq, Hkv, page, lens, new, seed, pad=0, extra_pages=0):
        g = gen(seed)
        self.skv, self.kind, self.d, self.Hq, self.Hkv, self.page = skv, kind, d, Hq, Hkv, page
        self.lens, self.new = lens, new
        B = len(lens)
        need = [-(-max(t, 0) // page) for t in lens]
        self.n_pages = max(max(need), 1) + extra_pages
        blocks = sum(need) + 3
        perm = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32).cpu().numpy()
        self.table = np.full((B, self.n_pages), -1, np.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = perm[at:at + m]
            at += m
        rows = blocks * page
        owned = torch.zeros(rows, dtype=torch.bool)
        for b, t in enumerate(lens):
            x = np.arange(max(t, 0))
            owned[torch.from_numpy(self.table[b][x // page].astype(np.int64) * page + x % page)] = True
        self.owned = owned = owned.cuda()
        if kind == skv.KV_INT8:
            self.k, self.v = (torch.randint(-127, 128, (rows, Hkv, d), generator=g, device="cuda", dtype=torch.int8)
                              for _ in range(2))
            self.ks, self.vs = (((torch.rand((rows, Hkv), generator=g, device="cuda") + 0.5) / 73).half()
                                for _ in range(2))
            self.ks[~owned] = float("nan")
            self.vs[~owned] = float("inf")
        else:
            self.k, self.v, self.ks, self.vs = randn(g, rows, Hkv, d), randn(g, rows, Hkv, d), None, None
            self.k[~owned] = float("nan")
            self.v[~owned] = float("inf")
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        n = int(self.starts[-1]) + pad
        self.q = randn(g, n, Hq, d, scale=1.5)
        self.scale = d ** -0.5

    def values(self):
        k, v = f64(self.k), f64(self.v)
        if self.ks is not None:
            k, v = k * f64(self.ks)[..., None], v * f64(self.vs)[..., None]
        return k, v

    def run(self, S=0, W=0, q=None, ws=None, single=False, stream=None):
        skv, B = self.skv, len(self.lens)
        q = self.q if q is None else q
        n = q.shape[0]
        self.out = torch.full((n, self.Hq, self.d), 123.0, dtype=torch.bfloat16, device="cuda")
        if ws is None:
            ws = torch.zeros((skv.paged_attend_workspace_size(B, n, self.Hq, self.Hkv, self.d),), dtype=torch.uint8,
                             device="cuda")
        self.ws, self.st = ws, status()
        self.dev = [T.dev(self.table), T.dev(np.array(self.lens, np.int32)),
                    None if single else T.dev(self.starts)]
        self.call = lambda: skv.paged_attend(
            self.kind, q, self.k, self.v, self.dev[0], self.page, self.dev[1], self.scale, self.out, ws,
            q_start=self.dev[2], S=S, W=W, k_scale=self.ks, v_scale=self.vs, status=self.st, stream=stream)
        self.call()
        return self.out

    def check(self, S=0, W=0, **kw):
        out = self.run(S, W, **kw)
        assert int(self.st.item()) == 0
        m = int(self.starts[-1])
        k, v = self.values()
        ref, spread = plain.paged_attend(f64(self.q)[:m], k, v, self.table, self.page, self.lens, self.scale,
                                         self.starts, S, W)
        got = f64(out)
        assert (got[m:] == 123).all()  # rows behind the last request are left as they were
        err, tol = np.abs(got[:m] - ref), 2.0 ** -8 * np.abs(ref) + 2 * (2.0 ** -8 + 2.0 ** -10) * (spread + np.abs(ref))
        finite = bool(np.isfinite(got).all())
        assert finite
        worst = float((err / np.maximum(tol, 1e-300)).max())
        assert worst <= 1


KINDS = ["bf16", "int8"]


def kind_of(skv, name):
    return skv.KV_INT8 if name == "int8" else skv.KV_BF16


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,Hq,Hkv,page", [(256, 24, 4, 16), (256, 16, 2, 64), (128, 8, 8, 8), (128, 32, 8, 48),
                                           (256, 5, 1, 128), (128, 128, 1, 256), (256, 7, 7, 24)])
def test_single_tokens(skv, kind, d, Hq, Hkv, page):
    lens = [1, 2, 7, 63, 64, 65, 127, 128, 129, 300, 1000, 0]
    Case(skv, kind_of(skv, kind), d, Hq, Hkv, page, lens, [1] * len(lens), seed=d + Hq).check(single=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,Hq,Hkv,page", [(256, 24, 4, 16), (256, 16, 2, 64), (128, 8, 8, 8), (128, 32, 8, 48),
                                           (256, 6, 1, 40), (128, 12, 4, 512), (256, 100, 1, 32)])
def test_chunks(skv, kind, d, Hq, Hkv, page):
    """Ragged chunks: none, one, some tokens, whole prompts; padding behind the last; more tokens than the cache
    holds (the first of them see nothing)."""
    lens = [10, 1, 5, 257, 300, 700, 3, 128]
    new = [0, 1, 5, 130, 300, 64, 9, 127]
    Case(skv, kind_of(skv, kind), d, Hq, Hkv, page, lens, new, seed=d + Hq + 1, pad=5, extra_pages=2).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("S,W", [(0, 1), (0, 16), (4, 100), (64, 128), (500, 7), (3, 5000), (129, 255), (0, 64)])
def test_window_and_sinks(skv, kind, S, W):
    lens, new = [1, 40, 129, 700, 1100, 900], [1, 40, 1, 300, 17, 1]
    d, Hq, Hkv = (256, 12, 2) if kind == "int8" else (128, 8, 2)
    Case(skv, kind_of(skv, kind), d, Hq, Hkv, 16, lens, new, seed=S + W, pad=1).check(S=S, W=W)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,lens,new,S,W", [
    (256, [5000], [1], 0, 0), (256, [5001], [3], 0, 0), (128, [9000, 20], [1, 1], 0, 0),
    (256, [4097], [300], 0, 0), (128, [3000, 3000], [500, 2], 0, 0), (256, [6000], [150], 64, 1024),
])
def test_long_axis_split(skv, kind, d, lens, new, S, W):
    """Few rows over many keys: the keys are split and joined."""
    Case(skv, kind_of(skv, kind), d, 8, 2, 64, lens, new, seed=lens[0]).check(S=S, W=W)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,lo,hi,n", [(40, 300, 1500, 1), (24, 10, 4000, 1), (30, 200, 900, 3), (7, 1000, 5000, 1)])
def test_ragged_batches_are_shared_out(skv, kind, B, lo, hi, n):
    """Ragged requests whose keys the CTAs share evenly: most items are cut, anywhere."""
    rng = np.random.default_rng(B + hi)
    lens = [int(x) for x in np.exp(rng.uniform(math.log(lo), math.log(hi), B))]
    c = Case(skv, kind_of(skv, kind), 256 if n == 1 else 128, 8, 2, 16, lens, [n] * B, seed=B)
    c.check(single=n == 1)


@pytest.mark.parametrize("kind", KINDS)
def test_many_requests(skv, kind):
    rng = np.random.default_rng(3)
    lens = [int(x) for x in np.exp(rng.uniform(0, math.log(600), 150))]
    new = [min(t, int(rng.integers(0, 4))) for t in lens]
    Case(skv, kind_of(skv, kind), 128, 4, 2, 16, lens, new, seed=11).check()


def test_peaked_and_flat_logits(skv):
    """A row whose logits span hundreds (one key takes all) and a row of equal logits."""
    c = Case(skv, skv.KV_BF16, 256, 4, 2, 16, [400, 400], [3, 200], seed=12)
    c.q[:2] = c.q[:2] * 40
    c.q[2] = 0
    c.check()


@pytest.mark.parametrize("kind", KINDS)
def test_growing_logits(skv, kind):
    """Keys whose logits climb by tile: the running maximum moves many times."""
    c = Case(skv, kind_of(skv, kind), 256, 4, 1, 64, [1500, 900], [2, 130], seed=13)
    ramp = torch.ones(c.k.shape[0], device="cuda")
    for b, t in enumerate(c.lens):
        x = np.arange(t)
        r = torch.from_numpy(c.table[b][x // 64].astype(np.int64) * 64 + x % 64).cuda()
        ramp[r] = torch.from_numpy(0.05 + x / 100.0).float().cuda()
    if kind == "int8":
        c.ks = (c.ks.float() * ramp[:, None]).half()
    else:
        c.k = (c.k.float() * ramp[:, None, None]).bfloat16()
    # logits of tens: their fp32 error grows with them, and with it the change of a weight
    c.q = (c.q.float() * 0.5).bfloat16()
    c.check()


@pytest.mark.parametrize("kind", KINDS)
def test_masked_values_may_hold_anything(skv, kind):
    """NaN and infinities in keys and values that a token does not see change nothing for it; in a value that it
    sees they reach its output."""
    c = Case(skv, kind_of(skv, kind), 256, 4, 1, 16, [300], [40], seed=14)
    row = lambda t: int(c.table[0][t // 16]) * 16 + t % 16  # noqa: E731
    clean = f64(c.run(S=2, W=50))
    late, gone, col = row(285), row(100), 77
    for t in (late, gone):
        if kind == "int8":
            c.ks[t], c.vs[t] = float("nan"), float("nan")
        else:
            c.k[t], c.v[t, 0, col] = float("inf"), float("nan")
    got = f64(c.run(S=2, W=50))
    sees = np.arange(260, 300) >= 285  # token 100 is outside every window here
    np.testing.assert_array_equal(got[~sees], clean[~sees])
    assert np.isnan(got[sees][..., col]).all()
    if kind == "bf16":  # an infinite value in one column, finite keys
        c = Case(skv, skv.KV_BF16, 256, 4, 1, 16, [300], [40], seed=14)
        c.v[late, 0, col] = float("-inf")
        c.v[gone, 0, col] = float("nan")
        got = f64(c.run(S=2, W=50))
        assert (got[sees][..., col] == -np.inf).all()
        np.testing.assert_array_equal(got[~sees], clean[~sees])
        keep = np.arange(256) != col
        np.testing.assert_array_equal(got[sees][..., keep], clean[sees][..., keep])


def test_pages_outside_the_window_may_be_gone(skv):
    c = Case(skv, skv.KV_BF16, 256, 8, 2, 16, [1000, 700], [1, 5], seed=15)
    want = c.run(S=16, W=64).clone()
    c.table[0, 1:(1000 - 64) // 16] = -1
    c.table[1, 1:(700 - 5 - 63) // 16] = 1 << 30
    assert torch.equal(c.run(S=16, W=64), want) and int(c.st.item()) == 0


@pytest.mark.parametrize("bad", [-1, 1 << 20])
def test_bad_pages_are_skipped_and_flagged(skv, bad):
    c = Case(skv, skv.KV_INT8, 256, 8, 2, 16, [200, 150], [4, 1], seed=16)
    c.run()
    want = c.out.clone()
    c.table[0, 3] = bad
    got = c.run()
    assert int(c.st.item()) == skv.DEV_RANGE
    assert torch.equal(got[4:], want[4:])
    k, v = c.values()
    t = np.array([x for x in range(200) if x // 16 != 3])
    rows = c.table[0][t // 16].astype(np.int64) * 16 + t % 16
    for i in range(4):
        m = t <= 196 + i
        for g in range(8):
            z = f64(c.q)[i, g] @ k[rows[m], g // 4].T * c.scale
            w = np.exp(z - z.max())
            w /= w.sum()
            ref, spread = w @ v[rows[m], g // 4], w @ np.abs(v[rows[m], g // 4])
            err = np.abs(f64(got)[i, g] - ref)
            assert (err <= 2.0 ** -8 * np.abs(ref) + 2 * (2.0 ** -8 + 2.0 ** -10) * (spread + np.abs(ref))).all()


def test_a_length_past_the_table_is_flagged(skv):
    c = Case(skv, skv.KV_BF16, 128, 4, 2, 16, [160, 40], [2, 2], seed=17)
    want = c.run().clone()
    c.lens = [200, 40]
    got = c.run()
    assert int(c.st.item()) == skv.DEV_RANGE
    assert torch.equal(got[2:], want[2:]) and torch.isfinite(got).all()


@pytest.mark.parametrize("starts", [[0, 5, 3, 9], [0, 5, 9, 400], [-3, 2, 4, 9], [2, 4, 6, 9]])
def test_bad_offsets_are_flagged(skv, starts):
    """Offsets that descend, pass the tokens or start below zero: flagged, nothing outside is touched."""
    c = Case(skv, skv.KV_BF16, 128, 4, 2, 16, [64, 64, 64], [3, 3, 3], seed=18)
    c.starts = np.array(starts, np.int32)
    got = c.run()
    assert got.shape[0] == 9 and torch.isfinite(got).all()
    assert (int(c.st.item()) == skv.DEV_RANGE) == (starts != [2, 4, 6, 9])


def test_query_views_and_other_streams(skv):
    c = Case(skv, skv.KV_BF16, 256, 8, 2, 16, [300, 20], [60, 3], seed=19)
    want = c.run().clone()
    wide = torch.full((63, 14, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:11] = c.q
    assert torch.equal(c.run(q=wide[:, 3:11]), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = c.run(stream=side)
    side.synchronize()
    assert torch.equal(out, want)


def test_workspace_serves_calls_of_any_size(skv):
    big = Case(skv, skv.KV_BF16, 256, 8, 2, 16, [3000, 700, 90], [1, 300, 2], seed=20)
    small = Case(skv, skv.KV_INT8, 128, 8, 2, 16, [2500], [1], seed=21)
    a, b = big.run().clone(), small.run().clone()
    n = max(skv.paged_attend_workspace_size(3, 303, 8, 2, 256), skv.paged_attend_workspace_size(1, 1, 8, 2, 128))
    ws = torch.zeros((n,), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(big.run(ws=ws), a) and torch.equal(small.run(ws=ws), b)


def test_graphs_share_a_workspace(skv):
    """Two captured calls on one workspace, replayed in turn with new lengths written in place."""
    c = Case(skv, skv.KV_BF16, 256, 8, 2, 64, [4000, 100], [1, 1], seed=22)
    d = Case(skv, skv.KV_INT8, 256, 8, 2, 64, [1500, 9], [200, 4], seed=23)
    n = max(skv.paged_attend_workspace_size(2, 2, 8, 2, 256), skv.paged_attend_workspace_size(2, 204, 8, 2, 256))
    ws = torch.zeros((n,), dtype=torch.uint8, device="cuda")
    graphs = []
    for x in (c, d):
        x.run(ws=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            x.call()
        graphs.append(graph)
    for lens in ([4000, 100], [37, 64], [2049, 1]):
        c.dev[1].copy_(torch.tensor(lens, dtype=torch.int32))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        kept, c.lens = [c.out.clone(), d.out.clone()], lens
        assert torch.equal(c.run(), kept[0]) and torch.equal(d.run(), kept[1])
        c.ws = ws
        # the graphs write the tensors of the captured call: capture again for the next lengths
        c.run(ws=ws), d.run(ws=ws)
        torch.cuda.synchronize()
        for i, x in enumerate((c, d)):
            graphs[i] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graphs[i]):
                x.call()


@pytest.mark.parametrize("kind", KINDS)
def test_repeated_calls_are_bit_identical(skv, kind):
    c = Case(skv, kind_of(skv, kind), 256, 12, 2, 16, [5000, 300, 1], [1, 200, 1], seed=24)
    want = c.run().clone()
    for _ in range(20):
        c.call()
        assert torch.equal(c.out, want)
    assert int(c.st.item()) == 0


def test_rows_past_32_bits(skv):
    """A pool whose element offsets pass 2^31: the used blocks are its last ones."""
    d, page, rows = 256, 64, (1 << 31) // 256 + 4096
    pool = torch.zeros((rows, 1, d), dtype=torch.bfloat16, device="cuda")
    g, T_, nb = gen(25), 1000, rows // page
    pool[-2048:] = randn(g, 2048, 1, d)
    table = torch.arange(nb - 1, nb - 1 - 16, -1, device="cuda", dtype=torch.int32)[None].contiguous()
    q, out, st = randn(g, 3, 4, d, scale=1.5), torch.zeros((3, 4, d), dtype=torch.bfloat16, device="cuda"), status()
    ws = torch.zeros((skv.paged_attend_workspace_size(1, 3, 4, 1, d),), dtype=torch.uint8, device="cuda")
    skv.paged_attend(skv.KV_BF16, q, pool, pool, table, page, T.dev(np.array([T_], np.int32)), d ** -0.5, out, ws,
                     q_start=T.dev(np.array([0, 3], np.int32)), status=st)
    assert int(st.item()) == 0
    lo = (nb - 16) * page
    tail = f64(pool[lo:])
    ref, spread = plain.paged_attend(f64(q), tail, tail, table.cpu().numpy() - (nb - 16), page, [T_], d ** -0.5, [0, 3],
                                     0, 0)
    tol = 2.0 ** -8 * np.abs(ref) + 2 * (2.0 ** -8 + 2.0 ** -10) * (spread + np.abs(ref))
    assert (np.abs(f64(out) - ref) <= tol).all()


@pytest.mark.parametrize("kind", KINDS)
def test_prompt_then_decode(skv, kind):
    """The operators together, as a layer uses them: a prompt in two chunks, then single tokens, each appended and
    attended over the same paged cache through the residency manager's block table."""
    d, Hq, Hkv, page, rot, S, W = 256, 8, 2, 16, 64, 8, 100
    g, total, k8 = gen(26), 237, kind == "int8"
    x = randn(g, total, Hq + 2 * Hkv, d)
    qw, kw = (1 + 0.2 * torch.randn((d,), generator=g, device="cuda") for _ in range(2))
    inv, res = freqs(rot), skv.Residency(40, page, 2, 20)
    shape = (40 * page, Hkv, d)
    pools = [torch.zeros(shape, dtype=torch.int8 if k8 else torch.bfloat16, device="cuda") for _ in range(2)]
    scales = [torch.zeros(shape[:2], dtype=torch.float16, device="cuda") if k8 else None for _ in range(2)]
    ws = torch.zeros((skv.paged_attend_workspace_size(1, 150, Hq, Hkv, d),), dtype=torch.uint8, device="cuda")
    st, outs, at = status(), [], 0
    res.add(0, 0)
    res.add(1, 50)  # another request holds blocks of the pool
    for n in [150, 80] + [1] * 7:
        res.append(0, n)
        table = T.dev(res.block_table()[:1])
        pos = torch.arange(at, at + n, device="cuda", dtype=torch.int32)
        rows = table[0].long()[pos.long() // page] * page + pos.long() % page
        y = x[at:at + n]
        q = torch.zeros((n, Hq, d), dtype=torch.bfloat16, device="cuda")
        out = torch.zeros_like(q)
        skv.norm_rope_append(y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:], pos, inv, q, *pools, q_weight=qw,
                             k_weight=kw, kv_kind=kind_of(skv, kind), k_scale=scales[0], v_scale=scales[1],
                             out_rows=rows, status=st)
        at += n
        start = None if n == 1 else T.dev(np.array([0, n], np.int32))
        skv.paged_attend(kind_of(skv, kind), q, *pools, table, page, T.dev(np.array([at], np.int32)), d ** -0.5, out,
                         ws, q_start=start, S=S, W=W, k_scale=scales[0], v_scale=scales[1], status=st)
        outs.append((q, out))
    assert int(st.item()) == 0
    q, out = (torch.cat([o[i] for o in outs]) for i in (0, 1))
    pos = torch.arange(total, device="cuda", dtype=torch.int32)
    check_norm(q, x[:, :Hq], qw, pos, inv, False)
    table = res.block_table()[:1]
    k, v = [f64(p) * (f64(s)[..., None] if k8 else 1.0) for p, s in zip(pools, scales)]
    ref, spread = plain.paged_attend(f64(q), k, v, table, page, [total], d ** -0.5, [0, total], S, W)
    tol = 2.0 ** -8 * np.abs(ref) + 2 * (2.0 ** -8 + 2.0 ** -10) * (spread + np.abs(ref))
    assert (np.abs(f64(out) - ref) <= tol).all()
    # the cache rows hold what the formula gives: int8 within half a code of the row's scale
    z, mag = plain.norm_rope(f64(x[:, Hq:Hq + Hkv]), f64(kw), 1e-6, pos.cpu().numpy(), f64(inv), False)
    t = np.arange(total)
    rows = table[0][t // page].astype(np.int64) * page + t % page
    tol = 2.0 ** -8 * np.abs(z) + 2.0 ** -19 * mag + (0.51 * f64(scales[0])[rows][..., None] if k8 else 0.0)
    assert (np.abs(k[rows] - z) <= tol).all()
    res.close()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,Hq,Hkv,page,lens,new", [
    (128, 128, 1, 8, [300, 5], [1, 3]), (256, 128, 1, 16, [40, 290], [40, 150]), (256, 100, 1, 2048, [3000], [7]),
    (128, 70, 10, 1000, [2100, 999], [300, 1]), (256, 2, 2, 24, [520], [520]),
])
def test_head_groups_and_page_sizes(skv, kind, d, Hq, Hkv, page, lens, new):
    Case(skv, kind_of(skv, kind), d, Hq, Hkv, page, lens, new, seed=30, pad=2).check()


def test_most_requests(skv):
    rng = np.random.default_rng(31)
    lens = [int(x) for x in rng.integers(0, 30, 4096)]
    Case(skv, skv.KV_BF16, 128, 2, 1, 8, lens, [min(t, 1) for t in lens], seed=31).check(S=1, W=9)
    Case(skv, skv.KV_INT8, 128, 2, 1, 8, [max(t, 1) for t in lens], [1] * 4096, seed=32).check(single=True)


def test_lengths_below_the_new_tokens(skv):
    """Tokens that stand before the cache's first row see nothing: zeros; so do all of a negative length."""
    c = Case(skv, skv.KV_BF16, 256, 8, 2, 16, [40, 3, 60, 0], [4, 9, 200, 5], seed=33)
    c.check()
    want = c.out.clone()
    assert (want[4:10] == 0).all() and (want[13:153] == 0).all() and (want[213:] == 0).all()
    c.lens = [40, 3, 60, -7]
    assert torch.equal(c.run(), want)
    c.lens = [40, -(1 << 31), 60, -7]
    got = c.run()
    assert torch.equal(got[:4], want[:4]) and (got[4:13] == 0).all() and torch.equal(got[13:], want[13:])


@pytest.mark.parametrize("kind", KINDS)
def test_a_window_as_long_as_the_table_is_none(skv, kind):
    c = Case(skv, kind_of(skv, kind), 128, 8, 2, 16, [200, 33], [130, 1], seed=34)
    want = c.run().clone()
    for W in (c.n_pages * 16, (1 << 31) - 1):
        assert torch.equal(c.run(W=W), want)


def test_two_calls_at_once(skv):
    """Two streams, a workspace each: chunks beside single tokens."""
    a = Case(skv, skv.KV_BF16, 256, 16, 2, 64, [9000], [600], seed=35)
    b = Case(skv, skv.KV_INT8, 256, 24, 4, 64, [4000, 17, 9000], [1, 1, 1], seed=36)
    want = a.run().clone(), b.run().clone()
    s = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        for x in s:
            x.wait_stream(torch.cuda.current_stream())
        out = a.run(stream=s[0]), b.run(stream=s[1])
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_captured_append(skv):
    """A captured append, replayed with new rows and positions written in place."""
    g, n, d = gen(37), 9, 128
    q, k, v = randn(g, n, 8, d), randn(g, n, 2, d), randn(g, n, 2, d)
    pos, rows = T.dev(np.arange(n, dtype=np.int32)), T.dev(np.arange(n, dtype=np.int64))
    inv = torch.logspace(0, -4, d // 2, device="cuda")
    out, kp, vp = torch.zeros_like(q), torch.zeros((64, 2, d), dtype=torch.bfloat16, device="cuda"), torch.zeros(
        (64, 2, d), dtype=torch.bfloat16, device="cuda")
    call = lambda: skv.norm_rope_append(q, k, v, pos, inv, out, kp, vp, out_rows=rows)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for shift in (5, 50):
        pos += shift
        rows += 1
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), kp.clone(), vp.clone()
        call()
        assert all(torch.equal(x, y) for x, y in zip(got, (out, kp, vp)))


def test_host_tensors_are_refused(skv):
    c = Case(skv, skv.KV_BF16, 128, 4, 2, 16, [20], [1], seed=38)
    c.run()
    for i in (0, 1):
        kept, c.dev[i] = c.dev[i], c.dev[i].cpu()
        with pytest.raises(ValueError):
            c.call()
        c.dev[i] = kept
    q = torch.zeros((1, 4, 128), dtype=torch.bfloat16)
    for at in ("q", "k"):
        x = {"q": c.q, "k": c.k[:1], at: q[:, :2] if at == "k" else q}
        with pytest.raises(ValueError):
            skv.norm_rope_append(x["q"], x["k"], None, c.dev[1], None, c.out, c.k, None)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,Hq,Hkv,B,n", [
    (256, 24, 4, 8, 8), (256, 24, 4, 3, 5), (256, 16, 1, 6, 8), (256, 128, 1, 4, 1), (256, 12, 2, 3, 4), (128, 24, 4, 8, 8),
    (128, 16, 1, 6, 8), (256, 8, 8, 2, 64),
])
def test_drafts_of_every_query_tile(skv, kind, d, Hq, Hkv, B, n):
    """From a few rows to the whole query tile of a single CTA: the more it takes, the fewer slots are left for keys."""
    rng = np.random.default_rng(40)
    Case(skv, kind_of(skv, kind), d, Hq, Hkv, 64, [int(x) for x in rng.integers(n, 1500, B)], [n] * B, seed=40).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,lens,new", [(256, [3000, 40], [1, 1]), (128, [2000, 900], [300, 5])])
def test_calls_back_to_back_see_each_other(skv, kind, d, lens, new):
    """Each call's queries are the last one's output, and its rows go over those the last one read: with the calls
    one behind the other, captured or not, as with a wait between them."""
    c = Case(skv, kind_of(skv, kind), d, 8, 2, 16, lens, new, seed=41)
    n = c.q.shape[0]
    pos, inv = torch.arange(n, device="cuda", dtype=torch.int32), torch.logspace(0, -3, 32, device="cuda")
    rows = torch.from_numpy(np.concatenate([
        c.table[b][np.arange(t - m, t) // 16].astype(np.int64) * 16 + np.arange(t - m, t) % 16
        for b, (t, m) in enumerate(zip(lens, new))])).cuda()
    c.run()
    first, pools = c.q.clone(), [x.clone() for x in (c.k, c.v)] + [None if x is None else x.clone() for x in (c.ks, c.vs)]
    x, y = torch.empty_like(c.q), torch.empty_like(c.q)

    def chain(wait):
        x.copy_(first)
        for dst, src in zip((c.k, c.v, c.ks, c.vs), pools):
            if dst is not None:
                dst.copy_(src)
        for _ in range(6):
            skv.norm_rope_append(x, x[:, 2:4], x[:, 4:6], pos, inv, y, c.k, c.v, kv_kind=c.kind, k_scale=c.ks,
                                 v_scale=c.vs, out_rows=rows, status=c.st)
            for a, b in ((y, x), (x, y), (y, x)):
                skv.paged_attend(c.kind, a, c.k, c.v, c.dev[0], 16, c.dev[1], 1.0, b, c.ws, q_start=c.dev[2],
                                 k_scale=c.ks, v_scale=c.vs, status=c.st)
                if wait:
                    torch.cuda.synchronize()
        return x.clone()

    want = chain(True)
    assert torch.isfinite(want).all() and torch.equal(chain(False), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(False)
    for _ in range(3):
        x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want)
    assert int(c.st.item()) == 0


def test_sparse_calls_behind_dense_ones(skv):
    """A sparse layer's attention on queries that came two dense calls before it, over rows just appended: queued
    without a wait between the calls as with one."""
    B, Hq, Hkv, d, page, t = 4, 16, 2, 256, 64, 5000
    c = Case(skv, skv.KV_BF16, d, Hq, Hkv, page, [t] * B, [1] * B, seed=42)
    other = Case(skv, skv.KV_BF16, d, Hq, Hkv, page, [t], [200], seed=43)
    c.run(), other.run()
    r = np.stack([c.table[b][np.arange(t - 300, t) // page] * page + np.arange(t - 300, t) % page for b in range(B)])
    rows, count = T.dev(r.astype(np.int32)), T.dev(np.full(B, 300, np.int32))
    last = torch.from_numpy(r[:, -1].astype(np.int64)).cuda()
    ws = torch.zeros((skv.attend_workspace_size(B, Hq, Hkv, d, 300),), dtype=torch.uint8, device="cuda")
    x, y = c.q.clone(), torch.zeros_like(c.q)
    out = torch.zeros((B, Hq, d), dtype=torch.float32, device="cuda")
    pos, inv = torch.arange(B, device="cuda", dtype=torch.int32), torch.logspace(0, -3, 32, device="cuda")
    pools = c.k.clone(), c.v.clone()

    def steps(wait):
        x.copy_(c.q), c.k.copy_(pools[0]), c.v.copy_(pools[1])
        got = []
        for _ in range(8):
            for call in (
                    lambda: skv.norm_rope_append(x, x[:, :2], x[:, 2:4], pos, inv, y, c.k, c.v, out_rows=last),
                    lambda: skv.paged_attend(c.kind, y, c.k, c.v, c.dev[0], page, c.dev[1], 0.1, x, c.ws, status=c.st),
                    lambda: other.call(),
                    lambda: skv.sparse_attend_decode(c.kind, x, c.k, c.v, rows, count, 0.1, out, ws, Hkv, status=c.st),
                    lambda: got.append(out.clone())):
                call()
                if wait:
                    torch.cuda.synchronize()
        return torch.stack(got)

    want = steps(True)
    assert torch.isfinite(want).all()
    for _ in range(5):
        assert torch.equal(steps(False), want)
    assert int(c.st.item()) == 0
