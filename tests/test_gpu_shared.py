"""skv_shared_attend against its plain fp64 form.

Tolerance, from the arithmetic (half a step of bf16 is 2^-8 of the value): weights
rounded to bf16 and divided by their rounded sums change the mean by at most
2 * 2^-8 of sum w |v| + |out|; a logit's fp32 error below 2^-10 (d products of a few
units, 2^-24 each) the same way, the fp32 factors that join two parts (2^-22) far
within it; and 2^-8 |out| for the output's rounding.
"""
import ctypes
import math
import os
import subprocess
import types

import numpy as np
import pytest
import torch

import skvtest as T
from oracle import shared as plain

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "int8"]


@pytest.fixture(scope="module")
def skv():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from sparse_kv_long_gb300 import _build
    _build.build()
    import sparse_kv_long_gb300 as m
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def tolerance(ref, spread):
    return 2.0 ** -8 * np.abs(ref) + 2 * (2.0 ** -8 + 2.0 ** -10) * (spread + np.abs(ref))


class Case:
    """Requests behind shared prefixes over one pool; rows that belong to no token hold NaN and infinities."""

    def __init__(self, skv, kind, d, Hq, Hkv, page, start, prefix, lens, new, seed, first=0, pad=0, extra_pages=0):
        self.skv, self.kind, self.d, self.Hq, self.Hkv, self.page = skv, kind, d, Hq, Hkv, page
        self.start, self.prefix, self.lens = np.array(start, np.int32), list(prefix), list(lens)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        need = [-(-t // page) for t in self.prefix + self.lens]
        blocks = sum(need) + 3
        perm = rng.permutation(blocks).astype(np.int32)
        owned = np.zeros(blocks * page, bool)

        def table(counts, lengths, at):
            x = np.full((len(counts), max([1, *counts]) + extra_pages), -1, np.int32)
            for i, (c, t) in enumerate(zip(counts, lengths)):
                x[i, :c] = perm[at:at + c]
                at += c
                s = np.arange(t)
                owned[x[i][s // page].astype(np.int64) * page + s % page] = True
            return x, at

        m = len(self.prefix)
        self.ptable, at = table(need[:m], self.prefix, 0)
        self.table, _ = table(need[m:], self.lens, at)
        self.owned = torch.from_numpy(owned).cuda()
        rows, none = blocks * page, ~self.owned

        def randn(*shape, scale=1.0):
            return (torch.randn(shape, generator=g, device="cuda") * scale).bfloat16()

        if kind == skv.KV_INT8:
            self.k, self.v = (torch.randint(-127, 128, (rows, Hkv, d), generator=g, device="cuda", dtype=torch.int8)
                              for _ in range(2))
            self.ks, self.vs = (((torch.rand((rows, Hkv), generator=g, device="cuda") + 0.5) / 73.3).half()
                                for _ in range(2))
            self.ks[none], self.vs[none] = float("nan"), float("inf")
        else:
            self.k, self.v, self.ks, self.vs = randn(rows, Hkv, d), randn(rows, Hkv, d), None, None
            self.k[none], self.v[none] = float("nan"), float("inf")
        self.starts = (first + np.concatenate([[0], np.cumsum(new)])).astype(np.int32)
        self.q = randn(int(self.starts[-1]) + pad, Hq, d, scale=1.5)
        self.scale = d ** -0.5

    def values(self):
        k, v = f64(self.k), f64(self.v)
        if self.ks is not None:
            with np.errstate(invalid="ignore"):
                k, v = k * f64(self.ks)[..., None], v * f64(self.vs)[..., None]
        return k, v

    def size(self, n):
        return self.skv.shared_attend_workspace_size(len(self.lens), len(self.prefix), n, self.Hq, self.Hkv, self.d)

    def run(self, single=False, q=None, ws=None, stream=None, out=None):
        skv, q = self.skv, self.q if q is None else q
        n = q.shape[0]
        self.out = torch.full((n, self.Hq, self.d), 123.0, dtype=torch.bfloat16, device="cuda") if out is None else out
        self.ws = torch.full((self.size(n),), 0x7F, dtype=torch.uint8, device="cuda") if ws is None else ws
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
        i32 = lambda x: T.dev(np.array(x, np.int32))  # noqa: E731
        self.dev = dict(group_start=i32(self.start), prefix_table=T.dev(self.ptable) if self.prefix else None,
                        prefix_lengths=i32(self.prefix), block_table=T.dev(self.table), lengths=i32(self.lens),
                        q_start=None if single else i32(self.starts))
        self.call = lambda stream=None: skv.shared_attend(
            self.kind, q, self.k, self.v, page=self.page, softmax_scale=self.scale, out=self.out, workspace=self.ws,
            k_scale=self.ks, v_scale=self.vs, status=self.st, stream=stream, **self.dev)
        self.call(stream)
        return self.out

    def reference(self):
        return plain.shared_attend(f64(self.q), *self.values(), self.start, self.ptable, self.prefix, self.table,
                                   self.page, self.lens, self.scale, self.starts)

    def check(self, status=0, **kw):
        got = f64(self.run(**kw))
        assert int(self.st.item()) == status
        ref, spread = self.reference()
        a, b = int(self.starts[0]), int(self.starts[-1])
        assert (got[:a] == 123).all() and (got[b:] == 123).all()  # padding is left as it was
        got, ref, spread = got[a:b], ref[a:b], spread[a:b]
        assert np.isfinite(got).all()
        worst = float((np.abs(got - ref) / np.maximum(tolerance(ref, spread), 1e-300)).max())
        assert worst <= 1, worst


def kind_of(skv, name):
    return skv.KV_INT8 if name == "int8" else skv.KV_BF16


HEADS = [(256, 24, 4, 16), (256, 16, 2, 64), (128, 8, 8, 8), (128, 32, 8, 48), (256, 5, 1, 128), (128, 128, 1, 256),
         (256, 7, 7, 24)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,Hq,Hkv,page", HEADS)
def test_single_tokens(skv, kind, d, Hq, Hkv, page):
    """Groups of none, one and several requests, prefixes and own keys from none to some tiles, requests outside."""
    lens = [1, 2, 63, 64, 65, 0, 129, 300, 1, 17, 0, 40, 128, 5]
    start = [1, 4, 4, 5, 9, 10, 12]
    prefix = [63, 64, 1, 200, 0, 129]
    c = Case(skv, kind_of(skv, kind), d, Hq, Hkv, page, start, prefix, lens, [1] * len(lens), seed=d + Hq, extra_pages=1)
    c.check(single=True)
    c.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,Hq,Hkv,page", [(256, 24, 4, 16), (128, 8, 8, 8), (128, 32, 8, 48), (256, 6, 1, 40),
                                           (256, 100, 1, 32)])
def test_chunks(skv, kind, d, Hq, Hkv, page):
    """Ragged chunks behind prefixes: no token, one, some, more than the request's own keys; padding on both sides."""
    lens = [10, 1, 5, 130, 70, 64, 0, 90]
    new = [0, 1, 5, 130, 7, 70, 3, 33]
    Case(skv, kind_of(skv, kind), d, Hq, Hkv, page, [0, 3, 7], [130, 257], lens, new, seed=d + Hq + 1, first=2, pad=5,
         extra_pages=2).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,B,P,n", [(256, 3, 5000, 1), (128, 2, 9001, 1), (256, 4, 4097, 3), (128, 9, 6000, 2),
                                     (256, 40, 3001, 1), (128, 70, 2500, 1), (256, 2, 3000, 90), (128, 3, 2049, 70)])
def test_long_prefixes_are_cut(skv, kind, d, B, P, n):
    """Few and many rows over a long prefix, as single CTAs and as pairs: the prefix's keys are split and joined with
    the requests' own."""
    rng = np.random.default_rng(P)
    lens = [int(x) + n for x in rng.integers(0, 200, B)]
    c = Case(skv, kind_of(skv, kind), d, 8, 2, 64, [0, B], [P], lens, [n] * B, seed=P)
    c.check(single=n == 1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,groups,n", [(40, 5, 1), (24, 2, 3), (100, 9, 1), (12, 3, 40), (33, 33, 2)])
def test_ragged_batches(skv, kind, B, groups, n):
    """Prefixes and own keys of all lengths, each item cut anywhere."""
    rng = np.random.default_rng(B + n)
    lens = [int(x) for x in np.exp(rng.uniform(0, math.log(1500 if n < 40 else 300), B))]
    new = [min(n, t) for t in lens]
    inner = np.sort(rng.choice(np.arange(1, B), groups - 1, replace=False))
    prefix = [int(x) for x in np.exp(rng.uniform(0, math.log(2000), groups))]
    c = Case(skv, kind_of(skv, kind), 256 if n == 1 else 128, 8, 2, 16, [0, *inner, B], prefix, lens, new, seed=B)
    c.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,new,single", [([1, 700, 64, 300], [1] * 4, True), ([700, 300, 5], [200, 3, 5], False)])
def test_without_prefixes_it_is_the_paged_attention(skv, kind, lens, new, single):
    """No groups at all (arrays left out or empty), and groups whose prefixes are empty."""
    c = Case(skv, kind_of(skv, kind), 256, 8, 2, 16, [0], [], lens, new, seed=5)
    c.check(single=single)
    c.dev["group_start"] = c.dev["prefix_lengths"] = None
    want = c.out.clone()
    c.call()
    assert torch.equal(c.out, want)
    ws = torch.zeros((skv.paged_attend_workspace_size(len(lens), c.q.shape[0], 8, 2, 256),), dtype=torch.uint8, device="cuda")
    got = torch.zeros_like(want)
    skv.paged_attend(c.kind, c.q, c.k, c.v, c.dev["block_table"], 16, c.dev["lengths"], c.scale, got, ws,
                     q_start=c.dev["q_start"], k_scale=c.ks, v_scale=c.vs)
    err, tol = np.abs(f64(got) - f64(want)), tolerance(*c.reference())
    assert (err <= 2 * tol).all()
    Case(skv, kind_of(skv, kind), 256, 8, 2, 16, [0, 1, len(lens)], [0, 0], lens, new, seed=5).check(single=single)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,B,groups,P,top", [(256, 70, 1, 5000, 3000), (256, 45, 1, 700, 9), (128, 150, 2, 1500, 2500),
                                               (256, 64, 1, 129, 5000), (128, 200, 1, 1, 40)])
def test_pairs_share_out_single_tokens(skv, kind, d, B, groups, P, top):
    """Many tokens behind a prefix run as pairs: the prefix's pieces are dealt out, the requests' own keys lie in a row
    that the pairs take stretches of, cut anywhere; some requests have none."""
    rng = np.random.default_rng(B + P)
    lens = [int(x) - 1 for x in np.exp(rng.uniform(0, math.log(top), B - 1))] + [top]
    inner = [B // 3] if groups == 2 else []
    prefix = [P] + [P // 2 + 1] * (groups - 1)
    # a wide table, as a server keeps for its longest prefix: pairs at 256 dims, single CTAs at 128
    c = Case(skv, kind_of(skv, kind), d, 8, 1, 64, [0, *inner, B - 2], prefix, lens, [1] * B, seed=B, extra_pages=512)
    c.check(single=True)
    c.check()
    c = Case(skv, kind_of(skv, kind), d, 8, 1, 64, [0, *inner, B - 2], prefix, lens, [1] * B, seed=B)
    c.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,new,start,prefix", [
    ([300, 300, 290], [300, 300, 290], [0, 3], [900]),       # whole chunks: one by one
    ([40, 33, 50, 41], [35, 33, 37, 36], [0, 4], [2000]),    # parts of tiles: together
    ([600, 3, 1, 1, 200], [500, 3, 1, 1, 200], [0, 1, 4], [129, 700]),
    ([200] * 40, [9] * 40, [0, 39], [300]),
])
def test_chunks_together_and_one_by_one(skv, kind, lens, new, start, prefix):
    c = Case(skv, kind_of(skv, kind), 256, 12, 2, 16, start, prefix, lens, new, seed=len(lens), first=1, pad=2)
    c.check()


FORMS = [([700, 64, 1, 300], [1] * 4, True), ([90, 20, 200], [3, 5, 7], False), ([300, 90, 100], [250, 90, 60], False)]


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("lens,new,single", FORMS)
def test_value_rows_of_zeros_and_scales_of_every_size(skv, d, lens, new, single):
    """int8: an all-zero value row has a zero scale and its weight counts; scales from the smallest subnormal to the
    largest number, in the prefix and in the requests' own rows."""
    for seed, lo, hi, share in ((90, -7.0, -6.0, 0.5), (91, -7.0, -6.0, 1.0), (92, -24.0, 15.9, 0.1), (93, -24.0, -20.0, 0.1),
                                (94, 10.0, 15.9, 0.1)):
        c = Case(skv, skv.KV_INT8, d, 8, 2, 16, [0, 2], [500], lens, new, seed=seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rand = lambda: torch.rand(c.vs.shape, generator=g, device="cuda")  # noqa: E731
        scale = torch.exp2(lo + (hi - lo) * rand()).half()
        scale = torch.where(rand() < 0.2, -scale, scale)
        scale[rand() < share] = 0
        c.v[(scale == 0) & c.owned[:, None]] = 0
        c.vs = torch.where(c.owned[:, None], scale, c.vs)
        ks = torch.exp2(-24.0 + 18.0 * rand()).half()
        ks[rand() < 0.1] = 0
        c.ks = torch.where(c.owned[:, None], ks, c.ks)
        c.check(single=single)
        if share == 1.0:
            assert (c.out == 0).all()


def test_a_prefix_of_several_groups_and_of_a_request(skv):
    """The same pages as the prefix of two groups and as the first pages of another request's own keys."""
    c = Case(skv, skv.KV_INT8, 256, 8, 2, 16, [0, 2, 4], [320, 320], [5, 40, 7, 1, 330], [1, 3, 2, 1, 4], seed=6)
    c.ptable[1] = c.ptable[0]
    c.table[4, :20] = c.ptable[0, :20]
    c.check()


@pytest.mark.parametrize("kind", KINDS)
def test_peaks_in_either_part(skv, kind):
    """Logits whose largest is hundreds above the rest, in the prefix for some tokens and in their own keys for
    others: the other part vanishes."""
    c = Case(skv, kind_of(skv, kind), 256, 4, 1, 16, [0, 3], [400], [50, 60, 70], [1, 1, 1], seed=7)
    for b, (pages, t) in enumerate([(c.ptable[0], 7), (c.table[1], 13), (c.ptable[0], 399)]):
        r = int(pages[t // 16]) * 16 + t % 16
        if kind == "int8":
            c.ks[r] = 0.2
        else:
            c.k[r] = 6 * c.q[b, 0]
    c.check(single=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("part", ["prefix", "own"])
@pytest.mark.parametrize("P,n", [(300, 1), (6000, 1), (700, 60)])
def test_values_that_are_not_finite(skv, kind, part, P, n):
    """A NaN in a value reaches the tokens that see it, wherever it lies, and no others; the rest is as without it."""
    B = 3
    c = Case(skv, kind_of(skv, kind), 256, 4, 1, 16, [0, 2], [P], [n + 40] * B, [n] * B, seed=8)
    clean = c.run(single=n == 1).clone()
    pages, t = (c.ptable[0], P - 2) if part == "prefix" else (c.table[1], 40 + n // 2)
    r, col = int(pages[t // 16]) * 16 + t % 16, 77
    if kind == "int8":
        c.vs[r] = float("nan")
    else:
        c.v[r, 0, col] = float("nan")
    got = c.run(single=n == 1)
    tok = torch.arange(B * n, device="cuda")
    sees = tok < 2 * n if part == "prefix" else (tok >= n) & (tok < 2 * n) & (tok - n + 40 >= t)
    assert sees.any() and torch.isnan(got[sees][..., col]).all()
    assert torch.equal(got[~sees], clean[~sees])
    if kind == "bf16":
        keep = torch.arange(256, device="cuda") != col
        assert torch.equal(got[..., keep], clean[..., keep])


@pytest.mark.parametrize("bad", [-1, 1 << 20])
@pytest.mark.parametrize("n", [1, 40])
def test_bad_pages_are_skipped_and_flagged(skv, bad, n):
    for where in ("ptable", "table"):
        c = Case(skv, skv.KV_INT8, 256, 8, 2, 16, [0, 2], [200], [150, 90, 60], [n] * 3, seed=9)
        getattr(c, where)[0, 2] = bad
        c.check(single=n == 1, status=skv.DEV_RANGE)


def test_lengths_past_the_tables_are_flagged(skv):
    for which in ("prefix", "lens"):
        c = Case(skv, skv.KV_BF16, 128, 4, 2, 16, [0, 1, 2], [160, 32], [40, 48], [2, 2], seed=10)
        want = c.run().clone()
        getattr(c, which)[0 if which == "prefix" else 1] += 100
        got = c.run()
        assert int(c.st.item()) == skv.DEV_RANGE and torch.isfinite(got).all()
        other = slice(2, 4) if which == "prefix" else slice(0, 2)
        assert torch.equal(got[other], want[other])


def test_negative_lengths_are_empty(skv):
    c = Case(skv, skv.KV_BF16, 128, 4, 2, 16, [0, 1, 2], [160, 32], [40, 48], [2, 2], seed=11)
    c.prefix[1], c.lens[0] = -5, -1
    c.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [3, 90])
@pytest.mark.parametrize("starts,group_start", [
    ([0, 5, 3, 9], None), ([0, 5, 9, 400], None), ([-3, 2, 4, 9], None), ([0, 9, 0, 9], None), (None, [0, 2, 1]),
    (None, [0, 1, 4]), (None, [-1, 1, 3]), (None, [2, 0, 3]), (None, [0, 1 << 30, 3]), ([0, 5, 3, 9], [2, 0, 3]),
])
def test_offsets_out_of_order_write_nothing(skv, kind, n, starts, group_start):
    c = Case(skv, kind_of(skv, kind), 128, 8, 2, 16, [0, 1, 3], [100, 700], [64, 700, 64], [n] * 3, seed=12)
    want = c.run().clone()
    good = c.starts.copy(), c.start.copy()
    if starts is not None:
        c.starts = np.array([x * n // 3 if x < 100 else x for x in starts], np.int32)
    if group_start is not None:
        c.start = np.array(group_start, np.int32)
    got = c.run(ws=c.ws)
    assert int(c.st.item()) == skv.DEV_RANGE and (got == 123).all()
    c.starts, c.start = good
    assert torch.equal(c.run(ws=c.ws), want) and int(c.st.item()) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 3, 90])
@pytest.mark.parametrize("group_start", [[0, -1, 3], [-1, 1, 3], [-2, -1, 3], [0, -(1 << 30), 3], [-(1 << 30), 1, 3],
                                         [-(1 << 31), 2, 3], [1, -(1 << 31), (1 << 31) - 1]])
def test_groups_that_begin_before_the_batch_write_nothing(skv, kind, n, group_start):
    c = Case(skv, kind_of(skv, kind), 256, 8, 2, 16, [0, 1, 3], [100, 700], [164, 700, 64], [n] * 3, seed=33)
    want = c.run().clone()
    good, c.start = c.start, np.array(group_start, np.int32)
    got = c.run(ws=c.ws)
    assert int(c.st.item()) == skv.DEV_RANGE and (got == 123).all()
    c.start = good
    assert torch.equal(c.run(ws=c.ws), want) and int(c.st.item()) == 0


def test_query_views_streams_and_output_in_their_place(skv):
    c = Case(skv, skv.KV_BF16, 256, 8, 2, 16, [0, 2], [700], [300, 20, 9], [60, 3, 1], seed=13)
    want = c.run().clone()
    wide = torch.full((64, 14, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:11] = c.q
    assert torch.equal(c.run(q=wide[:, 3:11]), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = c.run()
    b = c.run(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    for single in (True, False):
        c = Case(skv, skv.KV_INT8, 256, 8, 2, 16, [0, 2], [5000], [300, 20, 9], [1, 1, 1], seed=14)
        want = c.run(single=single).clone()
        q = c.q.clone()
        assert torch.equal(c.run(single=single, q=q, out=q), want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 50])
def test_captured_and_replayed_with_other_lengths(skv, kind, n):
    """A captured call replayed after its lengths, groups and tables have changed on the device; two graphs on one
    workspace, one after the other."""
    cases = [Case(skv, kind_of(skv, kind), 256, 8, 2, 16, s, p, lens, [n] * 4, seed=20 + i, extra_pages=200)
             for i, (s, p, lens) in enumerate([([0, 4], [2000], [60, 70, 80, 90]), ([1, 3], [50], [900, 51, 52, 300])])]
    want = [c.run(single=n == 1).clone() for c in cases]
    c = cases[0]
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(torch.cuda.current_stream())
        graphs.append(g)
    everything = [t for t in (*c.dev.values(), c.k, c.v, c.ks, c.vs, c.q) if t is not None]
    kept = [t.clone() for t in everything]
    other = [t for t in (*cases[1].dev.values(), *(getattr(cases[1], x) for x in ("k", "v", "ks", "vs", "q"))) if t is not None]
    for i in (0, 1, 0):
        for to, src in zip(everything, other if i else kept):
            both = tuple(slice(0, min(x, y)) for x, y in zip(to.shape, src.shape))  # tables and pools are long enough
            to[both] = src[both]
        for g in graphs:
            c.out.fill_(123)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(c.out, want[i])


def test_calls_of_many_sizes_queued_on_one_workspace(skv):
    """Calls of changing shapes one behind the other without a wait; results do not change from run to run."""
    cases = [Case(skv, kind_of(skv, k), d, 8, 2, 16, s, p, lens, new, seed=30 + i) for i, (k, d, s, p, lens, new) in enumerate([
        ("bf16", 256, [0, 3], [9000], [30, 1, 700], [1, 1, 1]), ("int8", 256, [0, 1, 3], [700, 20], [700, 500, 3], [2, 3, 1]),
        ("bf16", 128, [0, 2], [4000], [300, 200], [200, 190]), ("int8", 128, [1, 2], [64], [3, 6000, 5], [1, 1, 1]),
        ("int8", 256, [0, 2], [900], [80, 90], [80, 20])])]
    ws = torch.full((max(c.size(c.q.shape[0]) for c in cases),), 0x7F, dtype=torch.uint8, device="cuda")
    want = []
    for c in cases:
        want.append(c.run(ws=ws).clone())
        torch.cuda.synchronize()
    for _ in range(20):
        for c in cases:
            c.out.fill_(123)
        for c in cases + cases[::-1]:
            c.call()
        torch.cuda.synchronize()
        assert all(torch.equal(c.out, w) for c, w in zip(cases, want))
    assert all(int(c.st.item()) == 0 for c in cases)


@pytest.mark.parametrize("kind,new,start,prefix", [
    ("bf16", [1] * 4096, [0] + list(range(1, 4096)) + [4096], [5, 0, 64, 17] * 1024),  # a group for each request
    ("int8", [1, 0, 2, 1] * 1024, [0, 2000, 4096], [100, 130]),
    ("bf16", [3] * 4000, list(range(0, 4001, 40)), [70] * 100),
])
def test_the_largest_batches(skv, kind, new, start, prefix):
    """4096 requests and 4096 groups: plans of many windows, as single CTAs and as pairs."""
    lens = [m + i % 5 for i, m in enumerate(new)]
    for wide in (0, 2100):
        if wide and len(prefix) > 1000:
            continue
        c = Case(skv, kind_of(skv, kind), 256, 2, 1, 16, start, prefix, lens, new, seed=60, extra_pages=wide)
        got = f64(c.run(single=all(m == 1 for m in new)))
        assert int(c.st.item()) == 0
        tok = np.random.default_rng(0).choice(len(got), 300, replace=False)
        b = np.searchsorted(c.starts, tok, side="right") - 1
        k, v = c.values()
        for t, r in zip(tok, b):  # a request at a time: the plain form of one token
            m, g = int(c.starts[r + 1] - c.starts[r]), int(np.searchsorted(c.start, r, side="right") - 1)
            own = lens[r] - m + int(t - c.starts[r]) + 1
            ref, spread = plain.shared_attend(f64(c.q)[t:t + 1], k, v, [0, 1], c.ptable[g:g + 1], [prefix[g]], c.table[r:r + 1], 16,
                                              [own], c.scale, [0, 1])
            assert (np.abs(got[t] - ref[0]) <= tolerance(ref, spread)[0]).all()


@pytest.mark.parametrize("kind", KINDS)
def test_pages_past_32_bits(skv, kind):
    """Pages more than 2^32 bytes into their pools: the same bits as from the first ones."""
    for n in (1, 70):
        c = Case(skv, kind_of(skv, kind), 256, 16, 8, 16, [0, 2], [300], [n + 20] * 3, [n] * 3, seed=70)
        want, rows = c.run().clone(), c.k.shape[0]
        first = ((1 << 32) // (8 * 256 * c.k.element_size()) // 16 + 7) * 16
        for name in ("k", "v", "ks", "vs"):
            x = getattr(c, name)
            if x is not None:
                far = torch.zeros((first + rows, *x.shape[1:]), dtype=x.dtype, device="cuda")
                far[first:] = x
                setattr(c, name, far)
        for x in (c.ptable, c.table):
            x[x >= 0] += first // 16
        assert torch.equal(c.run(), want) and int(c.st.item()) == 0
        del c


def test_two_streams_at_once(skv):
    """Calls on two streams with a workspace each."""
    cases = [Case(skv, skv.KV_BF16, 256, 8, 2, 16, [0, 3], [3000 + 500 * i], [30, 1, 400], [1, 1, 1], seed=40 + i)
             for i in range(2)]
    want = [c.run().clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for c in cases:
        c.out.fill_(123)
    torch.cuda.synchronize()
    for _ in range(30):
        for c, s in zip(cases, streams):
            c.call(s)
    torch.cuda.synchronize()
    assert all(torch.equal(c.out, w) and int(c.st.item()) == 0 for c, w in zip(cases, want))


# ---------------------------------------------------------------------------
# waits that give up
# ---------------------------------------------------------------------------

@pytest.fixture(scope="module")
def hasty(skv, tmp_path_factory):
    """The attention built so that a wait gives up after its first look, in place of the library's."""
    from sparse_kv_long_gb300 import _build
    so = str(tmp_path_factory.mktemp("hasty") / "libhasty.so")
    cmd = [_build.nvcc(), *_build.ARCH, *_build.FLAGS, "-DSKV_PAGED_LOOKS=0", "-shared",
           os.path.join(_build.CSRC, "shared.cu"), "-o", so]
    subprocess.run(cmd, check=True, capture_output=True)
    lib, usual = ctypes.CDLL(so), skv.lib()
    names = ("skv_shared_attend", "skv_shared_attend_workspace_size")
    for name in names:
        f, u = getattr(lib, name), getattr(usual, name)
        f.argtypes, f.restype = u.argtypes, u.restype
    return types.SimpleNamespace(**{name: getattr(lib, name) for name in names})


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,P,lens,new,single,wide", [
    (256, 9000, [20, 2000, 30], [1, 1, 1], True, 0), (128, 20000, [30], [3], False, 0), (256, 3000, [30] * 9, [8] * 9, False, 0),
    (128, 9000, [300, 300], [300, 300], False, 0), (256, 9000, [20, 900, 1, 0] * 12, [1] * 48, True, 2048),
])
def test_waits_that_give_up(skv, hasty, monkeypatch, kind, d, P, lens, new, single, wide):
    """A call whose waits give up sets SKV_DEV_TIMEOUT and touches nothing but its tokens' output and its workspace,
    whatever that held; the next call on the same buffers is right."""
    c = Case(skv, kind_of(skv, kind), d, 8, 2, 16, [0, len(lens)], [P], lens, new, seed=50, pad=0 if single else 3,
             extra_pages=wide)
    want = c.run(single=single).clone()
    need = c.ws.numel()
    ws = torch.full((need + 4096,), 0x7F, dtype=torch.uint8, device="cuda")
    with monkeypatch.context() as m:
        m.setattr(skv, "_lib", hasty)
        got = c.run(single=single, ws=ws[:need])
        torch.cuda.synchronize()
    assert int(c.st.item()) == skv.DEV_TIMEOUT
    assert (got[int(c.starts[-1]):] == 123).all() and (ws[need:] == 0x7F).all()
    assert torch.equal(c.run(single=single, ws=ws[:need]), want) and int(c.st.item()) == 0
