"""skv_move_rows against its plain form.

Tolerances, from the arithmetic.  Parts that are not turned are exact: decoding is
exact in fp32, and the encodings are IEEE divisions and roundings, so codes and
scales are compared bit by bit.  A turned value is off by at most 2^-20 of
|x_a| + |x_b|: the angle by 2^-28 (two 64-bit fractions cut to 32 bits of a turn),
the sine and cosine by two steps (2^-23), two products and their sum by 2^-24 each.
Then half a step: bf16 2^-8 of the value, int8 and int4 half the scale (the largest
value may be 2^-11 beyond the largest code, which is within the half step).  The
scale itself: fp16's half step, 2^-11, and the turned values' error.
"""
import ctypes
import mmap

import numpy as np
import pytest
import torch

import skvtest as T
from oracle import rows as plain

pytestmark = pytest.mark.gpu
ALL = ["bf16", "int8", "int4"]


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


def host(t):
    return t.detach().float().cpu().numpy() if t.dtype is torch.bfloat16 else t.detach().cpu().numpy()


def freqs(rot, theta=1e6):
    return (theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().cuda()


class Rows:
    """K and V rows in one encoding; int4 rows as a tier (K and V side by side) or in arrays of their own."""

    def __init__(self, skv, kind, rows, H, d, seed=None, tier=True, keys=True, values=True):
        self.skv, self.kind, self.H, self.d, self.tier = skv, kind, H, d, tier
        self.parts = [p for p, there in ((0, keys), (1, values)) if there]
        g = gen(seed) if seed is not None else None

        def make(shape, dtype, draw):
            return draw() if g is not None else torch.full(shape, 99, dtype=dtype, device="cuda")

        self.s = [None, None]
        if kind == "int4":
            vec = d // 2 + d // 32
            shape = (rows, H, 2, vec) if tier else (2, rows, H, vec)

            def draw():
                codes = torch.randint(0, 256, (*shape[:-1], d // 2), generator=g, device="cuda", dtype=torch.uint8)
                s = ((torch.rand((*shape[:-1], d // 64), generator=g, device="cuda") + 0.1) / 3).half()
                return torch.cat([codes, s.view(torch.uint8)], -1)

            self.all = make(shape, torch.uint8, draw)
            self.x = [self.all[:, :, p] if tier else self.all[p] for p in range(2)]
        elif kind == "int8":
            self.x = [make((rows, H, d), torch.int8, lambda: torch.randint(
                -127, 128, (rows, H, d), generator=g, device="cuda", dtype=torch.int8)) for _ in range(2)]
            self.s = [make((rows, H), torch.float16, lambda: ((torch.rand(
                (rows, H), generator=g, device="cuda") + 0.1) / 73).half()) for _ in range(2)]
        else:
            self.x = [make((rows, H, d), torch.bfloat16, lambda: torch.randn(
                (rows, H, d), generator=g, device="cuda").bfloat16()) for _ in range(2)]

    def set(self):
        skv, (k, v) = self.skv, (0 in self.parts, 1 in self.parts)
        if self.kind == "int4" and self.tier:
            return skv.tier_rows(self.all, keys=k, values=v)
        kind = {"bf16": skv.KV_BF16, "int8": skv.KV_INT8, "int4": skv.KV_INT4}[self.kind]
        x = [self.x[p] if p in self.parts else None for p in range(2)]
        return skv.row_set(kind, *x, *(self.s if self.kind == "int8" else (None, None)))

    def raw(self, p):
        """(codes or values, scales) as numpy."""
        if self.kind == "int4":
            return plain.unpack_int4(host(self.x[p]))
        return host(self.x[p]), None if self.s[p] is None else host(self.s[p])

    def bits(self, p):
        x = self.x[p].contiguous()
        return [host(x.view(torch.int16) if x.dtype is torch.bfloat16 else x)] + (
            [] if self.s[p] is None else [host(self.s[p].view(torch.int16))])

    def values(self, p):
        return plain.decode(self.kind, *self.raw(p))


def check(src, dst, before, n, src_rows, dst_rows, angle, inter):
    """dst after a move of src's rows; `before`: dst's bits then."""
    frm = np.arange(n) if src_rows is None else src_rows.cpu().numpy()
    to = np.arange(n) if dst_rows is None else dst_rows.cpu().numpy()
    keep = (frm >= 0) & (to >= 0)
    frm, to = frm[keep], to[keep]
    for p in range(2):
        untouched = np.ones(len(dst.x[p]), bool)
        if p in dst.parts:
            untouched[to] = False
        for now, then in zip(dst.bits(p), before[p]):
            np.testing.assert_array_equal(now[untouched], then[untouched])
        if p not in dst.parts:
            continue
        if p == 1 or angle is None:
            if src.kind == dst.kind:
                for now, was in zip(dst.bits(p), src.bits(p)):
                    np.testing.assert_array_equal(now[to], was[frm])
                continue
            x = src.values(p)[frm]
            if dst.kind == "bf16":
                want = host(torch.from_numpy(x).bfloat16())
                np.testing.assert_array_equal(dst.values(p)[to], want)
            else:
                codes, scale = plain.encode(dst.kind, x)
                got = dst.raw(p)
                np.testing.assert_array_equal(got[0][to], codes)
                np.testing.assert_array_equal(got[1][to], scale)
            continue
        z, mag = plain.turn(src.values(p)[frm], angle[keep], inter)
        slack = 2.0 ** -20 * mag
        got = dst.values(p)[to].astype(np.float64)
        if dst.kind == "bf16":
            assert (np.abs(got - z) <= 2.0 ** -8 * np.abs(z) + slack).all()
            continue
        top = 127 if dst.kind == "int8" else 7
        s = dst.raw(p)[1][to].astype(np.float64)
        group = z.shape[-1] if dst.kind == "int8" else 64
        zz = np.abs(z).reshape(*z.shape[:-1], -1, group)
        ss = s[..., None] if dst.kind == "int8" else s
        most = slack.reshape(zz.shape).max(-1)
        assert (np.abs(ss - zz.max(-1) / top) <= 2.0 ** -11 * zz.max(-1) / top + 1.01 * most / top + 2.0 ** -25).all()
        step = np.repeat(ss, group, -1)
        assert (np.abs(got - z) <= 0.5 * step + 1.01 * slack).all()


def move(skv, src, dst, n, rot=0, inter=False, src_rows=None, dst_rows=None, old=None, new=None, theta=(1e6, 1e6),
         status=0):
    """Moves and checks.  old, new: positions or None."""
    before = [dst.bits(p) for p in range(2)]
    f = [freqs(rot, t) if rot else None for t in theta]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    keep = Rows.__new__(Rows)
    keep.__dict__.update(src.__dict__)
    keep.x, keep.s = [t.clone() for t in src.x], [None if t is None else t.clone() for t in src.s]  # src may be dst
    skv.move_rows(src.set(), dst.set(), n, src_rows=src_rows, dst_rows=dst_rows, old_positions=old,
                  old_inv_freq=f[0] if old is not None else None, new_positions=new,
                  new_inv_freq=f[1] if new is not None else None, interleaved=inter, status=st)
    assert int(st.item()) == status
    angle = None
    if rot and 0 in src.parts and (old is not None or new is not None):
        angle = np.zeros((n, rot // 2))
        for pos, fr, sign in ((old, f[0], -1), (new, f[1], 1)):
            if pos is not None:  # each product is exact in 64 bits: 24 bits by 22
                angle += sign * pos.cpu().numpy().astype(np.float64)[:, None] * host(fr).astype(np.float64)
    check(keep, dst, before, n, src_rows, dst_rows, angle, inter)


def positions(n, seed, far=1 << 20):
    return torch.randint(0, far, (n,), generator=gen(seed), device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("src,dst", [(a, b) for a in ALL for b in ALL])
@pytest.mark.parametrize("rot,inter", [(0, False), (64, False), (64, True), (256, False), (256, True), (16, False),
                                       (144, False), (240, True)])
def test_every_encoding(skv, src, dst, rot, inter):
    n, H = 61, 3
    a, b = Rows(skv, src, 80, H, 256, seed=1), Rows(skv, dst, 70, H, 256)
    perm = torch.randperm(80, generator=gen(2), device="cuda")[:n]
    to = torch.randperm(70, generator=gen(3), device="cuda")[:n]
    move(skv, a, b, n, rot, inter, perm, to, positions(n, 4), positions(n, 5))


@pytest.mark.parametrize("src,dst", [(a, b) for a in ALL[:2] for b in ALL[:2]])
@pytest.mark.parametrize("d,H", [(64, 1), (64, 5), (64, 8), (128, 1), (128, 3), (128, 8)])
@pytest.mark.parametrize("share", [0, 1, 2])
@pytest.mark.parametrize("inter", [False, True])
def test_other_heads(skv, src, dst, d, H, share, inter):
    rot = share * d // 2
    n = 37
    a, b = Rows(skv, src, n, H, d, seed=d + H), Rows(skv, dst, n + 3, H, d)
    move(skv, a, b, n, rot, inter, None, None, positions(n, 6), positions(n, 7))


@pytest.mark.parametrize("src,dst", [("bf16", "bf16"), ("int8", "int8"), ("int4", "int8"), ("bf16", "int4")])
@pytest.mark.parametrize("n", [1, 2, 1000, 12345])
def test_numbers_of_rows(skv, src, dst, n):
    a, b = Rows(skv, src, n, 2, 256, seed=n), Rows(skv, dst, n, 2, 256)
    move(skv, a, b, n, 64, False, None, torch.randperm(n, generator=gen(n), device="cuda"), positions(n, 8), positions(n, 9))


@pytest.mark.parametrize("src,dst", [("bf16", "int8"), ("int4", "bf16"), ("int8", "int8")])
@pytest.mark.parametrize("old,new", [(True, False), (False, True), (False, False)])
def test_keys_that_were_or_stay_unrotated(skv, src, dst, old, new):
    n = 50
    a, b = Rows(skv, src, n, 2, 256, seed=11), Rows(skv, dst, n, 2, 256)
    move(skv, a, b, n, 64, False, None, None, positions(n, 12) if old else None, positions(n, 13) if new else None)


@pytest.mark.parametrize("parts", [(True, False), (False, True)])
@pytest.mark.parametrize("src,dst", [("int8", "int4"), ("int4", "int4"), ("bf16", "bf16")])
def test_keys_or_values_alone(skv, parts, src, dst):
    n = 40
    a = Rows(skv, src, n, 2, 256, seed=14, tier=False, keys=parts[0], values=parts[1])
    b = Rows(skv, dst, n, 2, 256, keys=parts[0], values=parts[1])
    move(skv, a, b, n, 96, True, None, None, positions(n, 15), positions(n, 16))


@pytest.mark.parametrize("src,dst", [("int4", "int8"), ("int8", "int4"), ("int4", "int4")])
def test_int4_arrays_with_strides(skv, src, dst):
    """Int4 rows in arrays of their own, in a tier, and in rows with room between them."""
    n, H, vec = 33, 4, 136
    a = Rows(skv, src, n, H, 256, seed=17, tier=False)
    b = Rows(skv, dst, n, H, 256, tier=False)
    for x in (a, b):
        if x.kind == "int4":
            wide = torch.full((2, n, H + 1, vec + 12), 55, dtype=torch.uint8, device="cuda")
            view = wide[:, :, :H, 4:4 + vec]
            view.copy_(x.all)
            x.x = [view[0], view[1]]
            x.wide = wide
    move(skv, a, b, n, 64, False, None, None, positions(n, 18), positions(n, 19))
    for x in (a, b):
        if x.kind == "int4":
            assert (x.wide[:, :, H] == 55).all() and (x.wide[..., :4] == 55).all() and (x.wide[..., 4 + vec:] == 55).all()


@pytest.mark.parametrize("kind", ALL)
def test_padding_and_rows_out_of_range(skv, kind):
    n = 40
    a, b = Rows(skv, kind, n, 2, 256, seed=20), Rows(skv, "int8", n, 2, 256)
    frm, to = torch.arange(n, device="cuda"), torch.arange(n, device="cuda").flip(0)
    frm[3], frm[7], to[3], to[11], to[12] = -1, -(1 << 40), 1 << 40, -1, -7
    move(skv, a, b, n, 64, False, frm, to, positions(n, 21), positions(n, 22))
    frm[20], to[25], to[26] = n, n, 1 << 40
    want = frm.clone()
    want[[20, 25, 26]] = -1
    b2 = Rows(skv, "int8", n, 2, 256)
    move(skv, a, b2, n, 64, False, want, to, positions(n, 21), positions(n, 22))
    b3 = Rows(skv, "int8", n, 2, 256)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    skv.move_rows(a.set(), b3.set(), n, src_rows=frm, dst_rows=to, old_positions=positions(n, 21), old_inv_freq=freqs(64),
                  new_positions=positions(n, 22), new_inv_freq=freqs(64), status=st)
    assert int(st.item()) == skv.DEV_RANGE
    for p in range(2):
        assert torch.equal(b3.x[p], b2.x[p]) and torch.equal(b3.s[p], b2.s[p])


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("rot,inter", [(64, False), (256, True)])
def test_turned_in_place(skv, kind, rot, inter):
    """A cache that is its own destination: other rows keep their bits, values too."""
    n, d = 300, 256
    a = Rows(skv, kind, 400, 4, d, seed=23)
    rows = torch.randperm(400, generator=gen(24), device="cuda")[:n]
    move(skv, a, a, n, rot, inter, rows, rows, positions(n, 25), positions(n, 26))


@pytest.mark.parametrize("kind,d", [(k, 256) for k in ALL] + [(k, d) for k in ALL[:2] for d in (64, 128)])
@pytest.mark.parametrize("rot,inter", [(0, False), (32, False), (64, True)])
def test_moves_in_place_one_behind_the_other(skv, kind, d, rot, inter):
    """Four moves of one cache onto itself, queued without a wait, leave the bits that the same moves from one cache to
    another leave."""
    n, rows = 3000, 4000
    a, b = Rows(skv, kind, rows, 3, d, seed=43), Rows(skv, kind, rows, 3, d, seed=43)
    other = Rows(skv, kind, rows, 3, d, seed=44)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    at = torch.randperm(rows, generator=gen(45), device="cuda")[:n]
    pos = [positions(n, 46 + i) for i in range(5)]
    f = freqs(rot) if rot else None

    def step(src, dst, i):
        skv.move_rows(src.set(), dst.set(), n, src_rows=at, dst_rows=at, old_positions=pos[i] if rot else None,
                      old_inv_freq=f, new_positions=pos[i + 1] if rot else None, new_inv_freq=f, interleaved=inter,
                      status=st)

    for i in range(4):
        step(a, a, i)
    for i in range(0, 4, 2):
        step(b, other, i)
        step(other, b, i + 1)
    assert int(st.item()) == 0
    for p in range(2):
        for x, y in zip(a.bits(p), b.bits(p)):
            np.testing.assert_array_equal(x, y)


@pytest.mark.parametrize("inter", [False, True])
def test_far_positions_lose_nothing(skv, inter):
    """Positions of two thousand millions and below zero: with frequencies that are powers of two the angles of the
    plain form are exact."""
    n, rot = 64, 64
    a, b = Rows(skv, "bf16", n, 1, 256, seed=27), Rows(skv, "bf16", n, 1, 256)
    old = torch.randint(-(1 << 31), (1 << 31) - 1, (n,), generator=gen(28), device="cuda").int()
    new = torch.randint(-(1 << 31), (1 << 31) - 1, (n,), generator=gen(29), device="cuda").int()
    f = [(2.0 ** -(torch.arange(rot // 2) % 7 + k)).float().cuda() for k in (0, 2)]
    skv.move_rows(a.set(), b.set(), n, old_positions=old, old_inv_freq=f[0], new_positions=new, new_inv_freq=f[1],
                  interleaved=inter)
    angle = host(new).astype(np.float64)[:, None] * host(f[1]) - host(old).astype(np.float64)[:, None] * host(f[0])
    z, mag = plain.turn(a.values(0), angle, inter)
    assert (np.abs(b.values(0) - z) <= 2.0 ** -8 * np.abs(z) + 2.0 ** -20 * mag).all()


def test_frequencies_of_any_kind(skv):
    """Zero, negative, subnormal, large."""
    n, rot = 16, 32
    a, b = Rows(skv, "bf16", n, 1, 64, seed=30), Rows(skv, "bf16", n, 1, 64)
    f = torch.tensor([0.0, -0.0, -1.0, 1e-42, -3e-39, 2.0 ** 20, -1024.0, 6.0, 1e-8, -0.5, 3.5, 0.125, 1e-3, 1.0, 2.0 ** -30,
                      7.0], device="cuda")
    pos = torch.arange(n, device="cuda", dtype=torch.int32)
    skv.move_rows(a.set(), b.set(), n, new_positions=pos, new_inv_freq=f)
    z, mag = plain.turn(a.values(0), host(pos).astype(np.float64)[:, None] * host(f).astype(np.float64), False)
    assert (np.abs(b.values(0) - z) <= 2.0 ** -8 * np.abs(z) + 2.0 ** -20 * mag).all()
    assert rot == 2 * len(f)


@pytest.mark.parametrize("dst", ["int8", "int4"])
@pytest.mark.parametrize("src", ALL)
def test_values_at_the_ends_of_their_ranges(skv, src, dst):
    """Zeros, subnormals, values too small or too large for a scale, infinities, NaN; scales of any size."""
    n, H, d = 300, 2, 256
    a, b = Rows(skv, src, n, H, d, seed=31), Rows(skv, dst, n, H, d)
    g = gen(32)
    if src == "bf16":
        size = torch.exp2(torch.randint(-130, 127, (n, H, 1), generator=g, device="cuda").float())
        for p in range(2):
            a.x[p] = (a.x[p].float() * size).bfloat16()
            a.x[p][:8] = 0
            for i, value in enumerate([float("inf"), float("-inf"), float("nan"), 1e-40, 3.38e38, 127 * 2.0 ** -25]):
                m = torch.rand(a.x[p].shape, generator=g, device="cuda") < 0.01
                m[:40 + 40 * i] = False
                a.x[p][m] = value
    else:
        shape = a.s[0].shape if src == "int8" else (n, H, 4)
        for p in range(2):
            s = torch.exp2(-24 + 39.9 * torch.rand(shape, generator=g, device="cuda")).half()
            s[torch.rand(shape, generator=g, device="cuda") < 0.1] = 0
            s[torch.rand(shape, generator=g, device="cuda") < 0.1] *= -1
            zero = torch.rand(shape, generator=g, device="cuda") < 0.05
            s[zero] = float("inf")
            if src == "int8":
                a.s[p] = s
                a.x[p][zero] = 0
            else:
                a.x[p][..., 128:] = s.view(torch.uint8).view(n, H, 8)
                codes = a.x[p][..., :128].reshape(n, H, 4, 32)
                codes[zero] = 0
                a.x[p][..., :128] = codes.reshape(n, H, 128)
    if src == dst:
        return move(skv, a, b, n)
    with np.errstate(all="ignore"):
        move(skv, a, b, n)


def test_the_encodings_are_the_librarys_own(skv):
    """bf16 rows to int8 and int4 as the library's quantising calls write them."""
    n, H, d = 200, 4, 256
    a = Rows(skv, "bf16", n, H, d, seed=33)
    b, c = Rows(skv, "int8", n, H, d), Rows(skv, "int4", n, H, d)
    skv.move_rows(a.set(), b.set(), n)
    skv.move_rows(a.set(), c.set(), n)
    for p in range(2):
        q, s = torch.zeros_like(b.x[p]), torch.zeros_like(b.s[p])
        skv.quantize_int8_rows(a.x[p], q, s)
        assert torch.equal(q, b.x[p]) and torch.equal(s, b.s[p])
        out = torch.zeros((n, H, 136), dtype=torch.uint8, device="cuda")
        skv.quantize_int4_rows(a.x[p], out, H * 136, 136)
        assert torch.equal(out, c.x[p])


def test_a_key_moved_is_the_key_appended_there(skv):
    """Appended at one position and moved to another, against appended there: both within their roundings of the fp64
    key.  With bf16 rows each is off by 2^-8 of a value once more."""
    n, H, d, rot = 100, 2, 256, 64
    k = torch.randn((n, H, d), generator=gen(34), device="cuda").bfloat16()
    old, new, f = positions(n, 35), positions(n, 36), freqs(rot)
    rows = [torch.zeros_like(k) for _ in range(3)]
    skv.norm_rope_append(None, k, None, old, f, None, rows[0], None)
    skv.norm_rope_append(None, k, None, new, f, None, rows[1], None)
    skv.move_rows(skv.row_set(skv.KV_BF16, rows[0], None), skv.row_set(skv.KV_BF16, rows[2], None), n, old_positions=old,
                  old_inv_freq=f, new_positions=new, new_inv_freq=f)
    x = host(k).astype(np.float64)
    z, mag = plain.turn(x, host(new).astype(np.float64)[:, None] * host(f).astype(np.float64), False)
    mag = np.maximum(mag, np.abs(z))
    # the first row's rounding, 2^-8 of its values, turned: at most 2^-8 * sqrt(2) of the pair's length
    assert (np.abs(host(rows[1]) - z) <= 2.0 ** -8 * np.abs(z) + 2.0 ** -19 * mag).all()
    assert (np.abs(host(rows[2]) - z) <= 2.0 ** -8 * np.abs(z) + 1.5 * 2.0 ** -8 * mag).all()


def test_through_a_registered_host_tier(skv):
    """int8 rows spilled to int4 rows in host memory and brought back as bf16 rows, through the tier's alias."""
    n, H, d = 500, 4, 256
    vec = d // 2 + d // 32
    nbytes = n * H * 2 * vec
    buf = mmap.mmap(-1, nbytes)
    addr = ctypes.addressof(ctypes.c_char.from_buffer(buf))
    alias = skv.host_register(addr, nbytes)
    try:
        tier = skv.HostView(alias, (n, H, 2, vec), 1)
        a, b, c = Rows(skv, "int8", n, H, d, seed=37), Rows(skv, "bf16", n, H, d), Rows(skv, "int4", n, H, d)
        skv.move_rows(a.set(), skv.tier_rows(tier), n)
        skv.move_rows(a.set(), c.set(), n)
        torch.cuda.synchronize()
        seen = np.frombuffer(buf, np.uint8).reshape(n, H, 2, vec).copy()
        np.testing.assert_array_equal(seen, host(c.all))
        skv.move_rows(skv.tier_rows(tier), b.set(), n)
        check(c, b, [b.bits(p) for p in range(2)], n, None, None, None, False)
        torch.cuda.synchronize()
    finally:
        skv.host_unregister(addr)


def test_other_streams_and_graphs(skv):
    """On another stream, and captured and replayed after rows and positions have changed."""
    n, H, d, rot = 200, 2, 128, 128
    a, b = Rows(skv, "bf16", n, H, d, seed=38), Rows(skv, "int8", n, H, d)
    rows, old, new, f = torch.arange(n, device="cuda"), positions(n, 39), positions(n, 40), freqs(rot)
    sets = a.set(), b.set()

    def call(stream=None):
        skv.move_rows(*sets, n, src_rows=rows, dst_rows=rows, old_positions=old, old_inv_freq=f, new_positions=new,
                      new_inv_freq=f, stream=stream)

    def result():
        torch.cuda.synchronize()
        return [t.clone() for t in (*b.x, *b.s)]

    call()
    want = result()
    for t in (*b.x, *b.s):
        t.zero_()
    torch.cuda.synchronize()
    call(torch.cuda.Stream())
    assert all(torch.equal(x, y) for x, y in zip(result(), want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    new.copy_(positions(n, 41))
    rows.copy_(rows.flip(0))
    call()
    want = result()
    for t in (*b.x, *b.s):
        t.zero_()
    g.replay()
    assert all(torch.equal(x, y) for x, y in zip(result(), want))


@pytest.mark.parametrize("src,dst", [("bf16", "int8"), ("int8", "bf16")])
def test_rows_past_32_bits(skv, src, dst):
    """Rows more than 2^32 bytes into their pools."""
    H, d, n = 8, 256, 20
    big = (1 << 21) + 1000 if src == "bf16" else (1 << 22) + 1000
    a = Rows(skv, src, n, H, d, seed=42)
    far = Rows(skv, src, 1, H, d)
    far.x = [torch.zeros((big, H, d), dtype=a.x[0].dtype, device="cuda") for _ in range(2)]
    far.s = [None if s is None else torch.zeros((big, H), dtype=s.dtype, device="cuda") for s in a.s]
    rows = torch.arange(n, device="cuda") * 49 + big - 1000
    skv.move_rows(a.set(), far.set(), n, dst_rows=rows)
    for p in range(2):
        assert torch.equal(far.x[p][rows], a.x[p]) and (a.s[p] is None or torch.equal(far.s[p][rows], a.s[p]))
    b, c = Rows(skv, dst, n, H, d), Rows(skv, dst, n, H, d)
    skv.move_rows(far.set(), b.set(), n, src_rows=rows)
    skv.move_rows(a.set(), c.set(), n)
    for p in range(2):
        assert torch.equal(b.x[p], c.x[p]) and (b.s[p] is None or torch.equal(b.s[p], c.s[p]))
