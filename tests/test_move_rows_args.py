"""Refusals of skv_move_rows: decided on the host, before anything is launched,
so they run without a GPU; and the plain encodings against the oracle's."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

P = ctypes.c_void_p
OK, EINVAL, EUNSUPPORTED = 0, 1, 2
BF16, INT8, INT4 = 0, 1, 2


@pytest.fixture(scope="module")
def skv():
    from sparse_kv_long_gb300 import _build
    _build.build()
    import sparse_kv_long_gb300 as m
    return m


def rows(kind, **change):
    return {**dict(kind=kind, k=256, v=512, k_scale=64 if kind == INT8 else None, v_scale=64 if kind == INT8 else None,
                   n_rows=64, token_pitch=544 if kind == INT4 else 0, head_pitch=272 if kind == INT4 else 0), **change}


MOVE = dict(n=4, Hkv=2, d=256, src=rows(INT8), srows=P(256), dst=rows(BF16), drows=P(256), rot=64, inter=0, old=P(256),
            oldf=P(256), new=P(256), newf=P(256), st=None, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(n=0), OK), (dict(n=-1), EINVAL), (dict(Hkv=0), EINVAL), (dict(Hkv=4097), EINVAL), (dict(d=96), EUNSUPPORTED),
    (dict(d=512), EUNSUPPORTED), (dict(d=128, src=rows(INT4)), EUNSUPPORTED), (dict(d=64, dst=rows(INT4)), EUNSUPPORTED),
    (dict(rot=72), EINVAL), (dict(rot=272), EINVAL), (dict(rot=-16), EINVAL), (dict(inter=2), EINVAL),
    (dict(src=None), EINVAL), (dict(dst=None), EINVAL), (dict(src=rows(3)), EINVAL), (dict(dst=rows(-1)), EINVAL),
    (dict(src=rows(INT8, k=None, v=None), dst=rows(BF16, k=None, v=None)), EINVAL),
    (dict(src=rows(INT8, k=None)), EINVAL), (dict(dst=rows(BF16, v=None)), EINVAL),
    (dict(src=rows(INT8, k=264)), EINVAL), (dict(dst=rows(BF16, v=520)), EINVAL), (dict(src=rows(INT8, k_scale=None)), EINVAL),
    (dict(dst=rows(INT8, v_scale=None)), EINVAL), (dict(src=rows(INT8, n_rows=-1)), EINVAL),
    (dict(srows=None, src=rows(INT8, n_rows=3)), EINVAL), (dict(drows=None, dst=rows(BF16, n_rows=3)), EINVAL),
    (dict(oldf=None), EINVAL), (dict(newf=None), EINVAL), (dict(src=rows(INT4, k=258)), EINVAL),
    (dict(src=rows(INT4, head_pitch=270)), EINVAL), (dict(src=rows(INT4, head_pitch=132)), EINVAL),
    (dict(src=rows(INT4, head_pitch=1 << 62, token_pitch=1 << 62)), EINVAL), (dict(n=1 << 30), EINVAL),
    (dict(src=rows(INT4, token_pitch=540)), EINVAL), (dict(dst=rows(INT4, token_pitch=546)), EINVAL),
])
def test_move_rows_refuses(skv, change, want):
    a = {**MOVE, **change}
    for side in ("src", "dst"):
        if a[side] is not None:
            a[side] = skv.RowSet(*a[side].values())
    assert skv.lib().skv_move_rows(*a.values()) == want


def test_bindings_refuse_other_types_and_layouts(skv):
    x = torch.zeros((8, 2, 256), dtype=torch.bfloat16)
    q, s = torch.zeros((8, 2, 256), dtype=torch.int8), torch.zeros((8, 2), dtype=torch.float16)
    t = torch.zeros((8, 2, 136), dtype=torch.uint8)
    for bad in ((BF16, x.half(), x), (BF16, x, x[:7]), (BF16, x.transpose(0, 1), x.transpose(0, 1)), (INT8, x, x, s, s),
                (INT8, q, q, s[:7], s), (INT8, q, q, s.float(), s), (INT8, q, q[..., :128]), (INT4, t.char(), t),
                (INT4, t, t[:, :1]), (INT4, t, torch.zeros((8, 3, 136), dtype=torch.uint8)[:, :2]),
                (INT4, t.transpose(1, 2), t.transpose(1, 2))):
        with pytest.raises(ValueError, match="expected"):
            skv.row_set(*bad)
    for bad in (t, torch.zeros((8, 2, 2, 136)), torch.zeros((8, 2, 4, 136), dtype=torch.uint8)[:, :, :2]):
        with pytest.raises(ValueError, match="expected"):
            skv.tier_rows(bad)
    r = skv.tier_rows(torch.zeros((3, 5, 2, 2, 136), dtype=torch.uint8))
    assert (r.n_rows, r.token_pitch, r.head_pitch, r.v - r.k, r.shape) == (15, 544, 272, 136, (2, 256))
    r = skv.row_set(INT4, t, None)
    assert (r.n_rows, r.token_pitch, r.head_pitch, r.v, r.shape) == (8, 272, 136, None, (2, 256))


def test_binding_refuses_sets_that_do_not_match(skv, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # as the tensors here answer
    x = torch.zeros((8, 2, 256), dtype=torch.bfloat16)
    a, f = skv.row_set(BF16, x, x), torch.zeros((32,))
    with pytest.raises(ValueError, match="heads, values"):
        skv.move_rows(a, skv.row_set(BF16, x[..., :128].contiguous(), None), 4)
    with pytest.raises(ValueError, match="numbers of pairs"):
        skv.move_rows(a, a, 4, old_inv_freq=f, new_inv_freq=f[:16])
    i = torch.zeros((4,), dtype=torch.int32)
    for bad in (dict(src_rows=i), dict(dst_rows=i), dict(old_positions=i.long(), old_inv_freq=f),
                dict(new_positions=i[:3], new_inv_freq=f), dict(new_inv_freq=f.double()), dict(status=i.long())):
        with pytest.raises(ValueError, match="contiguous elements"):
            skv.move_rows(a, a, 4, **bad)


def test_rows_that_may_be_written_are_not_read_as_constant(skv):
    """A cache may be its own destination: the non-coherent loads are for memory that no one writes meanwhile."""
    src = open(os.path.join(os.path.dirname(skv.__file__), "csrc", "move_rows.cu")).read()
    assert not re.search(r"\.nc\b|\bld_stream|\bld_nc|__ldg\b|__restrict__", src)


def test_plain_encodings_are_the_oracles(orc):
    """oracle/rows.py against the C oracle's encodings of the same bf16 rows."""
    from oracle import rows as plain
    rng = np.random.default_rng(0)
    x = torch.from_numpy((rng.standard_normal((20, 3, 256)) * np.exp2(rng.integers(-20, 20, (20, 3, 1)))).astype(np.float32))
    x = x.bfloat16()
    bits = x.view(torch.int16).numpy().view(np.uint16)
    q, s = plain.encode("int8", x.float().numpy())
    oq, os_ = orc.quant_int8_rows(bits)
    np.testing.assert_array_equal(q, oq)
    np.testing.assert_array_equal(s.view(np.uint16), os_)
    packed = plain.pack_int4(*plain.encode("int4", x.float().numpy()))
    np.testing.assert_array_equal(packed.reshape(-1), np.asarray(orc.quant_int4_rows(bits)).reshape(-1))
    codes, scale = plain.unpack_int4(packed)
    np.testing.assert_array_equal(plain.pack_int4(codes, scale), packed)
