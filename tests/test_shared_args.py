"""Refusals of skv_shared_attend: decided on the host, before anything is
launched, so they run without a GPU."""
import ctypes
import os
import re

import pytest
import torch

from skvtest import ROOT

P = ctypes.c_void_p
OK, EINVAL, EUNSUPPORTED, ENOMEM = 0, 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    from sparse_kv_long_gb300 import _build
    _build.build()
    import sparse_kv_long_gb300 as skv
    return skv.lib()


ATT = dict(kind=0, B=2, n_tok=6, Hq=8, Hkv=2, d=256, q=P(256), qs=2048, kp=P(256), vp=P(256), ksc=None, vsc=None,
           n_rows=1024, page=16, groups=1, start=P(256), ptable=P(256), n_ppages=8, plen=P(256), table=P(256), n_pages=8,
           q_start=P(256), lengths=P(256), scale=0.1, out=P(256), ws=P(256), wsn=1 << 40, st=None, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(B=0), OK), (dict(n_tok=0), OK), (dict(kind=2), EINVAL), (dict(B=-1), EINVAL), (dict(n_tok=-1), EINVAL),
    (dict(B=4097), EINVAL), (dict(Hkv=3), EINVAL), (dict(Hkv=0), EINVAL), (dict(groups=-1), EINVAL),
    (dict(groups=4097), EINVAL), (dict(start=None), EINVAL), (dict(ptable=None), EINVAL), (dict(plen=None), EINVAL),
    (dict(n_ppages=0), EINVAL), (dict(n_ppages=-1), EINVAL), (dict(n_pages=0), EINVAL), (dict(n_pages=-1), EINVAL),
    (dict(d=64), EUNSUPPORTED), (dict(Hq=258, Hkv=2, qs=258 * 256), EUNSUPPORTED), (dict(page=4), EUNSUPPORTED),
    (dict(page=20), EUNSUPPORTED), (dict(page=0), EUNSUPPORTED), (dict(q=None), EINVAL), (dict(kp=None), EINVAL),
    (dict(vp=P(8)), EINVAL), (dict(table=None), EINVAL), (dict(lengths=None), EINVAL), (dict(out=P(8)), EINVAL),
    (dict(n_rows=15), EINVAL), (dict(kind=1), EINVAL), (dict(kind=1, ksc=P(256)), EINVAL), (dict(q_start=None), EINVAL),
    (dict(qs=2044), EINVAL), (dict(qs=1024), EINVAL), (dict(ws=None), ENOMEM), (dict(wsn=8), ENOMEM),
    (dict(ws=P(8)), ENOMEM), (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL), (dict(scale=float("nan")), EINVAL),
    (dict(scale=float("inf")), EINVAL), (dict(scale=2.5e38), EINVAL), (dict(groups=0, wsn=8, start=None, ptable=None,
                                                                          plen=None, n_ppages=0), ENOMEM),
    # what 32 bits do not hold
    (dict(n_pages=1 << 28), EINVAL), (dict(n_ppages=1 << 28), EINVAL), (dict(n_ppages=(1 << 62) // 16), EINVAL),
    (dict(n_tok=1 << 26), EINVAL), (dict(B=4000, n_tok=4000, n_pages=1 << 22), EINVAL),
    (dict(B=4000, n_tok=4000, groups=4000, n_ppages=1 << 22), EINVAL), (dict(n_rows=1 << 34), EINVAL),
])
def test_shared_attend_refuses(lib, change, want):
    assert lib.skv_shared_attend(*{**ATT, **change}.values()) == want


def test_workspace_sizes(lib):
    size = lib.skv_shared_attend_workspace_size
    sizes = [size(4, 2, n, 8, 2, 256) for n in (1, 2, 31, 32, 33, 40, 400, 4000)]
    assert sizes[0] > 0 and sizes == sorted(sizes)
    assert len({size(B, g, 40, 8, 2, 256) for B in (1, 40, 4096) for g in (0, 1, 40)}) == 1
    for n in (1, 32, 33, 40, 4000):  # 8 d + 24 bytes a token and query head beside the partial sums
        sums = lib.skv_paged_attend_workspace_size(4, n, 8, 2, 256)
        assert sums < size(4, 2, n, 8, 2, 256) <= sums * (1.25 if n * 4 > 128 else 1) + n * 8 * (8 * 256 + 24) + 1024
    for bad in [(0, 1, 1, 8, 2, 256), (1, -1, 1, 8, 2, 256), (1, 1, 0, 8, 2, 256), (1, 1, 1, 8, 3, 256), (1, 1, 1, 8, 2, 96),
                (1, 1, 1, 258, 2, 256), (1, 1, 1 << 26, 8, 2, 256)]:
        assert size(*bad) == 0


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 4), (6, 2), (8, 2), (128, 1)])
def test_workspace_of_a_token(lib, d, Hq, Hkv):
    """What the header says that a token more takes: 8 d + 16 bytes per query head, 32 per KV head (the parts are
    rounded up to 256 bytes, so over 1000 tokens, all of them past a full query tile)."""
    size = lib.skv_shared_attend_workspace_size
    text = re.sub(r"\s*\n \*\s*", " ", open(os.path.join(ROOT, "include", "sparsekv.h")).read())
    head, kv = map(int, re.search(r"holds 8 d \+ (\d+) bytes per token and query head and (\d+) per token and KV head",
                                  text).groups())
    more = size(4, 2, 2000, Hq, Hkv, d) - size(4, 2, 1000, Hq, Hkv, d)
    assert abs(more - 1000 * (Hq * (8 * d + head) + Hkv * kv)) <= 512


def test_binding_refuses_other_types_strides_and_sizes():
    import sparse_kv_long_gb300 as skv
    q = torch.zeros((4, 8, 256), dtype=torch.bfloat16)
    pool = torch.zeros((64, 2, 256), dtype=torch.bfloat16)
    i32 = torch.zeros((4,), dtype=torch.int32)
    good = dict(q=q, k_pool=pool, v_pool=pool, group_start=i32, prefix_table=torch.zeros((2, 3), dtype=torch.int32),
                prefix_lengths=i32, block_table=torch.zeros((4, 2), dtype=torch.int32), page=16, lengths=i32,
                softmax_scale=1.0, out=q, workspace=q)
    for bad in (dict(q=q.half()), dict(k_pool=pool.half()), dict(v_pool=torch.zeros((2, 64, 256)).bfloat16().transpose(0, 1)),
                dict(block_table=torch.zeros((2, 4), dtype=torch.int32).T), dict(lengths=i32.long()),
                dict(prefix_table=torch.zeros((3, 2), dtype=torch.int32).T), dict(prefix_lengths=i32.long()),
                dict(group_start=i32.long()), dict(group_start=i32[:2]), dict(prefix_lengths=i32[:1]),
                dict(out=q.float()), dict(q_start=i32.long()), dict(status=i32.long()), dict(k_scale=i32),
                dict(v_pool=pool[:63]), dict(out=q[:3]), dict(lengths=i32[:3]), dict(q_start=i32), dict(k_pool=pool[..., :128])):
        with pytest.raises(ValueError, match="contiguous|consecutive|queries of"):
            skv.shared_attend(skv.KV_BF16, **{**good, **bad})
    with pytest.raises(ValueError, match="on the current CUDA device"):  # nothing else is wrong with this one
        skv.shared_attend(skv.KV_BF16, **good)
