"""Refusals of skv_norm_rope_append and skv_paged_attend: decided on the host,
before anything is launched, so they run without a GPU."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
OK, EINVAL, EUNSUPPORTED, ENOMEM = 0, 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    from sparse_kv_long_gb300 import _build
    _build.build()
    import sparse_kv_long_gb300 as skv
    return skv.lib()


NORM = dict(n_tok=4, Hq=8, Hkv=2, d=256, rot=64, inter=0, q=P(256), qs=2048, k=P(256), ks=512, v=P(256), vs=512,
            qw=None, kw=None, eps=1e-6, pos=P(256), inv=P(256), q_out=P(256), kind=0, rows=P(256), n_rows=64,
            kp=P(256), vp=P(256), ksc=None, vsc=None, st=None, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(n_tok=0), OK), (dict(n_tok=-1), EINVAL), (dict(d=96), EUNSUPPORTED), (dict(d=512), EUNSUPPORTED),
    (dict(rot=72), EINVAL), (dict(rot=272), EINVAL), (dict(rot=-16), EINVAL), (dict(inter=2), EINVAL),
    (dict(q=None, k=None, v=None), EINVAL), (dict(inv=None), EINVAL), (dict(pos=None), EINVAL),
    (dict(q_out=None), EINVAL), (dict(q=P(8)), EINVAL), (dict(qs=2052), EINVAL), (dict(qs=2040), EINVAL),
    (dict(kp=None), EINVAL), (dict(vp=None), EINVAL), (dict(kp=P(24)), EINVAL), (dict(ks=256), EINVAL),
    (dict(kind=2), EINVAL), (dict(kind=1), EINVAL), (dict(kind=1, ksc=P(256)), EINVAL), (dict(eps=-1.0), EINVAL),
    (dict(eps=float("nan")), EINVAL), (dict(rows=None, n_rows=3), EINVAL), (dict(Hq=0), EINVAL),
    (dict(Hkv=0), EINVAL), (dict(n_rows=-1), EINVAL),
])
def test_norm_rope_append_refuses(lib, change, want):
    assert lib.skv_norm_rope_append(*{**NORM, **change}.values()) == want


ATT = dict(kind=0, B=2, n_tok=6, Hq=8, Hkv=2, d=256, q=P(256), qs=2048, kp=P(256), vp=P(256), ksc=None, vsc=None,
           n_rows=1024, page=16, table=P(256), n_pages=8, q_start=P(256), lengths=P(256), S=0, W=0, scale=0.1,
           out=P(256), ws=P(256), wsn=1 << 40, st=None, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(B=0), OK), (dict(n_tok=0), OK), (dict(kind=2), EINVAL), (dict(B=-1), EINVAL), (dict(n_tok=-1), EINVAL),
    (dict(B=4097), EINVAL), (dict(Hkv=3), EINVAL), (dict(Hkv=0), EINVAL), (dict(S=-1), EINVAL), (dict(W=-1), EINVAL),
    (dict(d=64), EUNSUPPORTED), (dict(Hq=258, Hkv=2, qs=258 * 256), EUNSUPPORTED), (dict(page=4), EUNSUPPORTED),
    (dict(page=20), EUNSUPPORTED), (dict(page=0), EUNSUPPORTED), (dict(q=None), EINVAL), (dict(kp=None), EINVAL),
    (dict(vp=P(8)), EINVAL), (dict(table=None), EINVAL), (dict(n_pages=0), EINVAL), (dict(lengths=None), EINVAL),
    (dict(out=P(8)), EINVAL), (dict(n_rows=15), EINVAL), (dict(kind=1), EINVAL), (dict(kind=1, ksc=P(256)), EINVAL),
    (dict(q_start=None), EINVAL), (dict(qs=2044), EINVAL), (dict(qs=1024), EINVAL), (dict(ws=None), ENOMEM),
    (dict(wsn=8), ENOMEM), (dict(ws=P(8)), ENOMEM), (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL),
    (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(n_pages=1 << 28), EINVAL),
])
def test_paged_attend_refuses(lib, change, want):
    assert lib.skv_paged_attend(*{**ATT, **change}.values()) == want


def test_workspace_sizes(lib):
    size = lib.skv_paged_attend_workspace_size
    assert size(1, 1, 8, 2, 256) > 0
    assert size(4, 400, 8, 2, 256) >= size(4, 40, 8, 2, 256) >= size(1, 1, 8, 2, 256)
    for bad in [(0, 1, 8, 2, 256), (1, 0, 8, 2, 256), (1, 1, 8, 3, 256), (1, 1, 8, 2, 96), (1, 1, 258, 2, 256)]:
        assert size(*bad) == 0


def test_binding_refuses_scattered_heads():
    import sparse_kv_long_gb300 as skv
    x = torch.zeros((4, 256, 8), dtype=torch.bfloat16).transpose(1, 2)  # a head's values 8 apart
    with pytest.raises(ValueError):
        skv.norm_rope_append(x, None, None, None, None, None, None, None)
    q, k = torch.zeros((4, 8, 256), dtype=torch.bfloat16), torch.zeros((5, 2, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        skv.norm_rope_append(q, k, None, None, None, None, None, None)


@pytest.mark.parametrize("change,want", [
    (dict(scale=2.5e38), EINVAL),  # finite, but not in units of log2
    (dict(n_pages=(1 << 62) // 16), EINVAL), (dict(n_pages=(1 << 27) - 64), EINVAL),
    (dict(n_pages=(1 << 27) - 100, W=(1 << 30) + 1), EINVAL),  # a window that is neither short nor everything
    (dict(n_tok=1 << 28), EINVAL), (dict(B=4000, n_tok=4000, n_pages=1 << 22), EINVAL), (dict(n_rows=1 << 34), EINVAL),
])
def test_paged_attend_refuses_what_32_bits_do_not_hold(lib, change, want):
    assert lib.skv_paged_attend(*{**ATT, **change}.values()) == want


def test_bindings_refuse_other_types_strides_and_sizes():
    import sparse_kv_long_gb300 as skv
    q = torch.zeros((4, 8, 256), dtype=torch.bfloat16)
    pool = torch.zeros((64, 2, 256), dtype=torch.bfloat16)
    i32 = torch.zeros((4,), dtype=torch.int32)
    good = dict(q=q, k_pool=pool, v_pool=pool, block_table=torch.zeros((4, 2), dtype=torch.int32), page=16, lengths=i32,
                softmax_scale=1.0, out=q, workspace=q)
    for bad in (dict(q=q.half()), dict(k_pool=pool.half()), dict(v_pool=torch.zeros((2, 64, 256)).bfloat16().transpose(0, 1)),
                dict(block_table=torch.zeros((2, 4), dtype=torch.int32).T), dict(lengths=i32.long()),
                dict(out=q.float()), dict(q_start=i32.long()), dict(status=i32.long()), dict(k_scale=i32),
                dict(v_pool=pool[:63]), dict(out=q[:3]), dict(lengths=i32[:3]), dict(q_start=i32), dict(k_pool=pool[..., :128])):
        with pytest.raises(ValueError, match="contiguous|consecutive|differ |queries of"):
            skv.paged_attend(skv.KV_BF16, **{**good, **bad})
    good = dict(q=q, k=q[:, :2], v=q[:, 2:4], positions=i32, inv_freq=torch.zeros((64,)), q_out=q, k_pool=pool, v_pool=pool)
    for bad in (dict(k=q[:, :2].half()), dict(positions=i32.long()), dict(inv_freq=torch.zeros((64,)).double()),
                dict(q_out=torch.zeros((8, 4, 256)).bfloat16().transpose(0, 1)), dict(k_pool=pool.to(torch.int8)),
                dict(out_rows=i32), dict(q_weight=q), dict(k_weight=torch.zeros((256,)).half()),
                dict(positions=i32[:3]), dict(q_out=q[:3]), dict(v_pool=pool[:63]), dict(q_weight=torch.zeros((255,)))):
        with pytest.raises(ValueError, match="contiguous|consecutive|differ |queries of"):
            skv.norm_rope_append(**{**good, **bad})


def test_bindings_refuse_pools_and_scales_of_another_layout():
    """Enough elements are not enough: rows of another length or heads, or pages where rows are expected, would be
    misread."""
    import sparse_kv_long_gb300 as skv
    q, i32 = torch.zeros((4, 8, 256), dtype=torch.bfloat16), torch.zeros((4,), dtype=torch.int32)
    pool, scale = torch.zeros((64, 2, 256), dtype=torch.int8), torch.zeros((64, 2), dtype=torch.float16)
    other = [pool.new_zeros(s) for s in ((64, 4, 256), (8, 16, 2, 256), (128, 1, 256), (64, 2, 512), (64, 1024), (63, 2, 256))]
    wide = [scale.new_zeros(s) for s in ((64, 4), (128, 1), (8, 16, 2), (256,), (63, 2))]
    good = dict(kv_kind=skv.KV_INT8, q=q, k_pool=pool, v_pool=pool, block_table=torch.zeros((4, 2), dtype=torch.int32),
                page=16, lengths=i32, softmax_scale=1.0, out=q, workspace=q, k_scale=scale, v_scale=scale)
    bad = [dict(v_pool=t) for t in other] + [{s: t} for s in ("k_scale", "v_scale") for t in wide]
    for b in bad:
        with pytest.raises(ValueError, match="expected contiguous rows"):
            skv.paged_attend(**{**good, **b})
    with pytest.raises(ValueError):
        skv.paged_attend(**{**good, "k_pool": other[1]})
    good = dict(q=q, k=q[:, :2], v=q[:, 2:4], positions=i32, inv_freq=torch.zeros((64,)), q_out=q, k_pool=pool, v_pool=pool,
                kv_kind=skv.KV_INT8, k_scale=scale, v_scale=scale)
    for b in bad + [dict(k_pool=t) for t in other[:2]] + [dict(k_pool=other[0], v_pool=other[0])]:
        with pytest.raises(ValueError, match="expected contiguous rows"):
            skv.norm_rope_append(**{**good, **b})
    for g in (good, {**good, "k": None}, {**good, "v": None}, {**good, "k": None, "k_pool": None, "k_scale": None}):
        with pytest.raises(ValueError, match="on the current CUDA device"):  # nothing else is wrong with these
            skv.norm_rope_append(**g)


@pytest.mark.parametrize("d,G,n,mb", [  # megabytes of the documentation, at 152 SMs
    (256, 16, 1, 5.1), (256, 1, 1, 0.33), (256, 4, 32, 41), (256, 6, 22, 84), (256, 6, 64, 161), (256, 24, 4000, 161),
    (128, 16, 1, 2.6), (128, 4, 32, 20.5), (128, 4, 33, 42), (128, 4, 4000, 81),
])
def test_workspace_sizes_are_the_documented_ones(lib, d, G, n, mb):
    sms = lib.skv_device_sm_count()
    sizes = {lib.skv_paged_attend_workspace_size(B, n, 2 * G, 2, d) for B in (1, 7, n, 4096)}
    assert len(sizes) == 1  # whatever the number of requests
    assert mb * 0.9e6 < sizes.pop() / (sms if sms > 0 else 152) * 152 <= mb * 1e6
    one = lib.skv_paged_attend_workspace_size(1, n, 2 * G, 2, d)
    assert all(lib.skv_paged_attend_workspace_size(1, m, 2 * G, 2, d) <= one for m in range(1, n, max(1, n // 50)))
