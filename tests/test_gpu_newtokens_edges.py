"""skv_norm_rope_append and skv_paged_attend where they could go wrong without
an ordinary call showing it: waits that give up, offsets out of order, values
and scales at the ends of their ranges."""
import ctypes
import os
import subprocess
import types

import pytest
import torch

from test_gpu_newtokens import KINDS, Case, kind_of, skv  # noqa: F401  (skv is a fixture)

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
