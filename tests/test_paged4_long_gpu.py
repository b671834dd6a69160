"""The paged 4-bit attention's kernel for many rows where requests have many row tiles,
so that a warp lays out a request together: (rows of new tokens - requests) * query
heads a kv head above 8192, row tiles of 256 rows, requests of more than 8 of them.
Each case also says which kernel it must reach, so that a choice between the kernels
that is measured anew does not move it off unseen."""
import pytest
import torch

import paged4_reference as ref
import tiled_online_softmax_02_gb300 as attn
from paged4_reference import Problem
from test_paged4_gpu import _compare, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_online_softmax_02_gb300 import build
    build.build()
    attn.load_library()
    torch.cuda.set_device(0)


def kernels(call):
    """Names of the kernels that call() launches; None where this machine records none."""
    from torch.profiler import ProfilerActivity, profile
    try:
        with profile(activities=[ProfilerActivity.CUDA]) as p:
            call()
            torch.cuda.synchronize()
        names = [e.name for e in p.events()]
    except RuntimeError:
        return None
    return names if any("attn_paged4" in n for n in names) else None


CASES = {
    "long_and_short": dict(new=(700, 1, 40), total=(1000, 500, 40), Hq=16, Hkv=1),
    "more_than_32_row_tiles": dict(new=(600,), total=(900,), Hq=16, Hkv=1),
    "kv_heads": dict(new=(530, 1, 500), total=(530, 300, 777), Hq=32, Hkv=2, D=64),
    "after_many_single_tokens": dict(new=(1,) * 300 + (900,) + (1,) * 230, total=tuple(1 + b % 50 for b in range(300)) + (950,) + (9,) * 230,
                                     Hq=16, Hkv=1, D=64, block=16),
    "two_among_many_single_tokens": dict(new=(400,) + (1,) * 520 + (0,) * 9 + (450,), total=(400,) + (40,) * 520 + (3,) * 9 + (500,),
                                         Hq=16, Hkv=1, D=64, block=32),
    "several_in_a_warp": dict(new=(600,) * 8, total=(600, 601, 700, 640, 900, 1000, 777, 600), Hq=4, Hkv=1, D=64),
    "window": dict(new=(700, 40), total=(1500, 90), Hq=16, Hkv=1, window=100, wide=False),
    "window_full": dict(new=(640, 9), total=(900, 900), Hq=16, Hkv=1, window=70, causal=False, D=64, wide=False),
    "softcap_f16": dict(new=(700, 5), total=(900, 70), Hq=16, Hkv=1, softcap=20.0, dtype="f16", q_std=5.0),
    "odd_group": dict(new=(700, 33), total=(800, 33), Hq=15, Hkv=1, block=128),
    "more_new_than_total": dict(new=(900, 2), total=(600, 0), Hq=12, Hkv=1, D=64, heads=True),
    "nothing_visible": dict(new=(700, 1), total=(0, 200), Hq=16, Hkv=1, D=64),
}


@pytest.mark.parametrize("name", list(CASES))
def test_requests_of_many_row_tiles(name):
    w = Problem(**{"wide": True, **CASES[name]})
    x = ref.make(w)
    T, group = x["q"].shape[0], w.Hq // w.Hkv
    assert (T - len(w.new)) * group > 8192 and max(w.new) * group > 8 * 256
    out, lse = _run(w, x)
    assert attn.get_device_status() == attn.ATTN_OK
    _compare(w, x, out, lse)
    names = kernels(lambda: _run(w, x))
    assert names is None or any("attn_paged4_tc_kernel" in n for n in names), names
    again, again_lse = _run(w, x)
    assert torch.equal(out, again) and torch.equal(lse, again_lse)


def test_kernels_are_recorded_by_the_calls_that_reach_them():
    """The few-rows kernel is told from the many-rows one, where kernels are recorded at all."""
    w = Problem(new=(1, 1), total=(300, 20))
    x = ref.make(w)
    _run(w, x)
    names = kernels(lambda: _run(w, x))
    if names is None:
        pytest.skip("this machine records no kernels")
    assert any("attn_paged4_dec_kernel" in n for n in names) and not any("attn_paged4_tc_kernel" in n for n in names)
