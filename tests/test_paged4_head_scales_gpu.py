"""Head scales at both ends of what the 4-bit cache takes, 2^-60 and 2^60: written, read
back and attended, whole units and units cut between CTAs."""
import numpy as np
import pytest
import torch

import paged4_reference as ref
import tiled_online_softmax_02_gb300 as attn
from paged4_reference import Problem
from test_paged4_gpu import _check_append, _compare, _empty_cache, _run

pytestmark = pytest.mark.gpu

ENDS = {"small": 2.0 ** -60, "small_odd": 1.3 * 2.0 ** -60, "large": 2.0 ** 60, "large_odd": 0.7 * 2.0 ** 60}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_online_softmax_02_gb300 import build
    build.build()
    attn.load_library()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("end", list(ENDS))
def test_append_and_read(end, dtype):
    T, Hkv, D, block, N = 50, 2, 64, 16, 5
    rng = np.random.Generator(np.random.PCG64(3))
    h = np.array([ENDS[end], 1.0], np.float32)
    x = [torch.from_numpy(rng.standard_normal((T, Hkv, D)) * h.astype(np.float64)[:, None]).to(ref.TORCH[dtype]) for _ in range(2)]
    slots = rng.permutation(N * block)[:T].astype(np.int64)
    got, want = _check_append(*x, slots, _empty_cache(N, Hkv, block, D), (h, h))
    heads = torch.from_numpy(h).cuda()
    k, v = attn.attn_cache_read_fp4(*got, torch.from_numpy(slots).cuda(), dtype=ref.TORCH[dtype], k_head_scales=heads, v_head_scales=heads)
    for y, c, s in ((k, want[0], want[2]), (v, want[1], want[3])):
        held = ref.values(c, s, h)[slots // block, :, slots % block]
        assert torch.equal(y.cpu(), torch.from_numpy(held).float().to(ref.TORCH[dtype]))


@pytest.mark.parametrize("ends", [("small", "large"), ("large", "small"), ("small_odd", "small_odd"), ("large_odd", "large_odd")], ids=str)
@pytest.mark.parametrize("new", [(1, 1), (150, 40)], ids=["few", "many"])
def test_attention(new, ends):
    """Few long requests: every unit is cut, and its partial rows are joined."""
    kh, vh = (ENDS[e] for e in ends)
    w = Problem(new=new, total=(3000, 900), Hq=4, Hkv=1, dtype="bf16", scale=0.1 / kh, wide=True)
    x = ref.make(w)
    x["k_heads"], x["v_heads"] = torch.tensor([kh]), torch.tensor([vh])
    out, lse = _run(w, x)
    assert attn.get_device_status() == attn.ATTN_OK
    _compare(w, x, out, lse)
