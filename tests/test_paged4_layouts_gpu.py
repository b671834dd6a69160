"""Rows of the 4-bit cache read into buffers where K and V lie between each other."""
import pytest
import torch

import tiled_online_softmax_02_gb300 as attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_online_softmax_02_gb300 import build
    build.build()
    attn.load_library()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,D", [(37, 3, 64), (1, 2, 128), (50, 1, 128)])
@pytest.mark.parametrize("order", ["thid", "tihd", "ithd", "htid", "ihtd", "hitd"])
def test_read_side_by_side(order, T, H, D, dtype):
    """`order`: how tokens, heads, k / v (i) and values lie in the buffer, the outermost first."""
    N, block = 4, 16
    g = torch.Generator(device="cuda").manual_seed(T)
    made = lambda w, top: torch.randint(0, top, (N, H, block, w), dtype=torch.uint8, device="cuda", generator=g)  # noqa: E731
    cache = [made(D // 2, 256), made(D // 2, 256), made(D // 16, 120), made(D // 16, 120)]
    slots = torch.randperm(N * block, device="cuda", generator=g)[:T]
    want = attn.attn_cache_read_fp4(*cache, slots, dtype=dtype)
    size = dict(t=T, h=H, i=2, d=D)
    buffer = torch.full((size[order[0]] + 1, *(size[c] for c in order[1:])), 7.0, dtype=dtype, device="cuda")
    k, v = (buffer[:-1].select(order.index("i"), i) for i in range(2))
    if order.replace("i", "") == "htd":
        k, v = k.transpose(0, 1), v.transpose(0, 1)
    got = attn.attn_cache_read_fp4(*cache, slots, k=k, v=v)
    assert got[0] is k and got[1] is v
    torch.cuda.synchronize()
    assert torch.equal(k, want[0]) and torch.equal(v, want[1]) and bool((buffer[-1] == 7).all())
