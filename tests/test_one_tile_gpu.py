"""Calls of the paged attention over tables of one key tile, after which no joining
kernel is launched: whatever comes next on the stream may begin as they drain."""
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


@pytest.mark.parametrize("new", [1, 100])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bits", [4, 8])
def test_products_between_calls(bits, D, new):
    """Matrix products (which may hold tensor memory) and further calls, back to back and one by one: the same bits."""
    B, Hq, Hkv, block = 48, 16, 2, 64
    g = torch.Generator(device="cuda").manual_seed(bits * D + new)
    randn = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    T, N = B * new, 2 * B
    q, k, v, a = randn(T, Hq, D), randn(B * 128, Hkv, D), randn(B * 128, Hkv, D), randn(4096, 4096)
    slots = torch.arange(B * 128, device="cuda")
    tables = torch.arange(N, dtype=torch.int32, device="cuda").view(B, 2)
    starts = torch.arange(0, T + 1, new, dtype=torch.int32, device="cuda")
    totals = torch.arange(B, dtype=torch.int32, device="cuda") % 28 + 100
    if bits == 4:
        cache = [torch.zeros((N, Hkv, block, w), dtype=torch.uint8, device="cuda") for w in (D // 2, D // 2, D // 16, D // 16)]
        attn.attn_cache_append_fp4(k, v, slots, *cache)
        attend = attn.attn_fwd_paged_fp4
    else:
        cache = [torch.zeros((N, Hkv, block, D), dtype=torch.uint8, device="cuda") for _ in range(2)] + \
                [torch.zeros((N, Hkv), device="cuda") for _ in range(2)]
        attn.attn_cache_append_fp8(k, v, slots, *cache)
        attend = attn.attn_fwd_paged_fp8

    def chain(sync):
        made, x = [], q
        for _ in range(6):
            x = attend(x, *cache, tables, starts, totals)
            sync()
            y = torch.mm(a, a)
            sync()
            made += [x, y]
        return made

    want = chain(torch.cuda.synchronize)
    got = chain(lambda: None)
    torch.cuda.synchronize()
    assert attn.get_device_status() == attn.ATTN_OK
    for x, y in zip(want, got):
        assert torch.equal(x, y)
