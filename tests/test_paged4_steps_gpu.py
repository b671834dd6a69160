"""Serving steps over the paged 4-bit cache issued back to back, with nothing between
their kernels: each reads what the one before it has just written, and may begin
while that one drains."""
import numpy as np
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


class Steps:
    """A batch's steps through some layers, in buffers that every step uses again."""

    def __init__(self, news, Hq, Hkv, D, block, layers, dtype, seed):
        B, T = len(news[0]), max(sum(n) for n in news)
        lengths = np.sum(news, 0)
        N = int(sum(-(-int(n) // block) for n in lengths)) + B
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.Hq, self.Hkv, self.block, self.T = Hq, Hkv, block, T
        self.news = [torch.tensor(n, dtype=torch.int32, device="cuda") for n in news]
        self.rows = [[torch.randn((T, Hq + 2 * Hkv, D), device="cuda", generator=g).to(dtype) for _ in range(layers)] for _ in news]
        self.past, self.starts, self.total, self.result = i32(B), i32(B + 1), i32(B), i32(1)
        self.tables, self.free = i32(B, int(max(lengths)) // block + 2).fill_(-1), torch.arange(N, dtype=torch.int32, device="cuda")
        self.count, self.slots = i32(1).fill_(N), torch.zeros(T, dtype=torch.int64, device="cuda")
        self.cache = [[torch.zeros((N, Hkv, block, w), dtype=torch.uint8, device="cuda") for w in (D // 2, D // 2, D // 16, D // 16)]
                      for _ in range(layers)]
        self.buffer = torch.zeros((T, Hq + 2 * Hkv, D), dtype=dtype, device="cuda")  # one for all layers
        self.freq, _ = attn.attn_rope_frequencies(D)

    def run(self, sync):
        """All steps; every layer's output, and the caches."""
        made = []
        for new, rows in zip(self.news, self.rows):
            attn.attn_cache_assign(self.past, new, self.tables, self.free, self.count, block_size=self.block, num_tokens=self.T,
                                   q_starts=self.starts, total_lengths=self.total, slot_map=self.slots, result=self.result)
            sync()
            q, k, v = self.buffer.split([self.Hq, self.Hkv, self.Hkv], 1)
            for layer, cache in zip(rows, self.cache):
                self.buffer.copy_(layer)
                sync()
                attn.attn_rope(q, k, self.freq, q_starts=self.starts, total_lengths=self.total, q_out=q, k_out=k)
                sync()
                attn.attn_cache_append_fp4(k, v, self.slots, *cache)
                sync()
                out = torch.full((self.T, self.Hq, q.shape[2]), 7.0, dtype=q.dtype, device="cuda")
                attn.attn_fwd_paged_fp4(q, *cache, self.tables, self.starts, self.total, out=out)
                sync()
                attn.attn_cache_read_fp4(*cache, self.slots, dtype=q.dtype, k=k, v=v)  # over the rows, as later work would
                sync()
                made += [out, self.buffer.clone()]
            self.past.copy_(self.total)
            sync()
        return made + [c for cache in self.cache for c in cache] + [self.tables, self.count, self.result]


CASES = {
    "decode": dict(news=[[3] * 4] + [[1] * 4] * 40, Hq=8, Hkv=2, D=64, block=16, layers=3, dtype=torch.float16),
    "batch": dict(news=[list(range(1, 65))] + [[1] * 64] * 20, Hq=32, Hkv=8, D=128, block=16, layers=2, dtype=torch.bfloat16),
    "prompts": dict(news=[[700, 1, 300], [90, 400, 1], [1, 2, 1]], Hq=32, Hkv=8, D=128, block=64, layers=3, dtype=torch.bfloat16),
}


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("seed", [0, 1])
def test_steps_back_to_back(name, seed):
    one = Steps(**CASES[name], seed=seed)
    want = one.run(torch.cuda.synchronize)
    assert int(want[-1]) == 0
    got = Steps(**CASES[name], seed=seed).run(lambda: None)
    torch.cuda.synchronize()
    assert attn.get_device_status() == attn.ATTN_OK
    for i, (a, b) in enumerate(zip(want, got)):
        assert torch.equal(a, b), i


def test_captured_steps_back_to_back():
    """The same in a graph, where the early launches are its edges."""
    case = CASES["decode"]
    want = Steps(**case, seed=3).run(torch.cuda.synchronize)
    one = Steps(**case, seed=3)
    state = [t.clone() for t in (one.past, one.tables, one.free, one.count)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = one.run(lambda: None)
    for _ in range(2):
        for t, c in zip((one.past, one.tables, one.free, one.count), state):
            t.copy_(c)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(want, got)):
            assert torch.equal(a, b), i
