"""Gradients through attn_rope: against autograd over the formula in 64 bits, and
against differences."""
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


def formula(x, pos, freq, layout, inverse, scale):
    """The definition on the CPU in 64 bits, differentiable."""
    R = 2 * len(freq)
    w = (pos.double()[:, None] * freq)[:, None].cpu()
    c, n = w.cos() * scale, w.sin() * (-scale if inverse else scale)
    i = torch.arange(R // 2)
    a, b = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + R // 2)
    turned = torch.cat([x[..., a] * c - x[..., b] * n, x[..., b] * c + x[..., a] * n], -1)
    order = torch.empty(R, dtype=torch.long)
    order[torch.cat([a, b])] = torch.arange(R)
    return torch.cat([turned[..., order], x[..., R:]], -1)


def close(got, want, size, dtype):
    """Sine and cosine off by 2^-22, three roundings of 2^-24 on values up to size in two products, and half a step of the type."""
    got, want = got.double().cpu(), want.detach()
    tol = torch.finfo(dtype).eps / 2 * want.abs() + 4 * 2.0 ** -21 * size
    assert bool(((got - want).abs() <= tol).all()), float(((got - want).abs() / tol).max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("Hk,R", [(2, 64), (0, 64), (1, 24), (3, 0)])
def test_gradients(dtype, layout, inverse, Hk, R):
    T, Hq, D, scale = 13, 4, 64, 1.25
    g = torch.Generator(device="cuda").manual_seed(R + Hk)
    rows = torch.randn((T, Hq + 5, D), device="cuda", generator=g).to(dtype).requires_grad_()  # q and k are slices of it
    q, k = rows[:, :Hq], rows[:, Hq:Hq + Hk] if Hk else None
    freq = attn.attn_rope_frequencies(R)[0] if R else torch.zeros(0, dtype=torch.float64, device="cuda")
    pos = torch.randint(0, 5000, (T,), device="cuda", generator=g).int()
    kw = dict(positions=pos, layout=layout, inverse=inverse, scale=scale)
    made = attn.attn_rope(q, k, freq, **kw)
    with torch.no_grad():
        plain = attn.attn_rope(q, k, freq, **kw)
    assert made[0].requires_grad and torch.equal(made[0], plain[0]) and not plain[0].requires_grad
    assert (made[1] is None) == (k is None)
    dy = [torch.randn(x.shape, device="cuda", generator=g).to(dtype) for x in made if x is not None]
    loss = sum((x * d).double().sum() for x, d in zip(made, dy))
    loss.backward()
    x = rows.detach().double().cpu().requires_grad_()
    want = formula(x[:, :Hq + Hk], pos.cpu(), freq.cpu(), layout, inverse, scale)
    d = torch.cat([y.double().cpu() for y in dy], 1)
    (want * d).sum().backward()
    close(torch.cat([y for y in made if y is not None], 1), want, 2 * float(x.detach().abs().max()), dtype)
    close(rows.grad, x.grad, 2 * float(d.abs().max()), dtype)


def test_gradients_of_differences():
    """<f(x + dx) - f(x), dy> = <dx, gradient>: the map is linear."""
    T, H, D = 9, 2, 128
    x, dx, dy = (torch.randn((T, H, D), device="cuda") for _ in range(3))
    freq, pos = attn.attn_rope_frequencies(D)[0], torch.arange(T, dtype=torch.int32, device="cuda") * 1000
    x.requires_grad_()
    f = lambda z: attn.attn_rope(z, None, freq, positions=pos, scale=0.7)[0]  # noqa: E731
    (f(x) * dy).sum().backward()
    with torch.no_grad():
        left, right = ((f(x + dx) - f(x)).double() * dy.double()).sum(), (dx.double() * x.grad.double()).sum()
    # values up to 8 in size, off by 2^-19 each, summed over all
    assert abs(float(left - right)) <= T * H * D * 2.0 ** -16


def test_rows_of_no_request_have_no_gradient():
    T, D = 10, 64
    q, k = (torch.randn((T, h, D), device="cuda", requires_grad=True) for h in (3, 1))
    starts, total = torch.tensor([1, 4, 7], dtype=torch.int32, device="cuda"), torch.tensor([90, 5], dtype=torch.int32, device="cuda")
    freq, _ = attn.attn_rope_frequencies(D)
    full = [torch.full((8, T, 3, D), float("nan"), device="cuda") for _ in range(4)]  # what freed memory may hold
    del full
    a, b = attn.attn_rope(q, k, freq, q_starts=starts, total_lengths=total)
    (a[1:7].sum() + b[1:7].sum()).backward()
    pos = torch.tensor([0, 87, 88, 89, 2, 3, 4], dtype=torch.int32, device="cuda")
    one = torch.ones((7, 3, D), device="cuda")
    want, _ = attn.attn_rope(one, None, freq, positions=pos, inverse=True)
    for x in (q, k):
        assert bool((x.grad[0] == 0).all()) and bool((x.grad[7:] == 0).all())
        assert torch.equal(x.grad[1:7], want[1:, :x.shape[1]])


def test_the_next_step_before_the_backward_pass():
    """A paged step's lengths, written anew in place by the next step: the gradient is that of the step's own positions."""
    T, D, block = 6, 64, 16
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    tables, free, count = torch.full((2, 8), -1, dtype=torch.int32, device="cuda"), torch.arange(16, dtype=torch.int32, device="cuda"), i32(16)
    starts, total = i32(0, 0, 0), i32(0, 0)
    assign = lambda past, new: attn.attn_cache_assign(past, new, tables, free, count, block_size=block, num_tokens=T,  # noqa: E731
                                                      q_starts=starts, total_lengths=total)
    freq, _ = attn.attn_rope_frequencies(D)
    q = torch.randn((T, 2, D), device="cuda", requires_grad=True)
    assign(i32(20, 7), i32(4, 2))
    y = attn.attn_rope(q, None, freq, q_starts=starts, total_lengths=total)[0]
    assign(total.clone(), i32(1, 5))
    y.sum().backward()
    assert starts.tolist() == [0, 1, 6]
    want, _ = attn.attn_rope(torch.ones_like(q), None, freq, positions=i32(20, 21, 22, 23, 7, 8), inverse=True)
    assert torch.equal(q.grad, want)


def test_one_output_used_and_second_derivatives():
    T, D = 6, 32
    q, k = (torch.randn((T, 2, D), device="cuda", requires_grad=True) for _ in range(2))
    freq, pos = attn.attn_rope_frequencies(D)[0], torch.arange(T, dtype=torch.int32, device="cuda")
    attn.attn_rope(q, k, freq, positions=pos)[1].sum().backward()
    assert bool((q.grad == 0).all()) and bool((k.grad != 0).any())
    # f' f'^T = 1 for a rotation: the gradient of |f^T dy|^2 / 2 with respect to dy is dy
    dy = torch.randn((T, 2, D), device="cuda", requires_grad=True)
    y = attn.attn_rope(q, None, freq, positions=pos)[0]
    dx, = torch.autograd.grad(y, q, dy, create_graph=True)
    back, = torch.autograd.grad((dx ** 2).sum() / 2, dy)
    # two rotations, each off by 2^-20 of values up to 2 |dy|
    assert float((back - dy).detach().abs().max()) <= 2 * 2.0 ** -19 * float(dy.detach().abs().max())


def test_only_k_requires_gradients_and_given_outputs():
    T, D = 4, 64
    q, k = torch.randn((T, 2, D), device="cuda"), torch.randn((T, 1, D), device="cuda", requires_grad=True)
    freq, pos = attn.attn_rope_frequencies(D)[0], torch.arange(T, dtype=torch.int32, device="cuda")
    a, b = attn.attn_rope(q, k, freq, positions=pos)
    assert b.requires_grad
    b.sum().backward()
    assert k.grad.shape == k.shape
    for kw in (dict(q_out=torch.empty_like(q)), dict(k_out=torch.empty_like(k)), dict(q_out=q)):
        with pytest.raises(ValueError, match="requires gradients"):
            attn.attn_rope(q, k, freq, positions=pos, **kw)
    with torch.no_grad():
        out = attn.attn_rope(q, k, freq, positions=pos, k_out=torch.empty_like(k))
    assert torch.equal(out[1], b)
    with pytest.raises(ValueError):  # refused as without gradients
        attn.attn_rope(q, k, freq)


def test_captured_backward():
    """Forward and backward of a step in a graph, replayed on other values."""
    T, D = 50, 128
    x = torch.randn((T, 8, D), device="cuda", dtype=torch.bfloat16)
    freq, pos = attn.attn_rope_frequencies(D)[0], torch.arange(T, dtype=torch.int32, device="cuda")

    def step(x):
        y = x.detach().requires_grad_()
        out = attn.attn_rope(y, None, freq, positions=pos)[0]
        return out.detach(), torch.autograd.grad(out.float().square().sum(), y)[0]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(x)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = step(x)
    for _ in range(2):
        x.copy_(torch.randn_like(x))
        graph.replay()
        torch.cuda.synchronize()
        want = step(x)
        assert torch.equal(made[0], want[0]) and torch.equal(made[1], want[1])
