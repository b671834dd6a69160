"""Rotary positions on a GPU against the definition in 64 bits, and the inverse
against the formula's gradient and differences."""
import numpy as np
import pytest
import torch

import paged4_reference as ref
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


def _tolerance(x, want, dtype, scale):
    """Half a step of the type on the result; before it sine and cosine off by 2^-22 (the angle by 2^-24 turns rounded
    to 24 bits, the functions by 2^-23, the factor's product by 2^-24) and three roundings of 2^-24 on values up to
    scale (|a| + |b|).  Subnormal results of f16 and bf16 have a step of their own."""
    info = torch.finfo(dtype)
    size = np.abs(x).max(-1, keepdims=True)
    return info.eps / 2 * np.abs(want) + abs(scale) * 2 * 2.0 ** -21 * size + info.smallest_normal * info.eps


CASES = [  # T, Hq, Hk, D, R, extra heads of the buffer
    (1, 1, 1, 64, 64, 0), (5, 4, 2, 128, 128, 0), (33, 32, 8, 128, 64, 0), (7, 3, 1, 96, 96, 2), (70, 8, 8, 256, 64, 1),
    (9, 2, 1, 64, 16, 0), (4, 5, 3, 80, 24, 0), (6, 2, 2, 50, 50, 1), (3, 1, 1, 7, 6, 0), (3, 2, 1, 2, 2, 0),
    (2, 2, 1, 512, 512, 0), (700, 6, 2, 64, 32, 0), (5, 3, 0, 128, 128, 0), (4, 2, 2, 64, 0, 0), (2, 40, 40, 128, 128, 0),
    (3, 2, 2, 1040, 1040, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_rope(case, layout, dtype):
    T, Hq, Hk, D, R, extra = case
    rng = np.random.Generator(np.random.PCG64(T * D + R))
    t = ref.TORCH[dtype]
    rows = lambda H: torch.from_numpy(rng.standard_normal((T, H + extra, D))).to(t).cuda()[:, :H]  # noqa: E731
    q, k = rows(Hq), rows(Hk) if Hk else None
    pos = rng.integers(0, 200000, T).astype(np.int32)
    pos[0] = 0
    freq = (10000.0 ** (-np.arange(0, R, 2) / max(R, 1))).astype(np.float64)
    for inverse, scale in ((False, 1.0), (True, 1.25)):
        got = attn.attn_rope(q, k, torch.from_numpy(freq).cuda(), positions=torch.from_numpy(pos).cuda(), layout=layout,
                             inverse=inverse, scale=scale)
        assert (got[1] is None) == (k is None)
        for x, y in zip((q, k), got):
            if x is None:
                continue
            x, y = x.double().cpu().numpy(), y.double().cpu().numpy()
            want = ref.rope(x, pos, freq, layout == "interleaved", inverse, scale)
            assert np.array_equal(y[..., R:], x[..., R:])
            assert (np.abs(y - want) <= _tolerance(x, want, t, scale)).all()


@pytest.mark.parametrize("freq", [1.0, 0.731, 1e-3, 6.5, 1000.0, 1e-12, 1e-30, -0.5, 0.0])
def test_angles_of_far_positions(freq):
    pos = np.array([0, 1, 2, 1000, 131071, 10 ** 6, 2 ** 30 + 1, 2 ** 31 - 1, -1, -77777, -2 ** 31], np.int64)
    q = torch.zeros((len(pos), 1, 2), device="cuda")
    q[..., 0] = 1.0
    got, _ = attn.attn_rope(q, None, torch.tensor([freq], dtype=torch.float64, device="cuda"),
                            positions=torch.from_numpy(pos.astype(np.int32)).cuda())
    x = q.double().cpu().numpy()
    want = ref.rope(x, pos, np.array([freq]), False, False, 1.0)
    assert (np.abs(got.double().cpu().numpy() - want) <= _tolerance(x, want, torch.float32, 1.0)).all()


@pytest.mark.parametrize("new,total", [((1, 1, 1), (5, 70000, 1)), ((0, 3, 0, 0, 4, 1, 0), (9, 3, 0, 8, 2, 100, 7)),
                                       ((200,), (131000,)), ((0,), (4,)), ((1, 0) * 500, (77,) * 1000), ((2,) * 8192, (9,) * 8192)])
def test_positions_of_a_step(new, total):
    T, D = sum(new) + 3, 64
    rng = np.random.Generator(np.random.PCG64(T))
    q, k = (torch.from_numpy(rng.standard_normal((T, H, D))).to(torch.float16).cuda() for H in (3, 1))
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    freq, _ = attn.attn_rope_frequencies(D)
    out = [torch.full_like(x, 7.0) for x in (q, k)]
    got = attn.attn_rope(q, k, freq, q_starts=torch.from_numpy(starts).cuda(),
                         total_lengths=torch.tensor(total, dtype=torch.int32, device="cuda"), q_out=out[0], k_out=out[1])
    assert got[0] is out[0] and got[1] is out[1]
    pos = np.concatenate([np.arange(t - n, t) for n, t in zip(new, total)]).astype(np.int32)
    n = sum(new)
    if n:
        want = attn.attn_rope(q[:n], k[:n], freq, positions=torch.from_numpy(pos).cuda())
        assert torch.equal(out[0][:n], want[0]) and torch.equal(out[1][:n], want[1])
    for x in out:
        assert bool((x[n:] == 7).all()), "rows of no request were written"


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("R", [128, 64, 6])
def test_in_place_in_a_fused_projection(layout, R):
    T, Hq, Hk, D = 37, 8, 2, 128
    rows = torch.randn((T, Hq + 2 * Hk, D), device="cuda").bfloat16()
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hk], rows[:, Hq + Hk:].clone()
    freq, _ = attn.attn_rope_frequencies(R)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 99
    want = attn.attn_rope(q, k, freq, positions=pos, layout=layout)
    assert attn.attn_rope(q, k, freq, positions=pos, layout=layout, q_out=q, k_out=k)[0] is q
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(rows[:, Hq + Hk:], v)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("R", [64, 48, 10])
def test_the_inverse_is_the_gradient(layout, R):
    T, H, D, scale = 11, 3, 64, 1.3
    rng = np.random.Generator(np.random.PCG64(R))
    x, dy, dx = (torch.from_numpy(rng.standard_normal((T, H, D))).float().cuda() for _ in range(3))
    freq, _ = attn.attn_rope_frequencies(R)
    pos = torch.from_numpy(rng.integers(0, 5000, T).astype(np.int32)).cuda()
    kw = dict(positions=pos, layout=layout, scale=scale)
    grad = attn.attn_rope(dy, None, freq, inverse=True, **kw)[0]
    # autograd over the formula, 64 bits
    y = x.double().cpu().requires_grad_()
    w = (pos.double()[:, None] * freq).cpu()[:, None]
    c, n = torch.cos(w) * scale, torch.sin(w) * scale
    i = torch.arange(R // 2)
    a, b = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + R // 2)
    turned = torch.cat([y[..., a] * c - y[..., b] * n, y[..., b] * c + y[..., a] * n], -1)
    order = torch.cat([a, b])
    d = dy.double().cpu()
    (turned * d[..., order]).sum().backward(retain_graph=True)
    want = y.grad.clone()
    want[..., R:] = d[..., R:]
    tol = _tolerance(d.numpy(), want.numpy(), torch.float32, scale)
    assert (np.abs(grad.double().cpu().numpy() - want.numpy()) <= tol).all()
    # differences: the map is linear, so f(x + dx) - f(x) = f(dx), and <f(dx), dy> = <dx, grad>
    f = lambda z: attn.attn_rope(z, None, freq, **kw)[0].double()  # noqa: E731
    left, right = ((f(x + dx) - f(x)) * dy.double()).sum(), (dx.double() * grad.double()).sum()
    # values up to 8 in size, off by 2^-19 each, summed over all
    assert abs(float(left - right)) <= T * H * D * 2.0 ** -16
    # there and back is scale^2 on what turns
    back = attn.attn_rope(attn.attn_rope(x, None, freq, **kw)[0], None, freq, inverse=True, **kw)[0].double().cpu()
    s = torch.ones(D, dtype=torch.float64)
    s[:R] = scale ** 2
    assert bool(((back - x.double().cpu() * s).abs() <= 2.0 ** -18 * x.abs().max().double().cpu() * scale ** 2).all())


def test_streams_and_graphs():
    q, k = torch.randn((50, 8, 128), device="cuda").half(), torch.randn((50, 2, 128), device="cuda").half()
    freq, _ = attn.attn_rope_frequencies(128)
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    want = attn.attn_rope(q, k, freq, positions=pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = attn.attn_rope(q, k, freq, positions=pos)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = attn.attn_rope(q, k, freq, positions=pos)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, other, made):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_refusals_of_the_binding():
    q, k = torch.randn((5, 4, 64), device="cuda"), torch.randn((5, 2, 64), device="cuda")
    f, pos = attn.attn_rope_frequencies(64)[0], torch.zeros(5, dtype=torch.int32, device="cuda")
    for bad in (lambda: attn.attn_rope(q, k, f), lambda: attn.attn_rope(q, k, f.float(), positions=pos),
                lambda: attn.attn_rope(q, k.half(), f, positions=pos), lambda: attn.attn_rope(q, k[:4], f, positions=pos),
                lambda: attn.attn_rope(q, k, f, positions=pos.long()), lambda: attn.attn_rope(q, k, f, positions=pos, layout="other"),
                lambda: attn.attn_rope(q, k, f, positions=pos, q_starts=pos, total_lengths=pos),
                lambda: attn.attn_rope(q, None, f, positions=pos, k_out=k), lambda: attn.attn_rope(q, k, f, q_starts=pos),
                lambda: attn.attn_rope(q.transpose(1, 2), None, f, positions=pos),
                lambda: attn.attn_rope(q, k, f, positions=pos, q_out=q.half())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: attn.attn_rope(q, k, attn.attn_rope_frequencies(66)[0], positions=pos),
                lambda: attn.attn_rope(q[:4], None, f, positions=pos[:4], q_out=q[1:])):
        with pytest.raises(attn.AttnError) as e:
            bad()
        assert e.value.status == attn.ATTN_ERR_INVALID_ARG
