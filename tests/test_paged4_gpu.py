"""The paged 4-bit KV cache on a GPU: append and read back bit for bit, attention
within derived tolerances, against plain 64-bit forms; a whole serving step
(blocks, rotary positions, append, attention) over a changing batch; captured,
on another stream, and with tables that name no block."""
import numpy as np
import pytest
import torch

import paged4_reference as ref
import tiled_online_softmax_02_gb300 as attn
from paged4_reference import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_online_softmax_02_gb300 import build
    build.build()
    attn.load_library()
    torch.cuda.set_device(0)


def gpu(a):
    return None if a is None else (torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else a).cuda()


# ---------------------------------------------------------- append and read
def _empty_cache(N, Hkv, block, D):
    rng = np.random.Generator(np.random.PCG64(N))
    shape = (N, Hkv, block, D // 2)
    return [rng.integers(0, 256, shape).astype(np.uint8) for _ in range(2)] + \
           [rng.integers(0, 127, (*shape[:3], D // 16)).astype(np.uint8) for _ in range(2)]


def _check_append(k, v, slots, cache, heads, strided=0):
    """Appends k, v (CPU tensors [T, Hkv, D]) on the GPU and in the reference; returns the GPU's cache."""
    wide = []
    for x in (k, v):
        y = torch.zeros((x.shape[0], x.shape[1] + strided, x.shape[2]), dtype=x.dtype)
        y[:, :x.shape[1]] = x
        wide.append(y.cuda()[:, :x.shape[1]])
    want = [c.copy() for c in cache]
    got = [gpu(c) for c in cache]
    kh, vh = heads
    attn.attn_cache_append_fp4(*wide, gpu(slots), *got, k_head_scales=gpu(kh), v_head_scales=gpu(vh))
    torch.cuda.synchronize()
    ref.append(k.double().numpy(), slots, want[0], want[2], kh)
    ref.append(v.double().numpy(), slots, want[1], want[3], vh)
    for name, g, w in zip(("k_cache", "v_cache", "k_scales", "v_scales"), got, want):
        differ = np.argwhere(g.cpu().numpy() != w)
        assert len(differ) == 0, f"{name}: {len(differ)} bytes, the first at {differ[:3].tolist()}"
    return got, want


HEADS = {"none": lambda H: (None, None),
         "powers": lambda H: tuple((2.0 ** np.arange(-3, H - 3)).astype(np.float32) for _ in range(2)),
         "any": lambda H: (np.linspace(0.1, 3.7, H).astype(np.float32), None)}


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Hkv,D,block", [(1, 64, 16), (3, 128, 32), (8, 128, 64), (2, 64, 128)])
@pytest.mark.parametrize("T", [1, 31, 333])
@pytest.mark.parametrize("heads", list(HEADS))
def test_append_and_read(dtype, Hkv, D, block, T, heads):
    rng = np.random.Generator(np.random.PCG64(T * D + Hkv))
    N = T // block + 5
    slots = rng.permutation(N * block)[:T].astype(np.int64)
    slots[rng.random(T) < 0.1] = -1
    if T > 3:
        slots[2], slots[3] = N * block, 2 ** 40  # no slots either
    x = [torch.from_numpy(rng.standard_normal((T, Hkv, D)) * np.exp(2 * rng.standard_normal((T, 1, 1)))).to(ref.TORCH[dtype])
         for _ in range(2)]
    hs = HEADS[heads](Hkv)
    got, want = _check_append(*x, slots, _empty_cache(N, Hkv, block, D), hs, strided=T % 2 * 2)
    # read some of those slots, twice each now and then, and other ones
    at = np.concatenate([slots, rng.integers(-3, N * block + 3, 50)]).astype(np.int64)
    there = (at >= 0) & (at < N * block)
    for to in ("bf16", "f16", "f32"):
        k, v = attn.attn_cache_read_fp4(*got, gpu(at), dtype=ref.TORCH[to], k_head_scales=gpu(hs[0]), v_head_scales=gpu(hs[1]))
        for y, c, s, h in ((k, want[0], want[2], hs[0]), (v, want[1], want[3], hs[1])):
            held = ref.values(c, s, h)[at[there] // block, :, at[there] % block]
            full = np.zeros((len(at), Hkv, D))
            full[there] = held
            # code * scale is exact; the head scale's product is rounded to f32 first
            assert torch.equal(y.cpu(), torch.from_numpy(full).float().to(ref.TORCH[to])), to


def test_read_into_head_major_rows():
    T, Hkv, D, block, N = 77, 3, 128, 32, 4
    cache = [gpu(c) for c in _empty_cache(N, Hkv, block, D)]
    slots = gpu(np.arange(T, dtype=np.int64))
    k, v = attn.attn_cache_read_fp4(*cache, slots, dtype=torch.float16)
    dense = torch.full((2, Hkv, 100, D), 7.0, dtype=torch.float16, device="cuda")
    out = [d[:, 5:5 + T].transpose(0, 1) for d in dense]
    attn.attn_cache_read_fp4(*cache, slots, k=out[0], v=out[1])
    assert torch.equal(out[0], k) and torch.equal(out[1], v)
    assert bool((dense[:, :, :5] == 7).all()) and bool((dense[:, :, 5 + T:] == 7).all())
    one = torch.zeros((1, Hkv, D), dtype=torch.float16, device="cuda")
    attn.attn_cache_read_fp4(*cache, slots[3:4], k=one, v=torch.empty_like(one))
    assert torch.equal(one[0], k[3])


@pytest.mark.parametrize("name", ["zeros", "tiny", "huge", "nonfinite", "edges", "subnormal"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("heads", list(HEADS))
def test_append_values(name, dtype, heads):
    T, Hkv, D, block, N = 40, 2, 64, 16, 4
    rng = np.random.Generator(np.random.PCG64(11))
    x = rng.standard_normal((2, T, Hkv, D))
    if name == "zeros":
        x[:, ::2] = 0.0
        x[:, 1::4] = -0.0
    elif name == "tiny":
        x *= 10.0 ** rng.uniform(-7, -2, (2, T, 1, 1))
    elif name == "huge":
        x *= 10.0 ** rng.uniform(2, 4.5 if dtype == "f16" else 37, (2, T, 1, 1))
    elif name == "nonfinite":
        x[rng.random(x.shape) < 0.02] = np.inf
        x[rng.random(x.shape) < 0.02] = -np.inf
        x[rng.random(x.shape) < 0.005] = np.nan
        x[:, 3] = np.inf
    elif name == "edges":  # on the borders between codes, for scales of every significand
        border = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
        s = (1 + rng.integers(0, 8, (2, T, Hkv, D // 16, 1)) / 8) * 2.0 ** rng.integers(-5, 5, (2, T, Hkv, D // 16, 1))
        g = rng.choice(border, (2, T, Hkv, D // 16, 16)) * rng.choice([-1, 1], (2, T, Hkv, D // 16, 16))
        g[..., 0] = 6.0
        x = (g * s).reshape(x.shape)
    else:
        x *= 2.0 ** (-20 if dtype == "f16" else -130)
    k, v = (torch.from_numpy(y).to(ref.TORCH[dtype]) for y in x)
    _check_append(k, v, rng.permutation(N * block)[:T].astype(np.int64), _empty_cache(N, Hkv, block, D), HEADS[heads](Hkv))


# --------------------------------------------------------------- attention
def _run(w, x, workspace=None, stream=None):
    g = {n: gpu(t) for n, t in x.items()}
    q = g["q"]
    if w.strided:
        wide = torch.zeros((q.shape[0], w.Hq + 2 * w.Hkv, w.D), dtype=q.dtype, device="cuda")
        wide[:, :w.Hq] = q
        q = wide[:, :w.Hq]
    out = torch.full((q.shape[0], w.Hq, w.D), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((q.shape[0], w.Hq), 7.0, device="cuda")
    attn.attn_fwd_paged_fp4(q, g["k_cache"], g["v_cache"], g["k_scales"], g["v_scales"], g["tables"], g["starts"],
                            g["totals"], k_head_scales=g["k_heads"], v_head_scales=g["v_heads"], causal=w.causal,
                            local_window=w.window, scale=w.scale, softcap=w.softcap, out=out, lse=lse,
                            workspace=workspace)
    torch.cuda.synchronize()
    return out, lse


def _compare(w, x, out, lse):
    want, wl, tol, ltol = ref.attend(w, x)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    rows = np.isnan(want).all((1, 2))
    assert (out[rows] == 7).all() and (lse[rows] == 7).all(), "rows of no request were written"
    ok = ~rows
    bad = ~(np.abs(out[ok] - want[ok]) <= tol[ok])
    assert not bad.any(), f"{bad.sum()} values, worst {np.nanmax(np.abs(out[ok] - want[ok]) / tol[ok]):.2f} tolerances"
    empty = np.isinf(wl[ok])
    assert (lse[ok][empty] == wl[ok][empty]).all()
    bad = ~(np.abs(lse[ok][~empty] - wl[ok][~empty]) <= ltol[ok][~empty])
    assert not bad.any(), f"lse: {bad.sum()} values"


def check(w):
    x = ref.make(w)
    out, lse = _run(w, x)
    assert attn.get_device_status() == attn.ATTN_OK
    _compare(w, x, out, lse)


HEADS_Q = [(1, 1), (4, 1), (8, 8), (15, 3), (12, 1), (32, 4), (16, 1), (9, 1), (40, 2)]


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64), ("bf16", 64), ("f16", 128)])
@pytest.mark.parametrize("Hq,Hkv", HEADS_Q)
def test_decode_heads(Hq, Hkv, dtype, D):
    check(Problem(new=(1, 1, 1), total=(300, 77, 1), Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, block=32))


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64), ("bf16", 64), ("f16", 128)])
@pytest.mark.parametrize("Hq,Hkv,block", [(4, 4, 16), (15, 3, 32), (40, 2, 128), (12, 1, 64)])
def test_many_rows_heads(Hq, Hkv, block, dtype, D):
    check(Problem(new=(80, 1, 200), total=(300, 77, 200), Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, block=block, wide=True))


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("total", [(1,), (127, 128, 129), (255, 256, 257, 15, 16, 17), (33, 2000)])
def test_decode_lengths(total, block):
    check(Problem(new=(1,) * len(total), total=total, block=block))


SHAPES = {
    "decode": dict(new=(1, 1, 1, 1), total=(1, 130, 700, 64)),
    "drafts": dict(new=(3, 0, 5, 1, 2), total=(3, 9, 600, 129, 260)),
    "prompts": dict(new=(100, 37), total=(100, 37)),
    "chunks": dict(new=(70, 1, 200, 0), total=(400, 900, 200, 50)),
    "more_new_than_total": dict(new=(5, 40, 3), total=(3, 20, 0)),
    "long_prompt": dict(new=(300,), total=(300,), Hq=16, Hkv=2),
}
FEATURES = {
    "plain": dict(), "full": dict(causal=False), "window": dict(window=50), "window_full": dict(window=33, causal=False),
    "window1": dict(window=1), "softcap": dict(softcap=5.0), "softcap_far": dict(softcap=1000.0, q_std=8.0),
    "scale": dict(scale=-0.2), "scale0": dict(scale=0.0), "strided_f16": dict(strided=True, dtype="f16"),
    "heads": dict(heads=True), "spread": dict(spread=True, scale=1e-5), "d64": dict(D=64, block=16, dtype="f16"),
    "d64_bf16": dict(D=64, block=128, window=100), "peaked": dict(q_std=12.0), "odd_group": dict(Hq=15, Hkv=3),
}


@pytest.mark.parametrize("feature", list(FEATURES))
@pytest.mark.parametrize("shape,wide", [(s, w) for s in SHAPES for w in (False, True) if not w or sum(SHAPES[s]["new"]) > 20])
def test_shapes_and_features(shape, wide, feature):
    check(Problem(**{**SHAPES[shape], **FEATURES[feature]}, wide=wide))


@pytest.mark.parametrize("feature", [dict(window=50), dict(window=1), dict(window=200, dtype="f16", heads=True),
                                     dict(window=33, causal=False), dict(window=300, D=64, softcap=5.0)], ids=str)
def test_windows_of_many_rows(feature):
    """Windows shorten what there may be to read, so it takes this many requests to fill the kernel for many rows."""
    new = tuple(100 + 37 * b % 56 for b in range(30))
    total = tuple(n + (0, 1, 90, 513)[b % 4] for b, n in enumerate(new))
    check(Problem(new=new, total=total, Hq=16, Hkv=8, **feature))


@pytest.mark.parametrize("new", [(5, 5, 7), (12, 1, 11), (3, 4, 5, 2)])
@pytest.mark.parametrize("feature", ["plain", "window", "d64_bf16", "d64", "odd_group"])
def test_units_of_8_and_of_16_rows(new, feature):
    """A mean of 23, 32 and 14 rows and a group that is no divisor of a unit; every request takes its own number of units."""
    check(Problem(**{**dict(new=new, total=tuple(300 * b + n for b, n in enumerate(new)), Hq=8, Hkv=2), **FEATURES[feature]}))


@pytest.mark.parametrize("new,Hq", [((300,) + (1,) * 100, 8), ((1,) * 40 + (500,) + (0,) * 9 + (1,) * 50 + (90,), 2),
                                    ((1,) * 150 + (400, 300) + (1,) * 148, 8), ((0,) * 33 + (350,), 6)],
                         ids=["first", "one_head_a_group", "300_requests", "alone"])
def test_prompts_among_single_tokens(new, Hq):
    """Requests of many units beside requests of one, in the kernel for few rows: 300 are more than a CTA has threads."""
    total = tuple(n + 7 * (b % 40) for b, n in enumerate(new))
    check(Problem(new=new, total=total, Hq=Hq, Hkv=2, D=64, block=32))


@pytest.mark.parametrize("new", [1, 3, 60, 200])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_one_key_far_above_the_others(new, dtype):
    check(Problem(new=(new,), total=(900,), dtype=dtype, sink=40.0, Hq=4, Hkv=1, wide=new == 200))


@pytest.mark.parametrize("new", [(2, 1), (150, 40)])
def test_growing_maximum(new):
    """Keys ever larger: every tile moves the running maximum."""
    w = Problem(new=new, total=(1100, 700), Hq=4, Hkv=1, dtype="f16", wide=True)
    x = ref.make(w)
    x["q"] = x["q"].abs()
    x["k_cache"] &= 0x77  # positive
    for b, t in enumerate(w.total):
        for p in range(t):
            x["k_scales"][int(x["tables"][b, p // w.block]), :, p % w.block] = 24 + min(p // 32, 60)
    out, lse = _run(w, x)
    _compare(w, x, out, lse)


def test_many_requests():
    rng = np.random.Generator(np.random.PCG64(4))
    n = 700
    check(Problem(new=tuple(rng.integers(0, 3, n)), total=tuple(rng.integers(2, 90, n)), Hq=2, Hkv=2, D=64, block=16))


def test_8192_requests():
    n = 8192
    check(Problem(new=(1,) * n, total=tuple(1 + np.arange(n) % 40), Hq=2, Hkv=1, D=64, block=16))


@pytest.mark.parametrize("new", [(1, 1), (70, 3)])
def test_tables_that_name_no_block_are_reported(new):
    w = Problem(new=new, total=(300, 200), block=32, wide=True)
    x = ref.make(w)
    x["tables"][0, 1] = -1
    x["tables"][1, 3] = x["k_cache"].shape[0]
    out, lse = _run(w, x)
    assert attn.get_device_status() == attn.ATTN_ERR_INVALID_ARG
    assert attn.get_device_status() == attn.ATTN_OK
    # the keys count as zeros
    y = {n: (None if t is None else t.clone()) for n, t in x.items()}
    grow = lambda t: torch.cat([t, torch.zeros_like(t[:1])])  # noqa: E731
    for n in ("k_cache", "v_cache", "k_scales", "v_scales"):
        y[n] = grow(y[n])
    y["tables"][0, 1] = y["tables"][1, 3] = y["k_cache"].shape[0] - 1
    _compare(w, y, out, lse)


@pytest.mark.parametrize("new", [(1, 1, 1), (200, 1, 33)])
def test_repeats_and_streams_give_the_same_bits(new):
    w = Problem(new=new, total=(2000, 300, 1000), Hq=8, Hkv=2, wide=True)
    x = ref.make(w)
    out, lse = _run(w, x)
    for _ in range(3):
        again = _run(w, x)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = _run(w, x)
    assert torch.equal(out, other[0]) and torch.equal(lse, other[1])


@pytest.mark.parametrize("new", [(2, 1), (80, 40)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rows_of_very_different_size_and_rows_not_finite(new, dtype):
    w = Problem(new=new, total=(400, 300), dtype=dtype, Hq=8, Hkv=2, wide=True)
    x = ref.make(w)
    e = torch.linspace(-100, 3, w.Hq) if dtype == "bf16" else torch.linspace(-12, 5, w.Hq)
    x["q"] = (x["q"].double() * 2.0 ** e.double()[None, :, None]).to(x["q"].dtype)
    out, lse = _run(w, x)
    _compare(w, x, out, lse)
    x["q"][0, 1, 5] = float("nan")
    x["q"][1, 6, 0] = float("inf")
    bad = _run(w, x)
    same = torch.ones(out.shape[:2], dtype=torch.bool)
    same[0, 1] = same[1, 6] = False
    assert torch.equal(bad[0].cpu()[same], out.cpu()[same]) and torch.equal(bad[1].cpu()[same], lse.cpu()[same])
    assert bool(bad[0][0, 1].isnan().all()) and bool(bad[0][1, 6].isnan().all())


@pytest.mark.parametrize("cap", [2.0, 50.0, 3e4, 1e30])
@pytest.mark.parametrize("new", [(2, 1), (150, 40)])
def test_soft_caps(cap, new):
    check(Problem(new=new, total=(500, 300), softcap=cap, q_std=20.0 if cap < 100 else 2.0, wide=True))


@pytest.mark.parametrize("new", [(2, 1), (150, 40)])
def test_caps_and_scales_at_their_ends(new):
    """Factors that pass fp32's range, either way: scores of zero stay zero, the others go to the cap's two ends or to zero."""
    w = Problem(new=new, total=(300, 200), wide=True, dtype="f16")
    x = ref.make(w)
    x["q"][:, 0] = 0.0
    for scale, cap in ((1e30, 1e-25), (1e-30, 1e30), (3e38, 1e-38)):
        out, lse = _run(w.replace(scale=scale, softcap=cap), x)
        assert bool(out[:sum(new)].isfinite().all()) and bool(lse[:sum(new)].isfinite().all())
        # caps of nothing leave every key its share, as does a scale of nothing
        want, _, tol, _ = ref.attend(w.replace(scale=0.0), x)
        rows = slice(0, sum(new))
        assert (np.abs(out.double().cpu().numpy()[rows] - want[rows]) <= 2 * tol[rows]).all()


@pytest.mark.parametrize("new", [(3, 4), (200, 100)])
def test_tables_without_blocks(new):
    w = Problem(new=new, total=(900, 400))
    x = ref.make(w)
    x["tables"] = x["tables"][:, :0].contiguous()
    out, lse = _run(w, x)
    n = sum(new)
    assert bool((out[:n] == 0).all()) and bool((lse[:n] == -np.inf).all()) and bool((out[n:] == 7).all())
    assert attn.get_device_status() == attn.ATTN_OK


def test_calls_without_rows():
    w = Problem(new=(3, 4), total=(90, 40))
    g = {n: gpu(t) for n, t in ref.make(w).items()}
    cache = [g[n] for n in ("k_cache", "v_cache", "k_scales", "v_scales")]
    before = [c.clone() for c in cache]
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    rows = torch.zeros((0, 2, 128), device="cuda")
    attn.attn_cache_append_fp4(rows, rows, none, *cache)
    assert [t.shape for t in attn.attn_cache_read_fp4(*cache, none)] == [(0, 2, 128)] * 2
    assert attn.attn_fwd_paged_fp4(g["q"][:0], *cache, g["tables"], g["starts"], g["totals"]).shape == (0, 8, 128)
    out = torch.full_like(g["q"], 7.0)
    empty = (g["tables"][:0], g["starts"][:1], g["totals"][:0])
    assert bool((attn.attn_fwd_paged_fp4(g["q"], *cache, *empty, out=out) == 7).all())
    freq = attn.attn_rope_frequencies(128)[0]
    assert attn.attn_rope(g["q"][:0], rows.bfloat16(), freq, positions=none.int())[0].shape == (0, 8, 128)
    assert bool((attn.attn_rope(g["q"], None, freq, q_starts=empty[1], total_lengths=empty[2], q_out=out)[0] == 7).all())
    torch.cuda.synchronize()
    for a, b in zip(before, cache):
        assert torch.equal(a, b)


def test_caller_workspace_and_float_views():
    w = Problem(new=(3, 4), total=(900, 40))
    x = ref.make(w)
    out, lse = _run(w, x)
    n = attn.attn_paged_fp4_workspace_bytes(x["q"].shape[0], 2, w.Hq, w.Hkv, w.D)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(_run(w, x, workspace=ws)[0], out)
    for s in ("k_scales", "v_scales"):
        x[s] = x[s].view(torch.float8_e4m3fn)
    if hasattr(torch, "float4_e2m1fn_x2"):
        for c in ("k_cache", "v_cache"):
            x[c] = x[c].view(torch.float4_e2m1fn_x2)
    assert torch.equal(_run(w, x)[0], out)


def test_refusals_of_the_binding():
    w = Problem(new=(3, 4), total=(90, 40))
    g = {n: gpu(t) for n, t in ref.make(w).items()}
    cache = [g[n] for n in ("k_cache", "v_cache", "k_scales", "v_scales")]
    rest = (g["tables"], g["starts"], g["totals"])
    call = attn.attn_fwd_paged_fp4
    for bad in (lambda: call(g["q"].float(), *cache, *rest), lambda: call(g["q"][..., :64], *cache, *rest),
                lambda: call(g["q"], *cache[:3], cache[3].float(), *rest), lambda: call(g["q"], *cache, *rest[:2], rest[2][:1]),
                lambda: call(g["q"], *cache, *rest, k_head_scales=torch.ones(3, device="cuda")),
                lambda: call(g["q"], *cache, *rest, out=torch.empty(3, device="cuda")),
                lambda: call(g["q"], *cache, *rest, workspace=torch.empty(8)),
                lambda: attn.attn_cache_read_fp4(*cache, g["starts"]),
                lambda: attn.attn_cache_read_fp4(*cache, g["starts"].long(), k=g["q"]),
                lambda: attn.attn_cache_read_fp4(*cache, g["starts"].long(), dtype=torch.float64),
                lambda: attn.attn_cache_append_fp4(g["q"], g["q"], torch.zeros(10, dtype=torch.int64, device="cuda"), *cache)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(attn.AttnError) as e:
        call(g["q"], *cache, *rest, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == attn.ATTN_ERR_INVALID_ARG


class _Ordinary:
    """The extension module, which must take the calls made through it."""

    def __init__(self, calls):
        self.calls, self.taken = calls, 0

    def __getattr__(self, name):
        def call(*args):
            made = getattr(self.calls, name)(*args)
            self.taken += made is not None
            return made
        return call


class _Nothing:
    """An extension module that takes no call."""

    def __getattr__(self, name):
        return lambda *args: None


@pytest.mark.parametrize("heads", [False, True])
def test_both_ways_of_marshalling(monkeypatch, heads):
    """Calls through the extension module and those that Python marshals: the same results and the same errors."""
    from tiled_online_softmax_02_gb300 import _binding
    w = Problem(new=(3, 4), total=(90, 40), heads=heads, window=30, softcap=20.0, strided=True)
    g = {n: gpu(t) for n, t in ref.make(w).items()}
    h = dict(k_head_scales=g["k_heads"], v_head_scales=g["v_heads"])
    freq = attn.attn_rope_frequencies(64)[0]
    slots = torch.tensor([5, 900000, 7, -1, 3, 66, 68], device="cuda")
    wide = torch.zeros((10, 12, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, :8] = g["q"]

    def everything():
        made = []
        cache = [g[n].clone() for n in ("k_cache", "v_cache", "k_scales", "v_scales")]
        made += attn.attn_rope(wide[:, :8], wide[:, 8:10], freq, positions=torch.arange(10, dtype=torch.int32, device="cuda"), scale=1.5)
        made += attn.attn_rope(g["q"], None, freq, q_starts=g["starts"], total_lengths=g["totals"], inverse=True, layout="interleaved",
                               q_out=torch.zeros_like(g["q"]))[:1]
        attn.attn_cache_append_fp4(wide[:7, :2], wide[:7, 2:4], slots, *cache, **h)
        made += cache
        made += attn.attn_cache_read_fp4(*cache, slots, dtype=torch.float16, **h)
        made.append(attn.attn_fwd_paged_fp4(wide[:, :8], *cache, g["tables"], g["starts"], g["totals"], local_window=w.window,
                                            softcap=w.softcap, scale=0.1, out=torch.full_like(g["q"], 7.0), **h))
        made.append(attn.attn_fwd_paged_fp4(g["q"], *cache, g["tables"], g["starts"], g["totals"], causal=False, **h)[:7])
        errors = []
        for bad in (lambda: attn.attn_fwd_paged_fp4(g["q"], *cache, g["tables"], g["starts"], g["totals"], scale=float("nan")),
                    lambda: attn.attn_rope(g["q"], None, freq, positions=g["totals"]),
                    lambda: attn.attn_rope(g["q"], None, torch.cat([freq] * 3), positions=torch.zeros(10, dtype=torch.int32, device="cuda")),
                    lambda: attn.attn_cache_read_fp4(*cache, slots.int()),
                    lambda: attn.attn_cache_append_fp4(wide[:7, :2], wide[:7, 2:4], slots[:3], *cache)):
            with pytest.raises((ValueError, attn.AttnError)) as e:
                bad()
            errors.append(str(e.value))
        torch.cuda.synchronize()
        return made, errors

    ordinary = _Ordinary(_binding._calls)
    monkeypatch.setattr(_binding, "_calls", ordinary)
    a, ae = everything()
    assert ordinary.taken == 8  # six results, and two statuses of the C ABI
    monkeypatch.setattr(_binding, "_calls", _Nothing())
    b, be = everything()
    assert ae == be and len(a) == len(b)
    for x, y in zip(a, b):
        assert x.dtype == y.dtype and torch.equal(x, y)


# ---------------------------------------------------------- a serving step
class Batch:
    """A batch's state on the GPU, and in plain numpy beside it."""

    def __init__(self, B=5, width=20, block=16, N=70, Hq=8, Hkv=2, D=64, dtype="bf16", layout="half", rotary=64):
        self.B, self.width, self.block, self.N, self.Hq, self.Hkv, self.D = B, width, block, N, Hq, Hkv, D
        self.dtype, self.layout = ref.TORCH[dtype], layout
        self.w = Problem(new=(), total=(), Hq=Hq, Hkv=Hkv, D=D, block=block, dtype=dtype)
        self.tables = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.free = torch.arange(N, dtype=torch.int32, device="cuda")
        self.count = torch.tensor([N], dtype=torch.int32, device="cuda")
        self.cache = [gpu(c) for c in _empty_cache(N, Hkv, block, D)]
        self.held = [c.cpu().numpy() for c in self.cache]
        self.past = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.freq, self.scale = attn.attn_rope_frequencies(rotary, scaling="parts", factor=4.0, original_length=512)

    def step(self, q, k, v, new, finished, T):
        """Blocks, rotary positions, the cache, attention: GPU calls only."""
        starts, total, slots, result = attn.attn_cache_assign(self.past, new, self.tables, self.free, self.count,
                                                              block_size=self.block, num_tokens=T, finished=finished)
        qr, kr = attn.attn_rope(q, k, self.freq, q_starts=starts, total_lengths=total, layout=self.layout, scale=self.scale,
                                q_out=torch.zeros_like(q), k_out=torch.zeros_like(k))
        attn.attn_cache_append_fp4(kr, v, slots, *self.cache)
        out = attn.attn_fwd_paged_fp4(qr, *self.cache, self.tables, starts, total, out=torch.full_like(q, 7.0))
        self.past.copy_(total)
        return dict(starts=starts, total=total, slots=slots, result=result, qr=qr, kr=kr, out=out)

    def verify(self, made, q, k, v):
        assert int(made["result"][0]) == 0
        starts, total = made["starts"].cpu().numpy(), made["total"].cpu().numpy()
        n = int(starts[-1])
        pos = np.concatenate([np.arange(t - (z - a), t) for a, z, t in zip(starts, starts[1:], total)] or [np.zeros(0)])
        # turned rows: an error of 2^-23 for the angle's sine and cosine, the products and the sum, then a rounding
        for x, y in ((q, made["qr"]), (k, made["kr"])):
            x, y = x[:n].double().cpu().numpy(), y[:n].double().cpu().numpy()
            want = ref.rope(x, pos, self.freq.cpu().numpy(), self.layout == "interleaved", False, self.scale)
            size = np.abs(x).max(-1, keepdims=True)
            tol = torch.finfo(self.dtype).eps / 2 * np.abs(want) + 2.0 ** -20 * size
            assert (np.abs(y - want) <= tol).all()
        slots = made["slots"].cpu().numpy()
        ref.append(made["kr"].double().cpu().numpy(), slots, self.held[0], self.held[2])
        ref.append(v.double().cpu().numpy(), slots, self.held[1], self.held[3])
        for g, h in zip(self.cache, self.held):
            assert np.array_equal(g.cpu().numpy(), h)
        x = dict(q=made["qr"].cpu(), k_cache=torch.from_numpy(self.held[0]), v_cache=torch.from_numpy(self.held[1]),
                 k_scales=torch.from_numpy(self.held[2]), v_scales=torch.from_numpy(self.held[3]), k_heads=None,
                 v_heads=None, tables=self.tables.cpu(), starts=made["starts"].cpu(), totals=made["total"].cpu())
        want, _, tol, _ = ref.attend(self.w, x)
        out = made["out"].double().cpu().numpy()
        assert (out[n:] == 7).all()
        assert (np.abs(out[:n] - want[:n]) <= tol[:n]).all()

    def rows(self, rng, T):
        r = lambda H: torch.from_numpy(rng.standard_normal((T, H, self.D))).to(self.dtype).cuda()  # noqa: E731
        return r(self.Hq), r(self.Hkv), r(self.Hkv)


STEPS = [([40, 1, 0, 7, 100], [0] * 5), ([1, 1, 90, 1, 1], [0] * 5), ([1, 2, 1, 30, 5], [1, 0, 0, 1, 0]), ([1] * 5, [0] * 5)]


@pytest.mark.parametrize("kw", [dict(), dict(block=64, D=128, dtype="f16", Hq=8, Hkv=1, N=40, width=9, layout="interleaved", rotary=32)])
def test_steps_of_a_batch(kw):
    batch, rng = Batch(**kw), np.random.Generator(np.random.PCG64(2))
    for new, fin in STEPS:
        T = sum(new) + 4
        q, k, v = batch.rows(rng, T)
        made = batch.step(q, k, v, gpu(np.array(new, np.int32)), gpu(np.array(fin, np.uint8)), T)
        torch.cuda.synchronize()
        batch.verify(made, q, k, v)


def test_captured_steps_of_a_batch():
    batch, rng, T = Batch(), np.random.Generator(np.random.PCG64(3)), 160
    q, k, v = batch.rows(rng, T)
    new, fin = (torch.zeros(5, dtype=t, device="cuda") for t in (torch.int32, torch.uint8))
    batch.step(q, k, v, new, fin, T)  # first calls on the device, before capturing
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = batch.step(q, k, v, new, fin, T)
    for n, f in STEPS:
        for x, y in zip((q, k, v), batch.rows(rng, T)):
            x.copy_(y)
        new.copy_(torch.tensor(n, dtype=torch.int32))
        fin.copy_(torch.tensor(f, dtype=torch.uint8))
        graph.replay()
        torch.cuda.synchronize()
        batch.verify(made, q, k, v)


def test_prompt_read_back_for_dense_attention():
    """A prompt's dense attention over what the cache holds equals the paged attention over it."""
    T, Hq, Hkv, D, block = 200, 8, 2, 128, 64
    rng = np.random.Generator(np.random.PCG64(8))
    r = lambda H: torch.from_numpy(rng.standard_normal((T, H, D))).to(torch.float16).cuda()  # noqa: E731
    q, k, v = r(Hq), r(Hkv), r(Hkv)
    N = 6
    cache = [gpu(c) for c in _empty_cache(N, Hkv, block, D)]
    tables = gpu(np.array([[4, 1, 5, 0]], np.int32))
    pos = torch.arange(T, device="cuda")
    slots = tables[0, pos // block].long() * block + pos % block
    attn.attn_cache_append_fp4(k, v, slots, *cache)
    dense = torch.zeros((2, 1, Hkv, 256, D), dtype=torch.float16, device="cuda")
    attn.attn_cache_read_fp4(*cache, slots, k=dense[0, 0, :, :T].transpose(0, 1), v=dense[1, 0, :, :T].transpose(0, 1))
    a = attn.attn_fwd(q.transpose(0, 1)[None].contiguous(), dense[0], dense[1], causal=True, seq_k=T)[0].transpose(0, 1)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    b = attn.attn_fwd_paged_fp4(q, *cache, tables, i32(0, T), i32(T))
    # the dense kernel rounds the weights to f16 too (2^-11 each), and both the results
    assert bool(((a - b).abs().double() <= 4 * 2.0 ** -11 * (1 + v.abs().max().double())).all())


@pytest.mark.parametrize("new", [(1, 2, 1), (150, 1, 20)])
def test_blocks_past_four_gigabytes(new):
    """A cache whose blocks lie past 2^32 bytes: its first and last blocks are used."""
    w = Problem(new=new, total=(300, 90, 130), block=128, Hq=8, Hkv=8, wide=True)
    x = ref.make(w)
    per = w.Hkv * w.block * w.D // 2
    N = (5 << 30) // per
    few = x["k_cache"].shape[0]
    tables = x["tables"].clone()
    inside = (tables >= 0) & (tables < few)
    far = torch.where(inside & (tables % 2 == 0), N - 1 - tables, torch.where(inside, tables, torch.full_like(tables, -1)))
    out, lse = _run(w, x)
    big = {}
    for n in ("k_cache", "v_cache", "k_scales", "v_scales"):
        t = torch.empty((N, *x[n].shape[1:]), dtype=torch.uint8, device="cuda")
        for i in range(few):
            t[N - 1 - i if i % 2 == 0 else i] = x[n][i].cuda()
        big[n] = t
    y = dict(x, **big, tables=far.int())
    o2, l2 = _run(w, y)
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    # and the writer and the reader of such a cache
    slots = torch.tensor([(N - 1) * 128 + 127, 5, (N - 1) * 128], device="cuda")
    k, v = (torch.randn((3, 8, 128), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    cache = [big[n] for n in ("k_cache", "v_cache", "k_scales", "v_scales")]
    attn.attn_cache_append_fp4(k, v, slots, *cache)
    got = attn.attn_cache_read_fp4(*cache, slots)
    for a, b in zip(got, (k, v)):
        code, byte = ref.quantise(b.double().cpu().numpy())
        want = np.stack([ref.values(ref.pack(code[i])[None, :, None], byte[i][None, :, None])[0, :, 0] for i in range(3)])
        assert np.array_equal(a.double().cpu().numpy(), want)


def test_two_graphs_replayed_at_once():
    """Two captured calls, each with a workspace of its own, replayed on two streams at once."""
    problems = [Problem(new=(1,) * 4, total=(3000, 2000, 100, 900), Hq=8, Hkv=2, seed=s) for s in (1, 2)]
    made = []
    for w in problems:
        x = ref.make(w)
        want, _ = _run(w, x)
        g = {n: gpu(t) for n, t in x.items()}
        out = torch.full_like(want, 7.0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            attn.attn_fwd_paged_fp4(g["q"], g["k_cache"], g["v_cache"], g["k_scales"], g["v_scales"], g["tables"], g["starts"],
                                    g["totals"], out=out)
        made.append((graph, out, want, g, torch.cuda.Stream()))
    for _ in range(20):
        for graph, out, _, _, s in made:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, out, want, _, _ in made:
        assert torch.equal(out, want)
