"""The paged 8-bit KV cache on a GPU: block assignment and quantised append bit
for bit, and attention within derived tolerances, against plain 64-bit forms;
the three together over steps of a changing batch; captured, on another
stream, and with tables that name no block."""
import numpy as np
import pytest
import torch

import paged_reference as ref
import tiled_online_softmax_02_gb300 as attn
from paged_reference import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_online_softmax_02_gb300 import build
    build.build()
    attn.load_library()
    torch.cuda.set_device(0)


# ------------------------------------------------------------------ assign
def _assign_state(B, width, block, past, seed, spare):
    rng = np.random.Generator(np.random.PCG64(seed))
    held = -(-past.astype(np.int64) // block)
    N = int(held.sum()) + spare
    pool = rng.permutation(N).astype(np.int32)
    tables = np.full((B, width), -1, np.int32)
    at = 0
    for b, n in enumerate(held):
        tables[b, :n] = pool[at:at + n]
        at += n
    free = np.full(N, -1, np.int32)
    free[:spare] = pool[at:]
    return tables, free, spare


def _run_assign(past, new, finished, tables, free, count, block, T):
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    g = [d(past), d(new), d(tables), d(free), d(np.array([count], np.int32))]
    made = attn.attn_cache_assign(*g, block_size=block, num_tokens=T,
                                  finished=None if finished is None else d(finished))
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in (*made, g[2], g[3], g[4])], g


@pytest.mark.parametrize("B,width,block,past_max,new_max,pad,fin", [
    (1, 1, 16, 0, 1, 0, 0.0), (1, 40, 16, 500, 100, 0, 0.0), (7, 9, 128, 900, 200, 5, 0.3),
    (64, 128, 64, 8000, 1, 0, 0.05), (33, 70, 32, 2000, 1, 31, 1.0), (300, 20, 16, 250, 40, 1000, 0.5),
    (3, 2100, 32, 100, 66000, 9, 0.4), (8192, 3, 16, 40, 2, 0, 0.2), (31, 8, 64, 0, 0, 4, 0.0),
])
def test_assign(B, width, block, past_max, new_max, pad, fin):
    rng = np.random.Generator(np.random.PCG64(B * 131 + width))
    past = rng.integers(0, past_max + 1, B).astype(np.int32)
    new = rng.integers(0, new_max + 1, B).astype(np.int32)
    finished = rng.random(B) < fin if fin > 0 else None
    tables, free, count = _assign_state(B, width, block, past, 3, int((-(-new // block) + 1).sum()) + 2)
    T = int(new.sum()) + pad
    got, _ = _run_assign(past, new, finished, tables, free, count, block, T)
    tb, fr = tables.copy(), free.copy()
    fin_ = np.zeros(B, bool) if finished is None else finished
    starts, totals, slots, result, n = ref.assign(past, new, fin_, tb, fr, count, block, T)
    assert result == 0 and got[3][0] == 0
    for a, b in zip(got, (starts, totals, slots, None, tb, fr, None)):
        if b is not None:
            assert np.array_equal(a, b)
    assert got[6][0] == n
    # no block is held twice, none is held and free
    live = tb[tb >= 0]
    assert len(np.unique(np.concatenate([live, fr[:n]]))) == len(live) + n


def test_assign_twice_keeps_the_blocks():
    past, new = np.array([5, 64, 0], np.int32), np.array([70, 1, 3], np.int32)
    tables, free, count = _assign_state(3, 4, 64, past, 1, 6)
    first, g = _run_assign(past, new, None, tables, free, count, 64, 80)
    again = attn.attn_cache_assign(*g, block_size=64, num_tokens=80)
    for a, b in zip(first, (*again, g[2], g[3], g[4])):
        assert np.array_equal(a, b.cpu().numpy())


@pytest.mark.parametrize("why,kw", [
    (1, dict(spare=1)), (2, dict(width=2)), (3, dict(T=100)), (4, dict(new=[-1, 3, 3])), (4, dict(past=[7, -1, 9])),
])
def test_assign_steps_that_cannot_be_done_change_nothing(why, kw):
    past = np.array(kw.get("past", [7, 100, 0]), np.int32)
    new = np.array(kw.get("new", [10, 30, 90]), np.int32)
    finished = np.array([False, True, False])
    tables, free, count = _assign_state(3, kw.get("width", 5), 32, np.minimum(np.maximum(past, 0), 60), 1, kw.get("spare", 9))
    if why == 1:
        finished[:] = False
    got, _ = _run_assign(past, new, finished, tables, free, count, 32, kw.get("T", 140))
    starts, totals, slots, result, n = ref.assign(past, new, finished, tables.copy(), free.copy(), count, 32, kw.get("T", 140))
    assert result == why and got[3][0] == why
    assert np.array_equal(got[4], tables) and np.array_equal(got[5], free) and got[6][0] == count
    assert (got[0] == 0).all() and np.array_equal(got[1], past) and (got[2] == -1).all()


@pytest.mark.parametrize("bad", ["count_high", "count_negative", "entry"])
def test_assign_refuses_lists_out_of_range(bad):
    past, new = np.array([64, 3], np.int32), np.array([1, 1], np.int32)
    tables, free, count = _assign_state(2, 3, 64, past, 1, 4)
    if bad == "entry":
        tables[0, 0] = len(free)
    else:
        count = len(free) + 1 if bad == "count_high" else -1
    got, _ = _run_assign(past, new, None, tables, free, count, 64, 2)
    assert got[3][0] == 5 and np.array_equal(got[4], tables) and got[6][0] == count


def test_assign_without_requests():
    z = np.zeros(0, np.int32)
    got, _ = _run_assign(z, z, None, np.zeros((0, 4), np.int32), np.arange(5, dtype=np.int32), 5, 64, 7)
    assert got[0].tolist() == [0] and (got[2] == -1).all() and got[3][0] == 0 and got[6][0] == 5


# ------------------------------------------------------------------ append
def _append_case(new, past, Hkv, D, block, dtype, seed=1, spread=1.0, fill=None, strided=False):
    rng = np.random.Generator(np.random.PCG64(seed))
    held = [-(-(p + n) // block) for p, n in zip(past, new)]
    N = sum(held) + 2
    pool = rng.permutation(N)
    slots, at = [], 0
    for p, n, hb in zip(past, new, held):
        pos = p + np.arange(n)
        slots.append(pool[at:at + hb][pos // block] * block + pos % block if n else np.zeros(0, np.int64))
        at += hb
    slots = np.concatenate(slots).astype(np.int64)
    T = len(slots)
    x = rng.standard_normal((2, T, Hkv, D)) * np.exp(spread * rng.standard_normal((2, T, Hkv, 1)))
    if fill is not None:
        fill(x, rng)
    kv = [torch.from_numpy(a).to(ref.TORCH[dtype]) for a in x]
    caches = [torch.from_numpy(rng.integers(0, 127, (N, Hkv, block, D), dtype=np.uint8)) for _ in range(2)]
    scales = [torch.from_numpy((2.0 ** rng.integers(-9, 2, (N, Hkv))).astype(np.float32)) for _ in range(2)]
    return kv, torch.from_numpy(slots), caches, scales


def _check_append(kv, slots, caches, scales, strided=False):
    want_c = [c.numpy().copy() for c in caches]
    want_s = [s.double().numpy().copy() for s in scales]
    for x, c, s in zip(kv, want_c, want_s):
        ref.append(x.double().numpy(), slots.numpy(), c, s)
    if strided:  # a token's rows inside a wider projection
        wide = [torch.full((x.shape[0], 3 * x.shape[1], x.shape[2]), float("nan"), dtype=x.dtype, device="cuda")
                for x in kv]
        g = []
        for y, x in zip(wide, kv):
            y[:, x.shape[1]:2 * x.shape[1]] = x.cuda()
            g.append(y[:, x.shape[1]:2 * x.shape[1]])
    else:
        g = [x.cuda() for x in kv]
    gc = [c.cuda() for c in caches]
    gs = [s.cuda() for s in scales]
    attn.attn_cache_append_fp8(*g, slots.cuda(), *gc, *gs)
    torch.cuda.synchronize()
    for a, b in zip(gs, want_s):
        assert np.array_equal(a.double().cpu().numpy(), b)
    for a, b in zip(gc, want_c):
        a = a.cpu().numpy()
        nan = (b & 127) == 127
        assert np.array_equal((a & 127) == 127, nan)
        a, b = np.where(nan, 0, a), np.where(nan, 0, b)
        # zeros of either sign are the same value
        assert np.array_equal(np.where(a == 128, 0, a), np.where(b == 128, 0, b))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Hkv,D,block", [(1, 64, 16), (3, 128, 32), (8, 128, 64), (2, 64, 128)])
@pytest.mark.parametrize("shape", ["decode", "ragged", "prompts", "one"])
def test_append(dtype, Hkv, D, block, shape):
    new, past = {"decode": ([1] * 37, [i * 7 for i in range(37)]),
                 "ragged": ([3, 0, 17, 1, 130, 5, 4, 6], [0, 9, block - 1, block, 5, 2 * block - 3, 13, 1]),
                 "prompts": ([2 * block + 5, 1100, block], [0, 0, 0]), "one": ([1], [0])}[shape]
    _check_append(*_append_case(new, past, Hkv, D, block, dtype), strided=shape != "prompts")


@pytest.mark.parametrize("name", ["zeros", "tiny", "huge", "nonfinite", "edge", "ties"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_values(name, dtype):
    def fill(x, rng):
        if name == "zeros":
            x[:, ::2] = 0.0
        elif name == "tiny":
            x *= 1e-37
        elif name == "huge":
            x *= 1e36
        elif name == "nonfinite":
            x[rng.random(x.shape) < 0.05] = np.inf
            x[rng.random(x.shape) < 0.05] = np.nan
            x[0, 3] = np.nan
        elif name == "edge":  # exactly 448 scales, and one step above
            x[..., 0] = 1.75 * 2.0 ** rng.integers(-6, 7, x.shape[:-1])
            x[:, ::3, :, 0] *= 1 + 2.0 ** -7
        else:  # halfway between two e4m3 values, subnormal ones among them
            x[:] = (rng.integers(0, 400, x.shape) + 0.5) * 2.0 ** rng.integers(-9, 1, x.shape)
    _check_append(*_append_case([1, 40, 1, 3, 64, 200], [0, 7, 63, 64, 0, 30], 2, 128, 64, dtype, fill=fill))


def test_append_passes_over_slots_of_no_block():
    kv, slots, caches, scales = _append_case([1, 40, 9], [3, 7, 0], 2, 64, 16, "f16")
    slots[[0, 5, 20, 49]] = torch.tensor([-1, -1, caches[0].shape[0] * 16, 2 ** 40])
    _check_append(kv, slots, caches, scales)


# --------------------------------------------------------------- attention
def _gpu(x, strided=False):
    g = {k: v.cuda() for k, v in x.items()}
    if strided:
        T, H, D = x["q"].shape
        wide = torch.full((T, H + 4, D), float("nan"), dtype=x["q"].dtype, device="cuda")
        wide[:, :H] = g["q"]
        g["q"] = wide[:, :H]
    return g


def _attend(w, g, out=None, lse=None, **kw):
    return attn.attn_fwd_paged_fp8(g["q"], g["k_cache"], g["v_cache"], g["k_scales"], g["v_scales"], g["tables"],
                                   g["starts"], g["totals"], causal=w.causal, local_window=w.window, scale=w.scale,
                                   softcap=w.softcap, out=out, lse=lse, **kw)


def _check_out(w, x, out, lse, mark=-7.0):
    want, want_lse, tol, ltol = ref.attend(w, x)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    none = np.isnan(want)
    assert (out[none] == mark).all() and (lse[np.isnan(want_lse)] == mark).all()  # rows of no request
    err = np.where(none, 0.0, np.abs(out - np.where(none, 0.0, want)))
    assert not np.isnan(err).any()
    bad = err > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, worst {np.max(err / np.maximum(tol, 1e-30)):.2f} tolerances"
    fin = np.isfinite(want_lse)
    assert (lse[np.isneginf(want_lse)] == -np.inf).all()
    assert (np.abs(lse[fin] - want_lse[fin]) <= ltol[fin]).all(), np.max(np.abs(lse[fin] - want_lse[fin]) / ltol[fin])


def _check(w):
    x = ref.make(w)
    g = _gpu(x, w.strided)
    out = torch.full(x["q"].shape, -7.0, dtype=x["q"].dtype, device="cuda")
    lse = torch.full(x["q"].shape[:2], -7.0, device="cuda")
    _attend(w, g, out, lse)
    torch.cuda.synchronize()
    assert attn.get_device_status() == attn.ATTN_OK
    _check_out(w, x, out, lse)
    return g, out


BASE = Problem(new=(1, 1, 1, 1), total=(1, 130, 700, 64))
HEADS = [(4, 4), (2, 1), (15, 3), (8, 2), (12, 1), (16, 1), (17, 1), (32, 4), (64, 2)]


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64), ("bf16", 64), ("f16", 128)])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_decode_heads(Hq, Hkv, dtype, D):
    _check(BASE.replace(Hq=Hq, Hkv=Hkv, dtype=dtype, D=D, total=(1, 130, 300, 64)))


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("total", [(1,), (127, 128, 129), (255, 256, 257, 15, 16, 17), (2000,)])
def test_decode_lengths(total, block):
    _check(BASE.replace(new=(1,) * len(total), total=total, block=block))


SHAPES = {
    "verify": dict(new=(3, 1, 5, 2, 4), total=(3, 200, 131, 2, 1000)),
    "none_new": dict(new=(0, 2, 0, 0, 1, 0), total=(50, 20, 0, 128, 1, 1)),
    "chunk": dict(new=(100, 37), total=(300, 37)),
    "chunk_short": dict(new=(40, 1, 3), total=(40, 500, 130)),
    "prompt": dict(new=(257,), total=(257,)),
    "mixed": dict(new=(1, 300, 1, 1), total=(900, 420, 7, 128)),
    "rows_before_the_start": dict(new=(9, 4), total=(3, 0)),  # more rows than the cache holds: the first see nothing
}
FEATURES = {
    "plain": {}, "f16_d64": dict(dtype="f16", D=64), "window": dict(window=50), "window_wide": dict(window=300),
    "softcap": dict(softcap=3.0, q_std=3.0), "not_causal": dict(causal=False),
    "not_causal_window": dict(causal=False, window=17, dtype="f16"), "scale": dict(scale=0.31),
    "negative_scale": dict(scale=-0.1), "free_scales": dict(free_scales=True), "strided": dict(strided=True),
    "block16": dict(block=16, D=64), "block128": dict(block=128, dtype="f16"), "sharp": dict(q_std=8.0),
    "mha": dict(Hq=3, Hkv=3), "group_of_15": dict(Hq=15, Hkv=1, dtype="f16"),
    "window_softcap": dict(window=100, softcap=20.0, q_std=4.0, D=64),
}


@pytest.mark.parametrize("feature", list(FEATURES))
@pytest.mark.parametrize("shape", list(SHAPES))
def test_shapes_and_features(shape, feature):
    _check(Problem(**SHAPES[shape]).replace(**FEATURES[feature]))


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_one_key_far_above_the_others(new, dtype):
    """The first key's score lies well above all others and its V row is small:
    what the many light keys add has to survive next to it."""
    _check(Problem(new=(new,), total=(3000,), Hq=4, Hkv=1, dtype=dtype, sink=14.0))


def test_growing_maximum():
    """Scores that grow from key to key, so the running maximum moves in every tile."""
    w = BASE.replace(new=(2, 40), total=(900, 700), Hq=4, Hkv=2)
    x = ref.make(w)
    x["q"] = x["q"].abs()
    for b, t in enumerate(w.total):
        for p in range(t):
            blk = int(x["tables"][b, p // w.block])
            x["k_cache"][blk, :, p % w.block] = int(ref.encode(np.array([2.0 + p / 8]))[0])
            x["k_scales"][blk] = 2.0 ** -4
    g = _gpu(x)
    out = torch.full(x["q"].shape, -7.0, dtype=x["q"].dtype, device="cuda")
    lse = torch.full(x["q"].shape[:2], -7.0, device="cuda")
    _attend(w, g, out, lse)
    _check_out(w, x, out, lse)


def test_zero_scales():
    """Blocks whose scale is 0: their keys score 0 and add nothing."""
    w = BASE.replace(new=(1, 30), total=(300, 200))
    x = ref.make(w)
    x["k_scales"][::2] = 0.0
    x["v_scales"][1::2] = 0.0
    g = _gpu(x)
    out = torch.full(x["q"].shape, -7.0, dtype=x["q"].dtype, device="cuda")
    lse = torch.full(x["q"].shape[:2], -7.0, device="cuda")
    _attend(w, g, out, lse)
    _check_out(w, x, out, lse)


@pytest.mark.parametrize("new", [(1, 1), (70, 3)])
def test_tables_that_name_no_block_are_reported(new):
    w = BASE.replace(new=new, total=(500, 300))
    x = ref.make(w)
    x["tables"][0, 2] = -1
    g = _gpu(x)
    out = _attend(w, g)
    assert attn.get_device_status() == attn.ATTN_ERR_INVALID_ARG
    assert attn.get_device_status() == attn.ATTN_OK
    x["tables"] = ref.make(w)["tables"]
    whole = _attend(w, _gpu(x))
    b = slice(int(x["starts"][1]), int(x["starts"][2]))  # the other request's rows are unharmed
    assert torch.equal(out[b], whole[b])
    assert attn.get_device_status() == attn.ATTN_OK


@pytest.mark.parametrize("new", [(1, 1, 1), (200, 1, 33)])
def test_repeats_and_streams_give_the_same_bits(new):
    w = BASE.replace(new=new, total=(1500, 700, 129))
    g, out = _check(w)
    for _ in range(3):
        again = torch.full_like(out, -7.0)
        _attend(w, g, again)
        assert torch.equal(again, out)
    s = torch.cuda.Stream()
    other = torch.full_like(out, -7.0)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _attend(w, g, other)
    s.synchronize()
    assert torch.equal(other, out)


@pytest.mark.parametrize("new", [(1, 1), (3, 2), (90, 30)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rows_of_very_different_size(new, dtype):
    """One head of one token 2^12 times the others: each row keeps its own accuracy."""
    w = BASE.replace(new=new, total=(300, 200), dtype=dtype, q_std=0.5)
    x = ref.make(w)
    x["q"][0, 1] *= 4096.0
    x["q"][-5, 2] *= 2.0 ** -9
    g = _gpu(x)
    out = torch.full(x["q"].shape, -7.0, dtype=x["q"].dtype, device="cuda")
    lse = torch.full(x["q"].shape[:2], -7.0, device="cuda")
    _attend(w, g, out, lse)
    _check_out(w, x, out, lse)


@pytest.mark.parametrize("new", [(2, 1), (80, 40)])
def test_a_row_that_is_not_finite_reaches_no_other(new):
    w = BASE.replace(new=new, total=(300, 200), Hq=8, Hkv=2)
    x = ref.make(w)
    whole = _attend(w, _gpu(x))
    x["q"][1, 2, 5] = float("nan")
    x["q"][1, 5, 100] = float("inf")
    got = _attend(w, _gpu(x))
    torch.cuda.synchronize()
    n = sum(new)
    assert got[1, 2].isnan().all() and got[1, 5].isnan().all()
    keep = torch.ones(n, 8, dtype=torch.bool, device="cuda")
    keep[1, 2] = keep[1, 5] = False
    assert torch.equal(got[:n][keep], whole[:n][keep])


def test_many_requests():
    rng = np.random.Generator(np.random.PCG64(4))
    total = tuple(int(t) for t in rng.integers(0, 40, 2500))
    new = tuple(min(t, int(n)) for t, n in zip(total, rng.integers(0, 3, 2500)))
    _check(Problem(new=new, total=total, Hq=2, Hkv=1, D=64, block=16))


def test_negative_totals_see_nothing():
    w = BASE.replace(new=(1, 2, 40), total=(-5, 100, -1))
    _check(w)


def test_calls_from_two_threads():
    """Each thread's calls on the default stream have a workspace of their own."""
    import threading
    w = [BASE.replace(new=(1,) * 8, total=tuple(range(900, 1700, 100)), seed=s) for s in (1, 2)]
    g = [_gpu(ref.make(v)) for v in w]
    want = [_attend(v, x).clone() for v, x in zip(w, g)]
    torch.cuda.synchronize()
    good = [0, 0]

    def work(i):
        for _ in range(200):
            good[i] += torch.equal(_attend(w[i], g[i])[:8], want[i][:8])

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert good == [200, 200]


def test_caller_workspace():
    w = BASE.replace(new=(1, 3), total=(3000, 500))
    g, out = _check(w)
    T, Hq, D = out.shape
    need = attn.attn_paged_workspace_bytes(T, 2, Hq, w.Hkv, D)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # nothing in it has to start at zero
    again = torch.full_like(out, -7.0)
    _attend(w, g, again, workspace=ws)
    assert torch.equal(again, out)
    with pytest.raises(attn.AttnError):
        _attend(w, g, again, workspace=ws[:need - 16])


def test_float8_and_uint8_caches_are_the_same():
    w = BASE
    g, out = _check(w)
    g["k_cache"], g["v_cache"] = (g[k].view(torch.float8_e4m3fn) for k in ("k_cache", "v_cache"))
    again = torch.full_like(out, -7.0)
    _attend(w, g, again)
    assert torch.equal(again, out)


# ------------------------------------------------------ the three together
class Server:
    """A batch of requests served with the library's calls, and the same in 64 bits."""

    def __init__(self, B=5, block=16, Hq=8, Hkv=2, D=64, dtype="bf16", N=120, width=40):
        self.rng = np.random.Generator(np.random.PCG64(8))
        self.B, self.block, self.N, self.T = B, block, N, 96
        self.w = Problem(new=(), total=(), Hq=Hq, Hkv=Hkv, D=D, block=block, dtype=dtype)
        self.dt = ref.TORCH[dtype]
        self.tables, self.free, self.count = np.full((B, width), -1, np.int32), np.arange(N, dtype=np.int32), N
        self.past = np.zeros(B, np.int32)
        self.c = [np.full((N, Hkv, block, D), 127, np.uint8) for _ in range(2)]
        self.s = [np.zeros((N, Hkv)) for _ in range(2)]
        d = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
        self.g = dict(tables=d(self.tables), free=d(self.free), count=d(np.array([N], np.int32)), k=d(self.c[0]),
                      v=d(self.c[1]), ks=torch.zeros((N, Hkv), device="cuda"), vs=torch.zeros((N, Hkv), device="cuda"),
                      past=torch.zeros(B, dtype=torch.int32, device="cuda"),
                      new=torch.zeros(B, dtype=torch.int32, device="cuda"),
                      fin=torch.zeros(B, dtype=torch.bool, device="cuda"),
                      qkv=torch.zeros((self.T, Hq + 2 * Hkv, D), dtype=self.dt, device="cuda"),
                      out=torch.zeros((self.T, Hq, D), dtype=self.dt, device="cuda"))

    def enqueue(self):
        g, w = self.g, self.w
        starts, totals, slots, result = attn.attn_cache_assign(
            g["past"], g["new"], g["tables"], g["free"], g["count"], block_size=self.block, num_tokens=self.T,
            finished=g["fin"])
        attn.attn_cache_append_fp8(g["qkv"][:, w.Hq:w.Hq + w.Hkv], g["qkv"][:, w.Hq + w.Hkv:], slots, g["k"], g["v"],
                                   g["ks"], g["vs"])
        attn.attn_fwd_paged_fp8(g["qkv"][:, :w.Hq], g["k"], g["v"], g["ks"], g["vs"], g["tables"], starts, totals,
                                out=g["out"])
        g["past"].copy_(totals)
        self.result = result

    def step(self, new, fin, go):
        w, g = self.w, self.g
        new, fin = np.array(new, np.int32), np.array(fin, bool)
        qkv = torch.from_numpy(self.rng.standard_normal(tuple(g["qkv"].shape))
                               * np.exp(self.rng.standard_normal((self.T, 1, 1)))).to(self.dt)
        g["qkv"].copy_(qkv)
        g["new"].copy_(torch.from_numpy(new))
        g["fin"].copy_(torch.from_numpy(fin))
        g["out"].fill_(-7.0)
        go()
        torch.cuda.synchronize()
        assert attn.get_device_status() == attn.ATTN_OK
        starts, totals, slots, result, self.count = ref.assign(self.past, new, fin, self.tables, self.free, self.count,
                                                               self.block, self.T)
        assert int(self.result) == result == 0
        assert np.array_equal(g["tables"].cpu().numpy(), self.tables) and int(g["count"]) == self.count
        for i, a in enumerate((w.Hq, w.Hq + w.Hkv)):
            ref.append(qkv[:, a:a + w.Hkv].double().numpy(), slots, self.c[i], self.s[i])
        self.past = totals
        x = dict(q=qkv[:, :w.Hq], k_cache=torch.from_numpy(self.c[0]), v_cache=torch.from_numpy(self.c[1]),
                 k_scales=torch.from_numpy(self.s[0]), v_scales=torch.from_numpy(self.s[1]),
                 tables=torch.from_numpy(self.tables), starts=torch.from_numpy(starts), totals=torch.from_numpy(totals))
        want, _, tol, _ = ref.attend(w, x)
        got = g["out"].double().cpu().numpy()
        none = np.isnan(want)
        assert (got[none] == -7.0).all()
        assert (np.abs(got - want)[~none] <= tol[~none]).all()


STEPS = [([30, 0, 41, 1, 0], [0, 0, 0, 0, 0]), ([1, 0, 1, 1, 0], [0, 0, 0, 0, 0]), ([1, 55, 1, 1, 9], [0, 0, 0, 0, 0]),
         ([1, 1, 20, 1, 1], [0, 0, 1, 0, 0]), ([4, 1, 1, 0, 3], [0, 1, 0, 1, 0]), ([1, 1, 1, 17, 1], [0, 0, 0, 0, 1])]


@pytest.mark.parametrize("kw", [dict(), dict(block=64, D=128, dtype="f16", Hq=8, Hkv=1, N=40, width=9)])
def test_steps_of_a_batch(kw):
    s = Server(**kw)
    for new, fin in STEPS:
        s.step(new, fin, s.enqueue)


def test_captured_steps_of_a_batch():
    """One graph of the three calls, replayed with other lengths and rows each time."""
    s = Server()
    s.step(*STEPS[0], s.enqueue)  # the first call on the device happens outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.enqueue()
    for new, fin in STEPS[1:]:
        s.step(new, fin, graph.replay)


# ------------------------------------------------------------ wide tables
@pytest.fixture
def wide(monkeypatch):
    """Tables for 2^21 keys a request: units of 16 and 256 rows instead of 8, whatever the lengths."""
    make = ref.make

    def widened(w):
        x = make(w)
        more = torch.full((len(w.new), 2 ** 21 // w.block), -3, dtype=torch.int32)
        x["tables"] = torch.cat([x["tables"], more], 1)
        return x
    monkeypatch.setattr(ref, "make", widened)


@pytest.mark.parametrize("feature", list(FEATURES))
@pytest.mark.parametrize("shape", list(SHAPES))
def test_wide_tables(shape, feature, wide):
    _check(Problem(**SHAPES[shape]).replace(**FEATURES[feature]))


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64), ("bf16", 64), ("f16", 128)])
@pytest.mark.parametrize("Hq,Hkv", [(9, 1), (12, 1), (16, 1), (17, 1), (32, 2), (40, 1)])
def test_wide_tables_heads(Hq, Hkv, dtype, D, wide):
    _check(BASE.replace(Hq=Hq, Hkv=Hkv, dtype=dtype, D=D, total=(1, 130, 300, 64)))


@pytest.mark.parametrize("new", [3, 60])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_wide_tables_extremes(new, dtype, wide):
    test_one_key_far_above_the_others(new, dtype)
    test_rows_of_very_different_size((new, 9), dtype)
    test_a_row_that_is_not_finite_reaches_no_other((new, 3))
    test_tables_that_name_no_block_are_reported((new, 3))
    test_growing_maximum()
    test_zero_scales()


@pytest.mark.parametrize("new", [(3, 4, 3), (200, 1, 33)])
def test_wide_tables_repeats_and_streams(new, wide):
    test_repeats_and_streams_give_the_same_bits(new)


# ------------------------------------------------- queries at their type's ends
def _extreme_queries(dtype, new):
    """Rows of the smallest and (float16) the largest magnitudes, zeros, and one that is not finite."""
    w = BASE.replace(new=new, total=(300, 250), dtype=dtype, Hq=8, Hkv=2)
    x = ref.make(w)
    n = sum(new)
    sign = torch.sign(x["q"].float())
    x["q"][0, 0] = (sign[0, 0] * 2.0 ** (-24 if dtype == "f16" else -110)).to(x["q"].dtype)
    x["q"][0, 1] = 0.0
    if dtype == "f16":
        x["q"][n - 1, 6] = (sign[n - 1, 6] * 65504.0).to(x["q"].dtype)
    x["q"][n - 1, 7, 3:] = 0.0
    bad = x["q"].clone()
    bad[1, 3, 9] = float("-inf")
    bad[1, 6, 0] = float("nan")
    return w, x, dict(x, q=bad)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new", [(2, 1), (3, 2), (150, 40)])
def test_queries_at_their_types_ends(new, dtype):
    w, x, odd = _extreme_queries(dtype, new)
    g = _gpu(x)
    out = torch.full(x["q"].shape, -7.0, dtype=x["q"].dtype, device="cuda")
    lse = torch.full(x["q"].shape[:2], -7.0, device="cuda")
    _attend(w, g, out, lse)
    _check_out(w, x, out, lse)
    got = torch.full_like(out, -7.0)
    _attend(w, _gpu(odd), got)
    assert got[1, 3].isnan().all() and got[1, 6].isnan().all()
    keep = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    keep[1, 3] = keep[1, 6] = False
    assert torch.equal(got[keep], out[keep])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new", [(2, 1), (3, 2), (150, 40)])
def test_wide_tables_queries_at_their_types_ends(new, dtype, wide):
    test_queries_at_their_types_ends(new, dtype)


# ------------------------------------------------ large caches, concurrent graphs
@pytest.mark.parametrize("new", [(1, 2, 1), (150, 1, 20)])
def test_blocks_past_four_gigabytes(new):
    """The same step over a small cache and over one whose blocks in use lie past 2^32 bytes: equal bits."""
    w = BASE.replace(new=new, total=(300, 200, 129), Hq=16, Hkv=8)
    x = ref.make(w)
    small = _gpu(x)
    N = x["k_cache"].shape[0]
    more = 2 ** 32 // (w.Hkv * w.block * w.D) + 5
    big = dict(small, tables=torch.where((small["tables"] >= 0) & (small["tables"] < N), small["tables"] + more, -1))
    for name in ("k_cache", "v_cache", "k_scales", "v_scales"):
        big[name] = torch.zeros((N + more, *small[name].shape[1:]), dtype=small[name].dtype, device="cuda")
        big[name][more:] = small[name]
    kv = [torch.randn(sum(new), w.Hkv, w.D, device="cuda").to(torch.bfloat16) for _ in range(2)]
    slots, tables = [], x["tables"].numpy()
    for b, n in enumerate(new):
        for pos in range(w.total[b] - n, w.total[b]):
            slots.append(int(tables[b, pos // w.block]) * w.block + pos % w.block)
    slots = torch.tensor(slots, device="cuda")
    outs = []
    for g, at in ((small, slots), (big, slots + more * w.block)):
        attn.attn_cache_append_fp8(*kv, at, g["k_cache"], g["v_cache"], g["k_scales"], g["v_scales"])
        out = torch.full(x["q"].shape, -7.0, dtype=x["q"].dtype, device="cuda")
        _attend(w, g, out)
        outs.append(out)
    torch.cuda.synchronize()
    assert attn.get_device_status() == attn.ATTN_OK
    assert torch.equal(outs[0], outs[1])
    for name in ("k_cache", "v_cache", "k_scales", "v_scales"):
        assert torch.equal(big[name][more:], small[name])


def test_two_graphs_replayed_at_once():
    """Two captured calls, each with the workspace its capture gave it, on two streams at the same time."""
    made = []
    for new, total, seed in (((1,) * 6, (900, 1700, 300, 2500, 40, 1100), 3), ((90, 200, 1), (1500, 700, 2000), 4)):
        w = BASE.replace(new=new, total=total, seed=seed)
        x = ref.make(w)
        g = _gpu(x)
        want = torch.full(x["q"].shape, -7.0, dtype=x["q"].dtype, device="cuda")
        _attend(w, g, want)
        out = torch.full_like(want, -7.0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _attend(w, g, out)
        made.append((graph, out, want, torch.cuda.Stream(), g))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, _, _, stream, _ in made:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, out, want, _, _ in made:
        assert torch.equal(out, want)
    assert attn.get_device_status() == attn.ATTN_OK
