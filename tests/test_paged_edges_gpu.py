"""The paged 8-bit KV cache at the ends of what its calls accept, on a GPU.
Attention is compared with 64 bits, within the kernels' own error bounds and
with nothing added for a hardware tanh."""
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


# Rows of a (request, kv head) and the table's width choose the kernel: 2^21 keys of width rule out units of 8 rows.
KINDS = {
    "rows4": dict(new=(1, 1), wide=False), "rows8": dict(new=(2, 2), wide=False), "rows16": dict(new=(4, 3), wide=True),
    "rows256": dict(new=(70, 9), wide=True),
}


def _problem(kind, **kw):
    """(problem, its tensors): four query heads a kv head, lengths that leave units cut between CTAs and a ragged last block."""
    w = Problem(new=KINDS[kind]["new"], total=(3001, 420), pad=0, **kw)
    x = ref.make(w)
    if KINDS[kind]["wide"]:
        x["tables"] = torch.cat([x["tables"], torch.full((2, 2 ** 21 // w.block), -3, dtype=torch.int32)], 1)
    return w, x


def _run(w, x):
    g = {k: v.cuda() for k, v in x.items()}
    out = torch.full(x["q"].shape, -7.0, dtype=x["q"].dtype, device="cuda")
    lse = torch.full(x["q"].shape[:2], -7.0, device="cuda")
    attn.attn_fwd_paged_fp8(g["q"], g["k_cache"], g["v_cache"], g["k_scales"], g["v_scales"], g["tables"], g["starts"],
                            g["totals"], causal=w.causal, local_window=w.window, scale=w.scale, softcap=w.softcap,
                            out=out, lse=lse)
    torch.cuda.synchronize()
    assert attn.get_device_status() == attn.ATTN_OK
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def _check(w, x, exact=False):
    """Every row against 64 bits.  With A = sum_j p_j |v_j|, p_j = exp(s_j - max s), l = sum_j p_j, u_j the V scale or
    2^-100 where that is larger:
      half a step of the output type on the result;
      weights of at least 11 bits: A 2^-11; below 2^-13 of the largest p_j u_j, which is what they are carried relative
      to, an absolute 2^-24 of it: 2^-24 max_j(p_j u_j) sum_j |v8_j| / l;
      scores off by at most e: 2 e A.  e has fp32's sums over the row, scale 2^-16 sum_d |q_d k_d|, Q's pieces, whose rest
      is at most 2^-17 of the row's largest element, scale 2^-17 max|q| sum_d |k_d|, and the score and log2 of the V
      scale as one fp32 number of up to 2^8, rounded three times: 2^-15.  Where `exact`, q and the key bytes are small
      whole numbers, so that pieces and sums are exact: 2^-21 |s| for the two scales in place of those two;
      a soft-cap c, whose derivative is at most 1, so that e of the score itself does not grow.  Few rows, c up to 512:
      1 - 2 / (e^2y + 1) has ex2's 2^-22 and the reciprocal's 2^-23, each at most doubled, so 2^-20 c.  Otherwise the
      GB300's tanh, 2^-16.6 of the value as measured: 2^-16 of the score.
    lse: e, and fp32's rounding of the result."""
    out, lse = _run(w, x)
    q = x["q"].double().numpy()
    starts, totals, tables = x["starts"].numpy(), x["totals"].numpy(), x["tables"].numpy()
    kc, vc = ref.E4M3[x["k_cache"].numpy()], ref.E4M3[x["v_cache"].numpy()]
    ks, vs = x["k_scales"].double().numpy(), x["v_scales"].double().numpy()
    T, Hq, D = q.shape
    Hkv, bs = kc.shape[1:3]
    scale = w.scale if w.scale is not None else D ** -0.5
    half = ref.HALF_STEP[w.dtype]
    few = sum(w.new) < 20  # the many-rows kernel has more
    for b, L in enumerate(totals):
        n = int(starts[b + 1] - starts[b])
        blk = tables[b, np.arange(L) // bs]
        k, v8, u = (kc[blk, :, np.arange(L) % bs] * ks[blk][..., None], vc[blk, :, np.arange(L) % bs], vs[blk])
        for t in range(starts[b], starts[b] + n):
            hi = int(L) - n + t - int(starts[b]) + 1
            for h in range(Hq):
                g = h * Hkv // Hq
                kk, vv8, uu = k[:hi, g], v8[:hi, g], u[:hi, g]
                vv = vv8 * uu[:, None]
                s = scale * (kk @ q[t, h])
                e = 2.0 ** -15 + (2.0 ** -21 * np.abs(s).max() if exact else
                                  abs(scale) * (2.0 ** -16 * (np.abs(kk) @ np.abs(q[t, h])).max()
                                                + 2.0 ** -17 * np.abs(q[t, h]).max() * np.abs(kk).sum(1).max()))
                if w.softcap > 0:
                    s = w.softcap * np.tanh(s / w.softcap)
                    e += 2.0 ** -20 * w.softcap if w.softcap <= 512 and few else 2.0 ** -16 * np.abs(s).max()
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
                want, want_lse = p @ vv / l, m + np.log(l)
                tol = (half * np.abs(want) + (2.0 ** -11 + 2 * e) * (p @ np.abs(vv)) / l
                       + 2.0 ** -24 * (p * np.maximum(uu, 2.0 ** -100)).max() * np.abs(vv8).sum(0) / l)
                err = np.abs(out[t, h] - want)
                assert (err <= tol).all(), f"row {t} head {h}: worst {np.nanmax(err / np.maximum(tol, 1e-300)):.3g} tolerances"
                assert abs(lse[t, h] - want_lse) <= e + 2.0 ** -21 * (1 + abs(want_lse) + abs(m)), \
                    f"lse of row {t} head {h}: {lse[t, h]} instead of {want_lse}"


# ---------------------------------------------------------------- V scales
def _set_v(w, x, name):
    """Scales in the order of each request's blocks, and zero bytes where the block is one of zeros."""
    tables, scales, cache = x["tables"].numpy(), x["v_scales"].numpy(), x["v_cache"].numpy()
    for b, total in enumerate(w.total):
        n = -(-total // w.block)
        for i, blk in enumerate(tables[b, :n]):
            zero = False
            if name == "zeros_next_to_huge":  # a block of zeros as the append writes it
                zero, s = i % 3 == 1, 2.0 ** 40
            elif name == "zeros_first":
                zero, s = i < 2, 2.0 ** 36
            elif name == "all_zeros":
                zero, s = True, 0.0
            elif name == "no_scale":
                s = 0.0
            elif name == "some_no_scale":
                s = 0.0 if i % 2 else 1.0
            elif name == "tiny":
                s = 1e-35 * (1 + i / n)
            elif name == "huge":
                s = 2.0 ** 105
            elif name == "rising":
                s = 2.0 ** (-100 + 190 * i // n)
            else:  # falling
                s = 2.0 ** (90 - 190 * i // n)
            if zero:
                s = 2.0 ** -100
                cache[blk][(cache[blk] & 127) != 127] = 0  # slots of no token stay NaN
            scales[blk] = s


V_SCALES = ["zeros_next_to_huge", "zeros_first", "all_zeros", "no_scale", "some_no_scale", "tiny", "huge", "rising",
            "falling"]


@pytest.mark.parametrize("name", V_SCALES)
@pytest.mark.parametrize("kind", list(KINDS))
def test_v_scales_of_any_size(kind, name):
    """Blocks whose V is 2^100 times smaller or larger than their neighbours' weigh by their scores alone."""
    w, x = _problem(kind, Hq=4, Hkv=1) if kind != "rows8" else _problem(kind, Hq=8, Hkv=2, D=64, block=32)
    _set_v(w, x, name)
    _check(w, x)


@pytest.mark.parametrize("name", ["all_zeros", "no_scale"])
@pytest.mark.parametrize("kind", ["rows4", "rows256"])
def test_no_values_for_half_queries(kind, name):
    w, x = _problem(kind, Hq=4, Hkv=1, dtype="f16", D=64)
    _set_v(w, x, name)
    _check(w, x)


# ---------------------------------------------------------------- soft-caps
def _whole_numbers(w, x, spread):
    """The problem with q and the keys' bytes as whole numbers, scores of standard deviation `spread`."""
    rng = np.random.Generator(np.random.PCG64(12))
    x["q"] = torch.from_numpy(rng.integers(-31, 32, tuple(x["q"].shape)).astype(np.float32)).to(x["q"].dtype)
    k = x["k_cache"].numpy()
    k[:] = np.where((k & 127) == 127, k, ref.encode(rng.integers(-15, 16, k.shape).astype(np.float64)))
    x["k_scales"].fill_(2.0 ** -4)
    raw = np.sqrt(w.D * (31 * 32 / 3) * (15 * 16 / 3))
    return w.replace(scale=float(np.float32(spread / raw * 2 ** 4))), x


@pytest.mark.parametrize("cap", [2.0, 20.0, 50.0, 1000.0])
@pytest.mark.parametrize("dtype,D", [("f16", 128), ("bf16", 64)])
@pytest.mark.parametrize("kind", list(KINDS))
def test_scores_near_the_cap(kind, dtype, D, cap):
    """Scores up to several times the cap."""
    w, x = _problem(kind, Hq=8, Hkv=2, dtype=dtype, D=D, softcap=cap)
    _check(*_whole_numbers(w, x, 0.8 * cap), exact=True)


@pytest.mark.parametrize("cap", [3e3, 3e4, 1e6, 1e8, 1e25, 1e31, 3e38])
@pytest.mark.parametrize("kind", list(KINDS))
def test_caps_far_above_the_scores(kind, cap):
    """A cap that changes nothing leaves the scores as they are, small ones too."""
    w, x = _problem(kind, Hq=8, Hkv=2, dtype="f16", softcap=cap)
    _check(*_whole_numbers(w, x, 4.0), exact=True)


@pytest.mark.parametrize("cap", [1e-3, 1e-20, 1e-42])
@pytest.mark.parametrize("kind", list(KINDS))
def test_caps_far_below_the_scores(kind, cap):
    """Nothing is left of the scores but, at most, their signs; keys of scale 0 score 0."""
    w, x = _problem(kind, Hq=8, Hkv=2, dtype="f16", softcap=cap)
    w, x = _whole_numbers(w, x, 4.0)
    x["k_scales"][::3] = 0.0
    x["k_scales"][1::3] = 2.0 ** 30
    _check(w, x, exact=True)


# ------------------------------------------------------------------- append
def _append(slots, N, Hkv=2, D=64, block=16, seed=3):
    rng = np.random.Generator(np.random.PCG64(seed))
    T = len(slots)
    kv = [torch.from_numpy((rng.standard_normal((T, Hkv, D), np.float32)
                            * np.exp2(rng.integers(-3, 4, (T, 1, 1))).astype(np.float32))).to(torch.bfloat16)
          for _ in range(2)]
    caches = [rng.integers(0, 127, (N, Hkv, block, D), dtype=np.uint8) for _ in range(2)]
    scales = [(2.0 ** rng.integers(-9, 2, (N, Hkv))).astype(np.float32) for _ in range(2)]
    g = [torch.from_numpy(a).cuda() for a in (*caches, *scales)]
    attn.attn_cache_append_fp8(kv[0].cuda(), kv[1].cuda(), torch.from_numpy(slots).cuda(), *g)
    torch.cuda.synchronize()
    live = np.flatnonzero((slots >= 0) & (slots < N * block))
    for i in range(2):
        s = scales[i].astype(np.float64)
        # the reference walks runs of adjacent tokens: those between them that have no slot stay
        ref.append(kv[i].double().numpy(), slots, caches[i], s)
        assert np.array_equal(g[2 + i].double().cpu().numpy(), s)
        got = g[i].cpu().numpy()
        assert np.array_equal(np.where(got == 128, 0, got), np.where(caches[i] == 128, 0, caches[i]))
    assert len(live) > 0


@pytest.mark.parametrize("T", [900, 5000, 70001])
@pytest.mark.parametrize("at", ["first", "last", "spread", "ends"])
def test_append_over_long_gaps(T, at):
    """A few tokens of two blocks among many that have no slot: one block's runs lie far apart and are taken in order."""
    n = 11
    where = {"first": np.arange(n), "last": T - n + np.arange(n),
             "spread": np.sort(np.random.default_rng(T).choice(T, n, replace=False)),
             "ends": np.concatenate([np.arange(5), T - 6 + np.arange(6)])}[at]
    slots = np.full(T, -1, np.int64)
    slots[where] = np.concatenate([16 * 3 + 5 + np.arange(6), 16 * 1 + 9 + np.arange(5)])
    slots[where[3]] = 2 ** 40  # a slot of no block is passed over too
    _append(slots, 5)


@pytest.mark.parametrize("seed", range(40))
def test_append_random_gaps(seed):
    """Runs of any length and order, and gaps between and inside them of every length around what a CTA looks at."""
    rng = np.random.default_rng(seed)
    block, gaps = int(rng.choice([16, 32, 64, 128])), [0, 0, 0, 1, 3, 28, 31, 33, 40, 64, 67, 129, 193, 300, 1500]
    slots = [-1] * int(rng.choice(gaps))
    for b in rng.permutation(30)[:int(rng.integers(1, 30))]:
        for _ in range(int(rng.integers(1, 4))):
            a = int(rng.integers(0, block))
            for s in range(a, int(rng.integers(a, block)) + 1):
                slots.append(b * block + s)
                if rng.random() < 0.08:
                    slots += [-1] * int(rng.choice(gaps[3:]))
            slots += [-1] * int(rng.choice(gaps))
    _append(np.array(slots, np.int64), 30, Hkv=1, block=block, seed=seed)


def test_append_many_short_runs():
    """1040 requests, a token or two each: just past the size where a CTA takes more tokens."""
    rng = np.random.default_rng(2)
    slots = []
    for b in rng.permutation(700):
        off = int(rng.integers(0, 15))
        slots += [b * 16 + off] + ([b * 16 + off + 1] if rng.random() < 0.5 else [])
    slots = np.array(slots, np.int64)
    assert len(slots) > 1024
    _append(slots, 700)


def test_append_does_not_wait_for_padding():
    """A decode step's 64 tokens in a slot map padded to 65536.  Passing over the tail 32 entries at a time, one load after
    the other, took 576 us; with 1024 on their way it is 105 us."""
    T, n, Hkv, D = 65536, 64, 8, 128
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    slots[:n] = torch.arange(n, device="cuda") * 64 + 17
    kv = [torch.randn((T, Hkv, D), device="cuda").to(torch.bfloat16) for _ in range(2)]
    c = [torch.zeros((n, Hkv, 64, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    s = [torch.ones((n, Hkv), device="cuda") for _ in range(2)]
    times = []
    for _ in range(8):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(10):
            attn.attn_cache_append_fp8(*kv, slots, *c, *s)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 100)
    assert min(times) < 300.0, times


# ------------------------------------------------------------------- assign
def _assign(past, new, tables, free, count, block, T, finished=None, outputs=()):
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    g = [d(np.array(past, np.int32)), d(np.array(new, np.int32)), d(tables), d(free), d(np.array([count], np.int32))]
    made = attn.attn_cache_assign(*g, block_size=block, num_tokens=T,
                                  finished=None if finished is None else d(finished), **dict(outputs))
    torch.cuda.synchronize()
    return made, [t.cpu().numpy() for t in (*made, g[2], g[3], g[4])]


@pytest.mark.parametrize("entry", [-1, -2 ** 31, 20, 2 ** 31 - 1])
@pytest.mark.parametrize("B", [3, 200])
@pytest.mark.parametrize("which", ["top", "deepest"])
def test_assign_refuses_a_free_list_entry_it_would_take(B, which, entry):
    """A stack entry that names no block is not handed out: the step is refused, nothing changes."""
    N = 20 + B
    entry = N if entry == 20 else entry
    tables = np.full((B, 3), -1, np.int32)
    tables[:, 0] = np.arange(B)
    free = np.full(N, -1, np.int32)
    free[:20] = B + np.arange(20)
    past, new = np.full(B, 16), np.zeros(B, np.int64)
    new[[0, B - 1]] = 17, 3  # two blocks and one: entries 19, 18, 17
    bad = free.copy()
    bad[19 if which == "top" else 17] = entry
    _, got = _assign(past, new, tables, bad, 20, 16, 40)
    assert got[3][0] == 5
    assert np.array_equal(got[4], tables) and np.array_equal(got[5], bad) and got[6][0] == 20
    assert (got[0] == 0).all() and np.array_equal(got[1], past) and (got[2] == -1).all()
    # an entry below those it takes is another step's
    bad = free.copy()
    bad[16] = entry
    _, got = _assign(past, new, tables, bad, 20, 16, 40)
    assert got[3][0] == 0 and got[4][0, 1:].tolist() == [B + 19, B + 18] and got[4][B - 1, 1] == B + 17


@pytest.mark.parametrize("B,each", [(1, 2000), (200, 60)])
@pytest.mark.parametrize("where", [0, 700, -1])
def test_assign_looks_at_all_of_a_long_take(B, each, where):
    """A step that takes thousands of blocks: a bad entry anywhere among them refuses it, one below them does not."""
    take = B * each
    N = take + 5
    tables = np.full((B, each), -1, np.int32)
    free = np.random.default_rng(B).permutation(N).astype(np.int32)
    past, new = np.full(B, 16 * each - 1), np.ones(B, np.int64)
    at = N - 1 - (where % take)
    bad = free.copy()
    bad[at] = -3
    _, got = _assign(past, new, tables, bad, N, 16, B)
    assert got[3][0] == 5 and np.array_equal(got[4], tables) and np.array_equal(got[5], bad) and got[6][0] == N
    bad = free.copy()
    bad[4] = N
    _, got = _assign(past, new, tables, bad, N, 16, B)
    assert got[3][0] == 0 and got[6][0] == 5 and np.array_equal(got[4].reshape(-1), free[:4:-1])


def test_assign_takes_returned_blocks_before_a_bad_entry():
    """Blocks given back by a finished row lie on top of the stack: an entry under them that is not taken is not looked at,
    one that is taken refuses the step and leaves the finished row its blocks."""
    tables = np.array([[0, 1, -1], [2, -1, -1]], np.int32)
    free = np.array([3, 99, -1, -1, -1, -1], np.int32)
    fin = np.array([True, False])
    _, got = _assign([32, 16], [5, 1], tables, free, 2, 16, 8, fin)
    assert got[3][0] == 0 and got[4].tolist() == [[1, -1, -1], [2, 0, -1]] and got[6][0] == 2
    _, got = _assign([32, 16], [5, 20], tables, free, 2, 16, 40, fin)
    assert got[3][0] == 5 and got[4].tolist() == tables.tolist() and got[5].tolist() == free.tolist() and got[6][0] == 2


@pytest.mark.parametrize("B", [2, 300])
def test_assign_resets_finished_rows_without_blocks(B):
    """A finished row's entries become -1, whichever negative numbers they were, though it gives no block back."""
    tables = np.full((B, 4), -1, np.int32)
    tables[:, 0], tables[:, 3] = -5, -2 ** 31
    free = np.arange(B, dtype=np.int32)
    fin = np.arange(B) % 2 == 1
    _, got = _assign(np.full(B, 9), np.arange(B) < 2, tables, free, B, 16, 2, fin)
    want = tables.copy()
    want[fin] = -1
    taken = np.flatnonzero(~fin | (np.arange(B) < 2))  # every row that goes on lacks its block, so does the one that begins
    want[taken, 0] = B - 1 - np.arange(len(taken))
    assert got[3][0] == 0 and np.array_equal(got[4], want) and got[6][0] == B - len(taken)
    _, got = _assign(np.full(B, 9), np.zeros(B), tables, free, B, 16, 0, np.ones(B, bool))
    assert got[3][0] == 0 and (got[4] == -1).all() and got[6][0] == B and np.array_equal(got[5], free)


def test_assign_into_the_callers_tensors():
    """q_starts, total_lengths, slot_map and result given by the caller are what the call writes and returns."""
    rng = np.random.Generator(np.random.PCG64(9))
    past, new = rng.integers(0, 200, 50).astype(np.int32), rng.integers(0, 40, 50).astype(np.int32)
    fin = rng.random(50) < 0.3
    tables = np.full((50, 20), -1, np.int32)
    free = rng.permutation(900).astype(np.int32)
    at = 900
    for b in range(50):
        for i in range(-(-int(past[b]) // 16)):
            at -= 1
            tables[b, i] = free[at]
    T = int(new.sum()) + 9
    mine = dict(q_starts=torch.full((51,), 77, dtype=torch.int32, device="cuda"),
                total_lengths=torch.full((50,), 77, dtype=torch.int32, device="cuda"),
                slot_map=torch.full((T,), 77, dtype=torch.int64, device="cuda"),
                result=torch.full((1,), 77, dtype=torch.int32, device="cuda"))
    made, got = _assign(past, new, tables, free, at, 16, T, fin, mine)
    for a, b in zip(made, mine.values()):
        assert a.data_ptr() == b.data_ptr()
    starts, totals, slots, result, n = ref.assign(past, new, fin, tables, free, at, 16, T)
    for a, b in zip(got, (starts, totals, slots, np.array([result]), tables, free, np.array([n]))):
        assert np.array_equal(a, b)
    for name, wrong in (("q_starts", 50), ("total_lengths", 51), ("slot_map", T - 1), ("result", 2)):
        with pytest.raises(ValueError, match=name):
            _assign(past, new, tables, free, at, 16, T, fin,
                    {name: torch.empty(wrong, dtype=mine[name].dtype, device="cuda")})
