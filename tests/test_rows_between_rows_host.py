"""Rows that lie between each other in one buffer: which calls attn_cache_read_fp4 and
attn_rope refuse (no GPU needed: the calls that pass this check are refused by a
later one, for blocks of 8 slots or a misaligned argument, before any CUDA call)."""
import numpy as np
import pytest

import tiled_online_softmax_02_gb300 as attn
from tiled_online_softmax_02_gb300 import build

A = [0x100000000 * (i + 1) for i in range(16)]  # never dereferenced
CLASH, PASSES = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return attn.load_library()


def read(lib, T, H, D, k, v, ks, vs):
    """ks, vs: (token stride, head stride) in elements of bf16."""
    return lib.attn_cache_read_fp4(A[3], A[4], A[5], A[6], None, None, A[2], k, v, T, H, D, *ks, *vs, 100, 8, attn.ATTN_BF16, None)


def rope(lib, **kw):
    a = dict(q=A[0], k=A[1], qo=A[2], ko=A[3], freq=A[4] + 4, pos=A[7], starts=None, totals=None, T=10, B=0, Hq=4, Hk=2,
             D=64, R=64, qst=256, kst=128, qost=256, kost=128, inter=0, inverse=0, scale=1.0, dtype=attn.ATTN_BF16)
    a.update(kw)
    return lib.attn_rope(*a.values(), None)


@pytest.mark.parametrize("T,H,D", [(7, 3, 64), (1, 3, 64), (7, 1, 128), (1, 1, 64)])
def test_k_and_v_side_by_side(lib, T, H, D):
    two = 2 * D
    for step, ks in ((D, (H * two, two)),            # [T, H, 2, D]
                     (H * D, (H * two, D)),          # [T, 2, H, D]
                     (T * H * D, (H * D, D)),        # [2, T, H, D]
                     (D, (two, T * two)),            # [H, T, 2, D]
                     (T * D, (D, T * two))):         # [H, 2, T, D]
        assert read(lib, T, H, D, A[0], A[0] + 2 * step, ks, ks) == PASSES, (step, ks)
        assert read(lib, T, H, D, A[0] + 2 * step, A[0], ks, ks) == PASSES, (step, ks)
        assert read(lib, T, H, D, A[0], A[0] + 2 * step - 16, ks, ks) == CLASH, (step, ks)
        assert read(lib, T, H, D, A[0], A[0], ks, ks) == CLASH


def test_all_that_meet_are_refused_and_no_others(lib):
    """Random strides and offsets against the rows' bytes one by one."""
    rng = np.random.Generator(np.random.PCG64(1))
    seen = {CLASH: 0, PASSES: 0}
    for _ in range(4000):
        T, H, D = int(rng.integers(1, 5)), int(rng.integers(1, 5)), int(rng.choice([64, 128]))
        inner = D + 8 * int(rng.integers(0, 40))
        heads_in = bool(rng.integers(0, 2))
        n = H if heads_in else T
        outer = (n - 1) * inner + D + 8 * int(rng.integers(0, 60))
        strides = (outer, inner) if heads_in else (inner, outer)
        step = 8 * int(rng.integers(-80, 400))
        pieces = lambda base: {(base + t * strides[0] + h * strides[1] + i * 8) for t in range(T) for h in range(H)  # noqa: E731
                               for i in range(D // 8)}  # offsets and strides are whole 8 elements
        want = CLASH if pieces(0) & pieces(step) else PASSES
        got = read(lib, T, H, D, A[0], A[0] + 2 * step, strides, strides)
        # beyond the last of its tokens (or heads) a set is taken to go on, so some calls of a few rows are refused for others'
        if want == PASSES and got == CLASH:
            long = {base + i * outer for i in range(-8, 9) for base in pieces(step)}
            assert pieces(0) & long
            continue
        assert got == want, (T, H, D, strides, step)
        seen[want] += 1
    assert min(seen.values()) > 500, seen


def test_a_single_token_in_place(lib):
    """The token stride of one token says nothing."""
    assert rope(lib, T=1, qo=A[0], qost=999, ko=A[1], kost=128) == PASSES
    assert rope(lib, T=1, qo=A[0] + 128, qost=999) == CLASH
    assert rope(lib, T=2, qo=A[0], qost=999) == CLASH
    assert rope(lib, qo=A[0], ko=A[1]) == PASSES
