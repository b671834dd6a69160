"""Host-side tests of the paged 8-bit KV cache (no GPU needed): every invalid
request is rejected with its documented status before any CUDA call, the
binding's checks, and the plain reference against hand-worked values."""
import math

import numpy as np
import pytest
import torch

import paged_reference as ref
import tiled_online_softmax_02_gb300 as attn
from tiled_online_softmax_02_gb300 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return attn.load_library()


# fake, aligned, non-overlapping device addresses: validation never dereferences them
A = [0x100000000 * (i + 1) for i in range(14)]


def assign(lib, **kw):
    a = dict(past=A[0], new=A[1], fin=None, tables=A[2], free=A[3], count=A[4], starts=A[5], totals=A[6], slots=A[7],
             result=A[8], B=4, width=8, block=64, N=100, T=4)
    a.update(kw)
    return lib.attn_cache_assign(*a.values(), None)


def append(lib, **kw):
    a = dict(k=A[0], v=A[1], slots=A[2], kc=A[3], vc=A[4], ks=A[5], vs=A[6], T=10, Hkv=2, D=64, kst=128, vst=128,
             N=100, block=64, dtype=attn.ATTN_BF16)
    a.update(kw)
    return lib.attn_cache_append_fp8(*a.values(), None)


def attend(lib, **kw):
    a = dict(q=A[0], kc=A[1], vc=A[2], ks=A[3], vs=A[4], tables=A[5], starts=A[6], totals=A[7], out=A[8], lse=None,
             T=10, B=3, Hq=4, Hkv=2, D=64, qst=256, N=100, block=64, width=8, causal=1, window=0, scale=0.1, softcap=0.0,
             dtype=attn.ATTN_BF16, ws=A[9], ws_bytes=1 << 31)
    a.update(kw)
    return lib.attn_fwd_paged_fp8(*a.values(), None)


CASES = [
    (assign, attn.ATTN_ERR_INVALID_ARG, [
        dict(B=-1), dict(width=-1), dict(N=-1), dict(T=-1), dict(block=0), dict(past=None), dict(new=None),
        dict(tables=None), dict(free=None), dict(count=None), dict(starts=None), dict(totals=None), dict(slots=None),
        dict(result=None), dict(totals=A[0]), dict(starts=A[2] + 64), dict(slots=A[3]), dict(fin=A[6])]),
    (assign, attn.ATTN_ERR_UNSUPPORTED, [
        dict(block=48), dict(block=256), dict(B=8193), dict(past=A[0] + 2), dict(slots=A[7] + 4), dict(count=A[4] + 1)]),
    (append, attn.ATTN_ERR_INVALID_ARG, [
        dict(dtype=3), dict(T=-1), dict(Hkv=0), dict(D=0), dict(N=-1), dict(block=0), dict(kst=127), dict(vst=0),
        dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vs=None), dict(vc=A[3] + 64),
        dict(ks=A[3]), dict(k=A[3]), dict(vs=A[2]), dict(N=2 ** 30, Hkv=4)]),
    (append, attn.ATTN_ERR_UNSUPPORTED, [
        dict(block=8), dict(D=96, kst=192, vst=192), dict(D=256, kst=512, vst=512), dict(k=A[0] + 8), dict(kst=129),
        dict(vc=A[4] + 4), dict(slots=A[2] + 4), dict(ks=A[5] + 2)]),
    (attend, attn.ATTN_ERR_INVALID_ARG, [
        dict(dtype=5), dict(T=-1), dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(D=0), dict(N=-1),
        dict(block=0), dict(width=-1), dict(causal=2), dict(scale=math.nan), dict(softcap=math.inf), dict(qst=255),
        dict(q=None), dict(kc=None), dict(vs=None), dict(tables=None), dict(starts=None), dict(totals=None),
        dict(out=None), dict(out=A[0]), dict(out=A[1] + 16), dict(lse=A[8]), dict(lse=A[6]), dict(width=2 ** 30),
        dict(T=2 ** 30), dict(Hq=65536, Hkv=65536, qst=65536 * 64)]),  # the last: caches of 27 GB overlap here
    (attend, attn.ATTN_ERR_UNSUPPORTED, [
        dict(dtype=attn.ATTN_F32), dict(D=96, qst=384), dict(D=256, qst=1024), dict(block=24), dict(B=8193), dict(Hq=65536, Hkv=1, qst=65536 * 64),
        dict(q=A[0] + 8), dict(qst=257), dict(out=A[8] + 2), dict(kc=A[1] + 8), dict(lse=A[10] + 1),
        dict(tables=A[5] + 2)]),
]


@pytest.mark.parametrize("call,status,kw", [(c, s, kw) for c, s, many in CASES for kw in many],
                         ids=lambda v: getattr(v, "__name__", str(v))[:40])
def test_refusals(lib, call, status, kw):
    assert call(lib, **kw) == status


def test_empty_problems_touch_nothing(lib):
    assert append(lib, T=0, k=None, v=None, slots=None) == attn.ATTN_OK
    assert append(lib, N=0) == attn.ATTN_OK
    assert attend(lib, T=0, q=None, out=None) == attn.ATTN_OK
    assert attend(lib, B=0, tables=None, starts=None, totals=None) == attn.ATTN_OK


@pytest.mark.parametrize("sizes", [(0, 4, 8, 2, 128), (5, 0, 8, 2, 128), (-1, 4, 8, 2, 128), (5, 4, 0, 2, 128),
                                   (5, 4, 1, 2, 128), (5, 4, 8, 0, 128), (5, 4, 8, 2, 0), (5, 4, 8, 2, -64)])
def test_sizes_of_no_call_need_no_workspace(lib, sizes):
    assert attn.attn_paged_workspace_bytes(*sizes) == 0
    assert attn.attn_paged_workspace_bytes(5, 4, 8, 2, 128) > 0


def test_binding_rejects_bad_tensors():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):  # CPU tensors
        attn.attn_cache_assign(i32(2), i32(2), i32(2, 4), i32(8), i32(1), block_size=16, num_tokens=2)
    c, s = torch.zeros((4, 2, 16, 64), dtype=torch.uint8), torch.zeros((4, 2))
    x = torch.zeros((3, 2, 64))
    with pytest.raises(ValueError):
        attn.attn_cache_append_fp8(x, x, torch.zeros(3, dtype=torch.int64), c, c.clone(), s, s.clone())
    with pytest.raises(ValueError):
        attn.attn_fwd_paged_fp8(torch.zeros((3, 4, 64), dtype=torch.float16), c, c, s, s, i32(1, 2), i32(2), i32(1))


# ------------------------------------------------ the reference itself
def test_reference_encodes_by_hand():
    x = np.array([0.0, 1.0, 1.0625, 1.1875, 448.0, 464.0, 1e9, -3.3, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -11, np.inf])
    want = [0.0, 1.0, 1.0, 1.25, 448.0, 448.0, 448.0, -3.25, 2.0 ** -9, 0.0, 2.0 ** -9, 448.0]
    assert ref.E4M3[ref.encode(x)].tolist() == want
    assert (ref.encode(np.array([np.nan]))[0] & 127) == 127
    # every value encodes to itself
    b = np.array([i for i in range(256) if (i & 127) != 127], np.uint8)
    assert np.array_equal(ref.encode(ref.E4M3[b]), b)


def test_reference_matches_torch_on_random_values():
    x = np.random.default_rng(1).standard_normal(20000) * 100
    x = x[np.abs(x) < 448].astype(np.float32)
    mine = ref.E4M3[ref.encode(x.astype(np.float64))]
    assert np.array_equal(mine, torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())


def test_reference_scales():
    assert ref.scale_for(448.0) == 1.0 and ref.scale_for(448.1) == 2.0 and ref.scale_for(224.0) == 0.5
    assert ref.scale_for(0.0) == 2.0 ** -100


def test_reference_attention_by_hand():
    """Two keys scoring equally: the mean of their V rows; a third one masked."""
    w = ref.Problem(new=(1,), total=(2,), Hq=1, Hkv=1, D=64, block=16, dtype="f16", pad=0)
    x = ref.make(w)
    x["q"].zero_()
    out, lse, _, _ = ref.attend(w, x)
    blk = int(x["tables"][0, 0])
    v = ref.E4M3[x["v_cache"][blk, 0, :2].numpy()] * float(x["v_scales"][blk, 0])
    assert np.allclose(out[0, 0], v.mean(0)) and np.isclose(lse[0, 0], math.log(2.0))
