"""Host-side tests of the paged 4-bit KV cache and of rotary positions (no GPU
needed): every invalid request is rejected with its documented status before any
CUDA call, the binding's checks, the frequencies, and the plain reference
against hand-worked values."""
import math

import numpy as np
import pytest
import torch

import paged4_reference as ref
import tiled_online_softmax_02_gb300 as attn
from tiled_online_softmax_02_gb300 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return attn.load_library()


# fake, aligned, non-overlapping device addresses: validation never dereferences them
A = [0x100000000 * (i + 1) for i in range(16)]


def append(lib, **kw):
    a = dict(k=A[0], v=A[1], slots=A[2], kc=A[3], vc=A[4], ks=A[5], vs=A[6], kh=None, vh=None, T=10, Hkv=2, D=64,
             kst=128, vst=128, N=100, block=64, dtype=attn.ATTN_BF16)
    a.update(kw)
    return lib.attn_cache_append_fp4(*a.values(), None)


def read(lib, **kw):
    a = dict(kc=A[3], vc=A[4], ks=A[5], vs=A[6], kh=None, vh=None, slots=A[2], k=A[0], v=A[1], T=10, Hkv=2, D=64,
             kst=128, khs=64, vst=128, vhs=64, N=100, block=64, dtype=attn.ATTN_BF16)
    a.update(kw)
    return lib.attn_cache_read_fp4(*a.values(), None)


def attend(lib, **kw):
    a = dict(q=A[0], kc=A[1], vc=A[2], ks=A[3], vs=A[4], kh=None, vh=None, tables=A[5], starts=A[6], totals=A[7],
             out=A[8], lse=None, T=10, B=3, Hq=4, Hkv=2, D=64, qst=256, N=100, block=64, width=8, causal=1, window=0,
             scale=0.1, softcap=0.0, dtype=attn.ATTN_BF16, ws=A[9], ws_bytes=1 << 31)
    a.update(kw)
    return lib.attn_fwd_paged_fp4(*a.values(), None)


def rope(lib, **kw):
    a = dict(q=A[0], k=A[1], qo=A[2], ko=A[3], freq=A[4], pos=None, starts=A[5], totals=A[6], T=10, B=3, Hq=4, Hk=2,
             D=64, R=64, qst=256, kst=128, qost=256, kost=128, inter=0, inverse=0, scale=1.0, dtype=attn.ATTN_BF16)
    a.update(kw)
    return lib.attn_rope(*a.values(), None)


CASES = [
    (append, attn.ATTN_ERR_INVALID_ARG, [
        dict(dtype=3), dict(T=-1), dict(Hkv=0), dict(D=0), dict(N=-1), dict(block=0), dict(kst=127), dict(vst=0),
        dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vs=None), dict(vc=A[3] + 64),
        dict(ks=A[3]), dict(k=A[3]), dict(vs=A[2]), dict(kh=A[5] + 16), dict(N=2 ** 30, Hkv=4)]),
    (append, attn.ATTN_ERR_UNSUPPORTED, [
        dict(block=8), dict(D=96, kst=192, vst=192), dict(D=256, kst=512, vst=512), dict(k=A[0] + 8), dict(kst=129),
        dict(vc=A[4] + 4), dict(slots=A[2] + 4), dict(ks=A[5] + 8), dict(kh=A[9] + 2)]),
    (read, attn.ATTN_ERR_INVALID_ARG, [
        dict(dtype=3), dict(T=-1), dict(Hkv=0), dict(D=0), dict(N=-1), dict(block=0), dict(kst=100), dict(khs=63),
        dict(vst=0), dict(vhs=-64), dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vs=None),
        dict(v=A[0] + 128), dict(k=A[3]), dict(k=A[2] + 16), dict(v=A[5] + 64), dict(khs=2 ** 60)]),
    (read, attn.ATTN_ERR_UNSUPPORTED, [
        dict(block=8), dict(D=96, kst=192, vst=192, khs=96, vhs=96), dict(k=A[0] + 8), dict(kst=132), dict(khs=68, kst=136),
        dict(vc=A[4] + 4), dict(slots=A[2] + 4), dict(ks=A[5] + 8), dict(vh=A[9] + 1)]),
    (attend, attn.ATTN_ERR_INVALID_ARG, [
        dict(dtype=5), dict(T=-1), dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(D=0), dict(N=-1),
        dict(block=0), dict(width=-1), dict(causal=2), dict(scale=math.nan), dict(softcap=math.inf), dict(qst=255),
        dict(q=None), dict(kc=None), dict(vs=None), dict(tables=None), dict(starts=None), dict(totals=None),
        dict(out=None), dict(out=A[0]), dict(out=A[1] + 16), dict(lse=A[8]), dict(lse=A[6]), dict(width=2 ** 30),
        dict(T=2 ** 30), dict(ws=None), dict(ws_bytes=64), dict(ws=A[3]), dict(N=0), dict(kh=A[8])]),
    (attend, attn.ATTN_ERR_UNSUPPORTED, [
        dict(dtype=attn.ATTN_F32), dict(D=96, qst=384), dict(D=256, qst=1024), dict(block=24), dict(B=8193),
        dict(Hq=65536, Hkv=1, qst=65536 * 64), dict(q=A[0] + 8), dict(qst=257), dict(out=A[8] + 2), dict(kc=A[1] + 8),
        dict(ks=A[3] + 8), dict(lse=A[10] + 1), dict(tables=A[5] + 2), dict(vh=A[10] + 2), dict(ws=A[9] + 8)]),
    (rope, attn.ATTN_ERR_INVALID_ARG, [
        dict(dtype=3), dict(T=-1), dict(B=-1), dict(Hq=0), dict(Hk=-1), dict(D=0), dict(R=63), dict(R=66), dict(R=-2),
        dict(inter=2), dict(inverse=-1), dict(scale=math.inf), dict(qst=255), dict(kost=127), dict(q=None),
        dict(qo=None), dict(k=None), dict(ko=None), dict(freq=None), dict(starts=None), dict(totals=None),
        dict(pos=A[7]), dict(qo=A[0] + 512), dict(qo=A[0], qost=512), dict(ko=A[0]), dict(qo=A[1]), dict(ko=A[2]),
        dict(qo=A[4]), dict(ko=A[6]),
        # slices of one buffer that do not fit between each other
        dict(q=A[0], k=A[0] + 500, qo=A[0], qst=400, kst=400, qost=400)]),
    (rope, attn.ATTN_ERR_UNSUPPORTED, [
        dict(q=A[0] + 1), dict(ko=A[3] + 1), dict(freq=A[4] + 4), dict(starts=A[5] + 2), dict(Hq=65535, qst=65535 * 64, qost=65535 * 64)]),
]


@pytest.mark.parametrize("call,status,kw", [(c, s, kw) for c, s, many in CASES for kw in many],
                         ids=lambda v: getattr(v, "__name__", str(v))[:40])
def test_refusals(lib, call, status, kw):
    assert call(lib, **kw) == status


def test_empty_problems_touch_nothing(lib):
    assert append(lib, T=0, k=None, v=None, slots=None) == attn.ATTN_OK
    assert append(lib, N=0) == attn.ATTN_OK
    assert read(lib, T=0, k=None, v=None, slots=None) == attn.ATTN_OK
    assert attend(lib, T=0, q=None, out=None) == attn.ATTN_OK
    assert attend(lib, B=0, tables=None, starts=None, totals=None) == attn.ATTN_OK
    assert rope(lib, T=0, q=None, qo=None) == attn.ATTN_OK
    assert rope(lib, B=0, starts=None, totals=None) == attn.ATTN_OK
    assert rope(lib, R=0, freq=None, qo=A[0], ko=A[1]) == attn.ATTN_OK  # in place, nothing turns


@pytest.mark.parametrize("sizes", [(0, 4, 8, 2, 128), (5, 0, 8, 2, 128), (-1, 4, 8, 2, 128), (5, 4, 0, 2, 128),
                                   (5, 4, 1, 2, 128), (5, 4, 8, 0, 128), (5, 4, 8, 2, 0), (5, 4, 8, 2, -64)])
def test_sizes_of_no_call_need_no_workspace(lib, sizes):
    assert attn.attn_paged_fp4_workspace_bytes(*sizes) == 0
    assert attn.attn_paged_fp4_workspace_bytes(5, 4, 8, 2, 128) > 0


def test_binding_rejects_bad_tensors():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    c, s = torch.zeros((4, 2, 16, 32), dtype=torch.uint8), torch.zeros((4, 2, 16, 4), dtype=torch.uint8)
    x, slots = torch.zeros((3, 2, 64)), torch.zeros(3, dtype=torch.int64)
    for call in (lambda: attn.attn_cache_append_fp4(x, x, slots, c, c.clone(), s, s.clone()),
                 lambda: attn.attn_cache_read_fp4(c, c, s, s, slots),
                 lambda: attn.attn_fwd_paged_fp4(x.half(), c, c, s, s, i32(1, 2), i32(2), i32(1)),
                 lambda: attn.attn_rope(x, x, torch.ones(32, dtype=torch.float64), positions=i32(3))):
        with pytest.raises(ValueError):  # CPU tensors
            call()


# ------------------------------------------------------------- frequencies
def test_frequencies():
    f, s = attn.attn_rope_frequencies(8, 10000.0, device="cpu")
    assert f.dtype == torch.float64 and s == 1.0
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14)
    g, s = attn.attn_rope_frequencies(8, 10000.0, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(g, f / 4, rtol=1e-14) and s == 1.0
    g, s = attn.attn_rope_frequencies(8, 10000.0, scaling="base", factor=4.0, device="cpu")
    assert g[0] == 1.0 and math.isclose(float(g[-1]), 0.001 / 4, rel_tol=1e-12) and s == 1.0
    g, s = attn.attn_rope_frequencies(128, 10000.0, scaling="parts", factor=8.0, original_length=4096, device="cpu")
    f = attn.attn_rope_frequencies(128, device="cpu")[0]
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(g[turns >= 32], f[turns >= 32])
    assert torch.allclose(g[turns <= 1], f[turns <= 1] / 8, rtol=1e-14)
    between = (turns > 1) & (turns < 32)
    assert between.any() and ((g < f) & (g > f / 8))[between].all()
    assert math.isclose(s, 0.1 * math.log(8.0) + 1)
    for kw in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, scaling="other"), dict(rotary_dim=8, base=0.0),
               dict(rotary_dim=8, scaling="parts"), dict(rotary_dim=2, scaling="base", factor=2.0),
               dict(rotary_dim=8, factor=-1.0, scaling="linear")):
        with pytest.raises(ValueError):
            attn.attn_rope_frequencies(device="cpu", **kw)


# ------------------------------------------------ the reference itself
def test_reference_encodes_by_hand():
    x = np.array([0.0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 9.0, np.inf, -0.3, -2.5, -1e9])
    want = [0.0, 0.0, 0.5, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 6.0, 6.0, -0.5, -2.0, -6.0]
    code = ref.encode_e2m1(x)
    assert (np.where(code & 8, -1.0, 1.0) * ref.E2M1[code & 7]).tolist() == want
    rows = np.zeros((1, 1, 64))
    rows[0, 0, :4] = [12.0, -6.0, 1.0, 0.5]     # scale 2: codes 6, -3, 0.5, 0 (a tie)
    rows[0, 0, 16] = 1e-6                        # below 6 * 2^-9: the smallest scale
    rows[0, 0, 32:34] = [np.inf, 6.0]            # the finite ones set the scale
    rows[0, 0, 48] = np.nan
    code, byte = ref.quantise(rows)
    held = ref.values(ref.pack(code)[:, :, None], byte[:, :, None])[0, 0, 0]
    assert held[:4].tolist() == [12.0, -6.0, 1.0, 0.0]
    assert byte[0, 0].tolist() == [64, 1, 56, 127] and held[16] == 0.0
    assert held[32:35].tolist() == [6.0, 6.0, 0.0] and np.isnan(held[48:]).all()


def test_two_products_round_as_the_quotient():
    """The codes of x rh + x rl, 1 / s as the sum of rh, rounded down, and rl, are those of x / s: for every scale, and
    every 16- and 32-bit x next to a border between codes, and many others."""
    f = np.float32
    rng = np.random.Generator(np.random.PCG64(3))
    for s in ref.E4M3[1:127]:
        rh = f(1 / s)
        if float(rh) > 1 / s:
            rh = np.nextafter(rh, f(0))
        rl = max(f(f(1 - float(rh) * s) * rh), f(rh * f(2.0 ** -60)))  # 1 - rh s is exact in 64 bits, as in the one rounding of an fma
        assert abs((float(rh) + float(rl)) * s - 1) < 2.0 ** -45
        near = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) * s
        x = []
        for t in (torch.bfloat16, torch.float16, torch.float32):
            y = torch.from_numpy(np.concatenate([near, rng.uniform(0, 8 * s, 200)])).to(t)
            bits = y.view(torch.int32 if t == torch.float32 else torch.int16)
            x += [(bits + i).view(t).double().numpy() for i in range(-2, 3)]
        x = np.concatenate(x)
        small = (x.astype(f) * rl).astype(f).astype(np.float64)
        # x rh is exact in 64 bits; the sum is rounded to 64 bits before 32, 2^-29 units of the last place apart
        q = (x * float(rh) + small).astype(f).astype(np.float64)
        assert np.array_equal(ref.encode_e2m1(q), ref.encode_e2m1(x / s)), s
