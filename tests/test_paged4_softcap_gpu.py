"""Soft-caps over the paged 4-bit cache at scores that reach the cap, in both kernels,
against 64 bits: the capped score is held to 2^-16 of itself, in the kernel for few
rows to 2^-19."""
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


def run(w, x):
    """(out, lse) of the call, in 64 bits on the CPU."""
    g = {n: None if t is None else t.cuda() for n, t in x.items()}
    lse = torch.zeros(g["q"].shape[:2], device="cuda")
    out = attn.attn_fwd_paged_fp4(g["q"], g["k_cache"], g["v_cache"], g["k_scales"], g["v_scales"], g["tables"], g["starts"],
                                  g["totals"], k_head_scales=g["k_heads"], v_head_scales=g["v_heads"], scale=w.scale,
                                  softcap=w.softcap, lse=lse)
    torch.cuda.synchronize()
    assert attn.get_device_status() == attn.ATTN_OK
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def attend(w, x, cap_error):
    """The causal definition, row by row: (out, lse, tolerance of each).

    Rows of q hold one value, so a raw score is one exact product: off by 2^-21 of itself (three roundings of factors, the
    product's), which the cap's slope of at most 1 lets through (and none of what passes 100 caps); the cap adds cap_error of the capped score.  For many rows that is what
    the call promises, 2^-16 (the hardware's tanh is off by 2^-16.46 of itself at most, over all fp32 arguments on this
    GPU); for few rows 2^-19 (a tanh to 2^-20 of itself, its product and the exponent's by 2^-24 each).  e is the sum of both, the lse is off by that and 2^-21 of its
    size, the output by 2 e A (A = sum p |v| / l), the weights' 2^-11 A, ex2 and sums 2^-18 A, half a step of the type, and
    weights below f16's range: 2^-29 sum |v| / l."""
    q = x["q"].double().numpy()
    num = lambda t: None if t is None else t.numpy()  # noqa: E731
    kc = ref.values(x["k_cache"].numpy(), x["k_scales"].numpy(), num(x["k_heads"]))
    vc = ref.values(x["v_cache"].numpy(), x["v_scales"].numpy(), num(x["v_heads"]))
    starts, totals, tables = (x[n].numpy() for n in ("starts", "totals", "tables"))
    T, Hq, D = q.shape
    scale = w.scale if w.scale is not None else D ** -0.5
    out, lse, tol, ltol = np.zeros((T, Hq, D)), np.zeros((T, Hq)), np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for b, L in enumerate(totals):
        at = np.arange(L)
        k, v = (c[tables[b, at // w.block], :, at % w.block] for c in (kc, vc))
        for t in range(starts[b], starts[b + 1]):
            n = L - (starts[b + 1] - 1 - t)  # keys it sees
            for h in range(Hq):
                kk, vv = k[:n, h * w.Hkv // Hq], v[:n, h * w.Hkv // Hq]
                raw = scale * (kk @ q[t, h])
                s = w.softcap * np.tanh(raw / w.softcap)
                e = (2.0 ** -21 * np.minimum(np.abs(raw), 100 * w.softcap) + cap_error * np.abs(s)).max()
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
                A = p @ np.abs(vv) / l
                out[t, h], lse[t, h] = p @ vv / l, m + np.log(l)
                tol[t, h] = (ref.HALF_STEP[w.dtype] * np.abs(out[t, h]) + A * (2.0 ** -11 + 2.0 ** -18 + 2 * e)
                             + 2.0 ** -29 * np.abs(vv).sum(0) / l + 1e-30)
                ltol[t, h] = e + 2.0 ** -21 * (1 + abs(lse[t, h]) + abs(m))
    return out, lse, tol, ltol


def check(w, x, cap_error):
    out, lse = run(w, x)
    want, wl, tol, ltol = attend(w, x, cap_error)
    n = sum(w.new)
    worst = np.abs(lse - wl)[:n] / ltol[:n]
    assert (worst <= 1).all(), f"lse: {worst.max():.2f} tolerances"
    worst = np.abs(out - want)[:n] / tol[:n]
    assert (worst <= 1).all(), f"out: {worst.max():.2f} tolerances"


@pytest.mark.parametrize("cap,std", [(1.0, 4.0), (50.0, 200.0), (50.0, 1000.0), (1000.0, 3e3), (3e4, 3e4)])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("new", [(2, 1), (150, 40)], ids=["few", "many"])
def test_capped_scores(new, dtype, D, cap, std):
    w = Problem(new=new, total=(400, 300), Hq=4, Hkv=1, D=D, dtype=dtype, softcap=cap, q_std=std, wide=True)
    x = ref.make(w)
    one = torch.randint(0, D, (*x["q"].shape[:2], 1), generator=torch.Generator().manual_seed(1))
    x["q"] = torch.zeros_like(x["q"]).scatter(2, one, x["q"].gather(2, one))
    x["q"].clamp_(-6e4, 6e4)  # finite in f16
    check(w, x, 2.0 ** (-16 if sum(new) > 100 else -19))


@pytest.mark.parametrize("cap", [2.0 ** 60, 2.0 ** 99])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new", [(2, 1), (150, 40)], ids=["few", "many"])
def test_large_caps_over_heads_of_small_keys(new, dtype, cap):
    """The factor from raw scores to the cap's argument lies below fp32's normal range: the scores are next to nothing, and
    every key has its share."""
    w = Problem(new=new, total=(400, 300), Hq=4, Hkv=1, D=64, dtype=dtype, softcap=cap, wide=True)
    x = ref.make(w)
    x["k_heads"] = torch.tensor([2.0 ** -60])
    x["q"] *= 8
    check(w, x, 2.0 ** -16)
