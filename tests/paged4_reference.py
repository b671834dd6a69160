"""The paged 4-bit KV cache and rotary positions in plain numpy: the operators'
definitions in 64 bits, and seeded problems.  Shares no code with the library."""
from __future__ import annotations

import dataclasses
from dataclasses import dataclass

import numpy as np
import torch

import paged_reference as ref8

TORCH, HALF_STEP, E4M3 = ref8.TORCH, ref8.HALF_STEP, ref8.E4M3
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
GROUP = 16


def encode_e2m1(x):
    """The code (sign in bit 3) of the e2m1 value nearest to x, ties to the even code, |x| cut at 6."""
    a = np.minimum(np.abs(x), 6.0)
    hi = np.clip(np.searchsorted(E2M1, a), 0, 7)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - E2M1[lo], E2M1[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def quantise(x, heads=None):
    """(codes [..., H, D], scale bytes [..., H, D / 16]) of rows [..., H, D] float64."""
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    h = np.ones(x.shape[-2], np.float32) if heads is None else heads.astype(np.float32)
    h = h[:, None]
    nan = np.isnan(g).any(-1)
    amax = np.where(np.isfinite(g), np.abs(g), 0.0).max(-1).astype(np.float32)
    with np.errstate(all="ignore"):
        byte = np.maximum(ref8.encode((amax / (np.float32(6) * h)).astype(np.float64)) & 127, 1)
        unit = (E4M3[byte].astype(np.float32) * h)[..., None]
        code = encode_e2m1((np.where(nan[..., None], 0.0, g).astype(np.float32) / unit).astype(np.float64))
    code = np.where(nan[..., None], 0, code).reshape(x.shape)
    return code.astype(np.uint8), np.where(nan, 127, byte).astype(np.uint8)


def pack(code):
    return (code[..., 0::2] | code[..., 1::2] << 4).astype(np.uint8)


def values(packed, scales, heads=None):
    """Values [..., H, ..., D] of bytes and scales whose axis 1 is the kv head (a whole cache's)."""
    code = np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)
    x = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7] * np.repeat(E4M3[scales], GROUP, -1)
    if heads is not None:
        x = x * heads.astype(np.float64).reshape(1, -1, *[1] * (x.ndim - 2))
    return x


def append(x, slots, cache, scales, heads=None):
    """x [T, Hkv, D] float64 into cache and scales, in place."""
    N, _, bs, _ = cache.shape
    code, byte = quantise(x, heads)
    for t, s in enumerate(slots):
        if 0 <= s < N * bs:
            cache[s // bs, :, s % bs] = pack(code[t])
            scales[s // bs, :, s % bs] = byte[t]


@dataclass(frozen=True)
class Problem:
    new: tuple          # new tokens of each request
    total: tuple        # cached length of each request, its new tokens among them
    Hq: int = 8
    Hkv: int = 2
    D: int = 128
    block: int = 64
    dtype: str = "bf16"
    causal: bool = True
    window: int = 0
    softcap: float = 0.0
    scale: float | None = None
    pad: int = 3        # rows behind the last request
    q_std: float = 1.0
    k_std: float = 1.0
    heads: bool = False     # head scales, no powers of two
    spread: bool = False    # group scales over all that e4m3 holds
    strided: bool = False
    wide: bool = False      # block tables as for contexts of a million tokens: calls with many rows go to their kernel
    sink: float = 0.0       # > 0: key 0 of every request points along every query, its V row is small
    seed: int = 5

    def replace(self, **kw):
        return dataclasses.replace(self, **kw)


def make(w: Problem) -> dict:
    """CPU tensors of a problem.  Slots at or past a request's length and blocks of
    no request have NaN scales; table entries past a request's blocks name nothing."""
    rng = np.random.Generator(np.random.PCG64(w.seed))
    B, T = len(w.new), sum(w.new) + w.pad
    held = [-(-max(t, 0) // w.block) for t in w.total]
    width, N = max(held + [1]) + 1 + (2 ** 20 // w.block if w.wide else 0), sum(held) + 2
    pool = rng.permutation(N)
    tables = rng.choice(np.array([-1, -7, N, N + 5, 2 ** 31 - 1]), size=(B, width)).astype(np.int64)
    at = 0
    for b, n in enumerate(held):
        tables[b, :n] = pool[at:at + n]
        at += n
    q = rng.standard_normal((T, w.Hq, w.D)) * w.q_std
    if w.sink > 0:
        q = np.abs(q)
    caches, scales, heads = [], [], []
    for std in (w.k_std, 1.0):
        h = rng.uniform(0.3, 3.0, w.Hkv).astype(np.float32) if w.heads else None
        x = rng.standard_normal((N, w.block, w.Hkv, w.D)) * std
        code, byte = quantise(x, h)
        if w.spread:
            byte = rng.integers(1, 127, size=byte.shape).astype(np.uint8)
        caches.append(np.ascontiguousarray(pack(code).swapaxes(1, 2)))
        scales.append(np.ascontiguousarray(byte.swapaxes(1, 2)))
        heads.append(h)
    used = np.zeros((N, w.block), bool)
    for b, t in enumerate(w.total):
        for p in range(max(t, 0)):
            used[tables[b, p // w.block], p % w.block] = True
        if w.sink > 0 and t > 0:
            blk = int(tables[b, 0])
            caches[0][blk, :, 0] = 0x77  # 6, 6
            scales[0][blk, :, 0] = ref8.encode(np.array([w.sink / 6]))[0]
            scales[1][blk, :, 0] = 8     # 2^-6
    for s in scales:
        s.swapaxes(1, 2)[~used] = 127
    starts = np.concatenate([[0], np.cumsum(w.new)])
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32))  # noqa: E731
    tensor = lambda a: None if a is None else torch.from_numpy(a)  # noqa: E731
    return dict(q=torch.from_numpy(q).to(TORCH[w.dtype]), k_cache=tensor(caches[0]), v_cache=tensor(caches[1]),
                k_scales=tensor(scales[0]), v_scales=tensor(scales[1]), k_heads=tensor(heads[0]),
                v_heads=tensor(heads[1]), tables=i32(tables), starts=i32(starts), totals=i32(w.total))


def attend(w: Problem, x: dict):
    """(out [T, Hq, D], lse [T, Hq], tolerance of out, tolerance of lse) in 64 bits; rows of no request are NaN.

    The tolerance of out, from the kernels' arithmetic (A = sum_j p_j |v_j| / l, l = sum of exp(s - max) >= 1):
      half a step of the output type on the result;
      weights rounded to f16: 2^-11 of themselves, or, below f16's normal range, an absolute 2^-25 where the row's
      largest is 2^5 or more (2^-24 allowed, relative to the largest):  A 2^-11 + 2^-29 sum |v_j| / l;
      the hardware's ex2 and the row sum, and fp32 sums over the keys (one addition of 16 keys a time at most, off
      by 2^-23 of A each):  A (2^-20 + L 2^-27);
      scores off by at most e:  2 e A, where e = scale (2^-16 sum_d |q_d k_d| + 2^-31 max|q| sum_d |k_d|) + 2^-21 |s|
      (exact products summed in fp32, off by 2^-23 of the magnitude for each of 128 additions; a bf16 row as f16 by
      a power of two loses what is 2^-31 of its largest element; three roundings of the factors), and with a
      soft-cap the hardware tanh's specification, 2^-11 of the capped score (2^-10.9 allowed);
    the tolerance of lse: e, and fp32's rounding of the result.
    """
    q = x["q"].double().numpy()
    starts, totals, tables = x["starts"].numpy(), x["totals"].numpy(), x["tables"].numpy()
    num = lambda t: None if t is None else t.numpy()  # noqa: E731
    kc = values(x["k_cache"].numpy(), x["k_scales"].numpy(), num(x["k_heads"]))
    vc = values(x["v_cache"].numpy(), x["v_scales"].numpy(), num(x["v_heads"]))
    T, Hq, D = q.shape
    Hkv, bs = kc.shape[1:3]
    scale = w.scale if w.scale is not None else D ** -0.5
    out, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    tol, ltol = np.zeros_like(out), np.zeros_like(lse)
    half = HALF_STEP[w.dtype]
    for b in range(len(totals)):
        L, n = max(int(totals[b]), 0), int(starts[b + 1] - starts[b])
        if n == 0:
            continue
        blk = tables[b, np.arange(L) // bs]
        rows = slice(int(starts[b]), int(starts[b + 1]))
        pos = (int(totals[b]) - n + np.arange(n))[:, None]
        key = np.arange(L)[None]
        hide = np.zeros((n, L), bool)
        if w.causal:
            hide |= key > pos
        if w.window > 0:
            hide |= key <= pos - w.window
        empty = hide.all(1)
        k, v = kc[blk, :, np.arange(L) % bs], vc[blk, :, np.arange(L) % bs]  # [L, Hkv, D]
        for h in range(Hq):
            kk, vv, qq = k[:, h * Hkv // Hq], v[:, h * Hkv // Hq], q[rows, h]
            s = scale * (qq @ kk.T)
            mag = np.where(hide, 0.0, np.abs(qq) @ np.abs(kk).T)
            e = np.zeros(n) if L == 0 else abs(scale) * (2.0 ** -16 * mag.max(1) + 2.0 ** -31 * np.abs(qq).max(1)
                                                          * np.abs(kk).sum(1).max())
            if L:
                e = e + 2.0 ** -21 * np.abs(np.where(hide, 0.0, s)).max(1)
            if w.softcap > 0:
                s = w.softcap * np.tanh(s / w.softcap)
                e = e + (2.0 ** -10.9 * np.abs(np.where(hide, 0.0, s)).max(1) if L else 0.0)
            s = np.where(hide, -np.inf, s)
            m = np.where(empty, 0.0, s.max(1, initial=-np.inf))
            p = np.exp(s - m[:, None])
            l = np.where(empty, 1.0, p.sum(1))
            o = p @ vv / l[:, None]
            A = p @ np.abs(vv) / l[:, None]
            most = np.where(hide, 0.0, 1.0) @ np.abs(vv) / l[:, None]
            out[rows, h] = o
            tol[rows, h] = (half * np.abs(o) + A * (2.0 ** -11 + 2.0 ** -20 + L * 2.0 ** -27 + 2 * e[:, None])
                            + 2.0 ** -29 * most + 1e-30)
            with np.errstate(divide="ignore"):
                lse[rows, h] = np.where(empty, -np.inf, m + np.log(l))
            ltol[rows, h] = np.where(empty, 0.0, e + 2.0 ** -21 * (1 + np.abs(np.where(empty, 0.0, lse[rows, h])) + np.abs(m)))
    return out, lse, tol, ltol


def rope(x, pos, freq, interleaved, inverse, scale):
    """x [T, H, D] float64 turned, pair by pair; angles in longdouble."""
    R = 2 * len(freq)
    turn = np.longdouble("6.28318530717958647692528676655900577")
    w = (pos.astype(np.longdouble)[:, None] * freq.astype(np.longdouble)) % turn
    c, n = np.cos(w.astype(np.float64))[:, None] * scale, np.sin(w.astype(np.float64))[:, None] * scale
    if inverse:
        n = -n
    y = x.copy()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y[..., a] = x[..., a] * c - x[..., b] * n
    y[..., b] = x[..., b] * c + x[..., a] * n
    return y
