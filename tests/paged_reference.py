"""The paged 8-bit KV cache in plain numpy: the operators' definitions in 64
bits, one request, one block and one row at a time, and seeded problems.
Shares no code with the library."""
from __future__ import annotations

import dataclasses
from dataclasses import dataclass

import numpy as np
import torch

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # half a step of the type, relative to the value

# value of every e4m3 byte (sign, 4 exponent bits biased by 7, 3 mantissa bits; 0x7f / 0xff NaN)
E4M3 = np.zeros(256)
for _byte in range(256):
    _e, _m = (_byte >> 3) & 15, _byte & 7
    _v = _m * 2.0 ** -9 if _e == 0 else (1 + _m / 8) * 2.0 ** (_e - 7)
    E4M3[_byte] = np.nan if (_byte & 127) == 127 else (-_v if _byte & 128 else _v)
_POSITIVE = E4M3[:127]


def encode(x: np.ndarray) -> np.ndarray:
    """The byte of the e4m3 value nearest to x (ties to the even mantissa), |x| cut at 448, NaN kept."""
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_POSITIVE, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    with np.errstate(invalid="ignore"):
        dl, dh = a - _POSITIVE[lo], _POSITIVE[hi] - a
        byte = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    byte = np.where(np.isnan(x), 127, byte)
    return (byte | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_for(amax: float) -> float:
    s = 2.0 ** -100
    while amax > 448.0 * s:
        s *= 2.0
    return s


def append(x, slots, cache, scales):
    """x [T, Hkv, D] float64 into cache (bytes [N, Hkv, bs, D]) and scales [N, Hkv], in place."""
    N, Hkv, bs, _ = cache.shape
    t = 0
    while t < len(slots):
        if not 0 <= slots[t] < N * bs:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and slots[t + n] == slots[t] + n and slots[t + n] % bs != 0:
            n += 1
        blk, off = int(slots[t] // bs), int(slots[t] % bs)
        for h in range(Hkv):
            rows = x[t:t + n, h]
            finite = np.abs(rows[np.isfinite(rows)])
            s = scale_for(float(finite.max()) if finite.size else 0.0)
            if off > 0:
                s = max(s, float(scales[blk, h]))
                if s > scales[blk, h]:
                    cache[blk, h, :off] = encode(E4M3[cache[blk, h, :off]] * (float(scales[blk, h]) / s))
            cache[blk, h, off:off + n] = encode(rows / s)
            scales[blk, h] = s
        t += n


def assign(past, new, finished, tables, free, count, block, T):
    """One step; returns (q_starts, totals, slot_map, result, count) and updates tables and free in place."""
    B, width = tables.shape
    tb, fr, n = tables.copy(), free.copy(), int(count)
    zero = (np.zeros(B + 1, np.int32), past.copy(), np.full(T, -1, np.int64))
    p = np.where(finished, 0, past)
    if (past < 0).any() or (new < 0).any():
        return (*zero, 4, int(count))
    need = -(-(p.astype(np.int64) + new) // block)
    if (need > width).any():
        return (*zero, 2, int(count))
    if new.sum() > T:
        return (*zero, 3, int(count))
    for b in np.flatnonzero(finished):
        for e in tb[b]:
            if e >= 0:
                fr[n] = e
                n += 1
        tb[b] = -1
    for b in range(B):
        for i in range(need[b]):
            if tb[b, i] < 0:
                if n == 0:
                    return (*zero, 1, int(count))
                n -= 1
                tb[b, i] = fr[n]
    tables[:], free[:] = tb, fr
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    slots = np.full(T, -1, np.int64)
    for b in range(B):
        pos = p[b] + np.arange(new[b])
        slots[starts[b]:starts[b + 1]] = tb[b][pos // block].astype(np.int64) * block + pos % block
    return starts, (p + new).astype(np.int32), slots, 0, n


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
    free_scales: bool = False   # scales that are no powers of two, far apart
    strided: bool = False
    sink: float = 0.0   # > 0: key 0 of every request points along every query, its V row is small
    seed: int = 5

    def replace(self, **kw):
        return dataclasses.replace(self, **kw)


def make(w: Problem) -> dict:
    """CPU tensors of a problem.  Slots at or past a request's length and blocks of
    no request hold NaN bytes; table entries past a request's blocks name nothing."""
    rng = np.random.Generator(np.random.PCG64(w.seed))
    B, T = len(w.new), sum(w.new) + w.pad
    held = [-(-max(t, 0) // w.block) for t in w.total]
    width, N = max(held + [1]) + 1, sum(held) + 2
    pool = rng.permutation(N)
    tables = rng.choice(np.array([-1, -7, N, N + 5, 2 ** 31 - 1]), size=(B, width)).astype(np.int64)
    at = 0
    for b, n in enumerate(held):
        tables[b, :n] = pool[at:at + n]
        at += n
    q = rng.standard_normal((T, w.Hq, w.D)) * w.q_std
    caches, scales = [], []
    for _ in range(2):
        c = encode(rng.standard_normal((N, w.Hkv, w.block, w.D)) * rng.choice([20.0, 60.0, 150.0], size=(N, w.Hkv, 1, 1)))
        s = 2.0 ** rng.integers(-8, -3, size=(N, w.Hkv))
        if w.free_scales:
            s = s * rng.uniform(0.5, 2.0, size=s.shape)
        caches.append(c)
        scales.append(s.astype(np.float32))
    if w.free_scales:  # V scales of very different size from block to block
        scales[1] *= np.float32(2.0) ** rng.integers(-12, 12, size=scales[1].shape).astype(np.float32)
    if w.sink > 0:
        q = np.abs(q)
    used = np.zeros((N, w.block), bool)
    for b, t in enumerate(w.total):
        for p in range(max(t, 0)):
            used[tables[b, p // w.block], p % w.block] = True
        if w.sink > 0 and t > 0:
            blk = int(tables[b, 0])
            caches[0][blk, :, 0] = encode(np.full(w.D, w.sink))
            scales[0][blk] = 2.0 ** -4
            caches[1][blk, :, 0] = encode(np.full(w.D, 2.0 ** -6))
    for c in caches:
        c.transpose(0, 2, 1, 3)[~used] = 127
    starts = np.concatenate([[0], np.cumsum(w.new)])
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32))  # noqa: E731
    return dict(q=torch.from_numpy(q).to(TORCH[w.dtype]), k_cache=torch.from_numpy(caches[0]),
                v_cache=torch.from_numpy(caches[1]), k_scales=torch.from_numpy(scales[0]),
                v_scales=torch.from_numpy(scales[1]), tables=i32(tables), starts=i32(starts), totals=i32(w.total))


def attend(w: Problem, x: dict):
    """(out [T, Hq, D], lse [T, Hq], tolerance of out, tolerance of lse) in 64 bits; rows of no request are NaN.

    The tolerance of out, from the kernels' arithmetic (A = sum_j p_j |v_j|, l = sum of exp(s - max)):
      half a step of the output type on the result;
      weights carried to at least 11 bits (relative 2^-11), and below 2^-13 of the
      row's largest to an absolute 2^-24:  A 2^-11 + 2^-24 sum |v_j| / l;
      scores off by at most e:  2 e A, where e = scale (2^-16 sum_d |q_d k_d| + 2^-18 max|q| sum_d |k_d|)
      (fp32 sums over the row; q in pieces whose rest is below 2^-18 of the row's largest element),
      and with a soft-cap the hardware tanh's 2^-10.9: softcap 2^-10.9;
    the tolerance of lse: e, and fp32's rounding of the result.
    """
    q = x["q"].double().numpy()
    starts, totals, tables = x["starts"].numpy(), x["totals"].numpy(), x["tables"].numpy()
    kc, vc = E4M3[x["k_cache"].numpy()], E4M3[x["v_cache"].numpy()]
    ks, vs = x["k_scales"].double().numpy(), x["v_scales"].double().numpy()
    T, Hq, D = q.shape
    Hkv, bs = kc.shape[1:3]
    scale = w.scale if w.scale is not None else D ** -0.5
    out, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    tol, ltol = np.zeros_like(out), np.zeros_like(lse)
    half = HALF_STEP[w.dtype]
    for b in range(len(totals)):
        L, n = max(int(totals[b]), 0), int(starts[b + 1] - starts[b])
        blk = tables[b, np.arange(L) // bs]
        k = kc[blk, :, np.arange(L) % bs] * ks[blk][..., None]  # [L, Hkv, D]
        v = vc[blk, :, np.arange(L) % bs] * vs[blk][..., None]
        for i in range(n):
            t, pos = int(starts[b]) + i, int(totals[b]) - n + i
            lo = max(0, pos + 1 - w.window) if w.window > 0 else 0
            hi = min(L, pos + 1) if w.causal else L
            if hi <= lo:
                out[t], lse[t] = 0.0, -np.inf
                continue
            for h in range(Hq):
                kk, vv, qq = k[lo:hi, h * Hkv // Hq], v[lo:hi, h * Hkv // Hq], q[t, h]
                s = scale * (kk @ qq)
                e = abs(scale) * (2.0 ** -16 * (np.abs(kk) @ np.abs(qq)).max()
                                  + 2.0 ** -18 * np.abs(qq).max() * np.abs(kk).sum(1).max())
                if w.softcap > 0:
                    s = w.softcap * np.tanh(s / w.softcap)
                    e += w.softcap * 2.0 ** -10.9
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
                out[t, h] = p @ vv / l
                lse[t, h] = m + np.log(l)
                A = p @ np.abs(vv) / l
                tol[t, h] = (half * np.abs(out[t, h]) + A * (2.0 ** -11 + 2 * e) + 2.0 ** -24 * np.abs(vv).sum(0) / l
                             + 1e-30)
                ltol[t, h] = e + 2.0 ** -21 * (1 + abs(lse[t, h]) + abs(m))
    return out, lse, tol, ltol
