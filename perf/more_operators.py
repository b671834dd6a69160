"""A paged KV cache held in 4 bits, and rotary positions: what is measured of them, and the operators' plain forms.

Four operators serve one step of a batch of requests beside the block assignment of the paged cache:
  rope     rotary positions onto the step's query and key rows, and their inverse for gradients
  append   the new K / V rows into the cache as e2m1, with one e4m3 scale for every 16 values of a row,
           and back out of it
  read     rows of the cache as 16- or 32-bit values
  attend   attention of the new tokens over the cache
`run` is one pass through one of them: the library's calls where `own` is true, elementary torch operations in 32
bits where it is false.  `exact` is the definition again in 64 bits.
"""
import math

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
GROUP = 16  # values of a row that share a scale
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one decode step of a full batch: a token each, q and k as slices of a fused projection's output
        dict(name="rope_decode", op="rope", B=64, Hq=32, Hkv=8, D=128, rotary=128, dtype="bf16", new_min=1, new_max=1,
             past_max=8000, layout="half", stretch=1.0, inverse=False, strided=True, given="lengths"),
        # gradients of two whole sequences far out in a stretched context, half of each head rotated, pairs side by side
        dict(name="rope_gradients", op="rope", B=2, Hq=32, Hkv=8, D=128, rotary=64, dtype="bf16", new_min=4096,
             new_max=4096, past_max=120000, layout="interleaved", stretch=8.0, inverse=True, strided=False,
             given="positions"),
        # the decode step's K / V rows, and the rows as the cache holds them
        dict(name="append_decode", op="append", B=64, Hkv=8, D=128, block=64, dtype="bf16", new_min=1, new_max=1,
             past_max=8000, strided=False, head_scales=False),
        # whole prompts, whose dense attention sees what the cache holds
        dict(name="append_prompts", op="append", B=8, Hkv=8, D=128, block=64, dtype="bf16", new_min=1, new_max=4096,
             past_max=0, strided=True, head_scales=True),
        # a ragged batch's contexts, in a slot map padded for a captured graph
        dict(name="read_ragged", op="read", B=13, Hkv=4, D=64, block=16, dtype="f16", past_min=1, past_max=900, pad=77,
             head_scales=True),
        # one long request leaves for another place
        dict(name="read_long", op="read", B=1, Hkv=8, D=128, block=64, dtype="bf16", past_min=32700, past_max=32700,
             pad=0, head_scales=False),
        # one request's next token: latency
        dict(name="decode_one", op="attend", B=1, Hq=32, Hkv=8, D=128, block=64, dtype="bf16", new_min=1, new_max=1,
             past_min=3000, past_max=4000, causal=True, window=0, softcap=0.0, pad=0, head_scales=False),
        # few requests with long contexts (the decode workload of the benchmark, its cache in 4 bits)
        dict(name="decode_long", op="attend", B=8, Hq=32, Hkv=8, D=128, block=64, dtype="bf16", new_min=1, new_max=1,
             past_min=9000, past_max=32700, causal=True, window=0, softcap=0.0, pad=0, head_scales=False),
        # a full batch, eight query heads to a kv head, small blocks
        dict(name="decode_batch", op="attend", B=64, Hq=32, Hkv=4, D=128, block=16, dtype="f16", new_min=1, new_max=1,
             past_min=100, past_max=8000, causal=True, window=0, softcap=0.0, pad=0, head_scales=True),
        # a few drafted tokens to verify in each request, sliding window and soft-cap
        dict(name="verify_window", op="attend", B=19, Hq=16, Hkv=8, D=64, block=32, dtype="f16", new_min=1, new_max=5,
             past_min=0, past_max=8000, causal=True, window=1024, softcap=50.0, pad=0, head_scales=False),
        # chunked prefill over ragged caches (the benchmark's ragged workload), its rows padded for a captured graph
        dict(name="chunk_ragged", op="attend", B=8, Hq=32, Hkv=4, D=128, block=64, dtype="f16", new_min=100,
             new_max=128, past_min=0, past_max=3900, causal=True, window=0, softcap=0.0, pad=107, head_scales=False),
        # a large chunk far into long contexts
        dict(name="chunk_long", op="attend", B=2, Hq=32, Hkv=8, D=128, block=128, dtype="bf16", new_min=1500,
             new_max=2048, past_min=9000, past_max=14000, causal=True, window=0, softcap=0.0, pad=0,
             head_scales=False),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "read", "attend", "attend", "attend", "attend"])
    heads = rng.choice([(32, 8), (32, 4), (16, 8), (8, 8), (15, 3), (12, 1)])
    base = dict(op=op, Hkv=heads[1], D=rng.choice([64, 128]), dtype=rng.choice(["bf16", "f16"]))
    if op == "rope":
        D = rng.choice([64, 96, 128, 256])
        B = _log_uniform(rng, 1, 64)
        new_max = rng.choice([1, _log_uniform(rng, 1, 8192 // B)])
        return dict(base, Hq=heads[0], D=D, rotary=rng.choice([D, D, D // 2, D // 4]), B=B, new_min=1 if B < 4 else 0,
                    new_max=new_max, past_max=_log_uniform(rng, 1, 200000), layout=rng.choice(["half", "interleaved"]),
                    stretch=rng.choice([1.0, 4.0, 16.0]), inverse=rng.random() < 0.4, strided=rng.random() < 0.5,
                    given=rng.choice(["lengths", "positions"]), dtype=rng.choice(["bf16", "f16", "f32"]))
    base = dict(base, block=rng.choice([16, 32, 64, 128]), head_scales=rng.random() < 0.5)
    if op == "append":
        B = _log_uniform(rng, 1, 100)
        return dict(base, B=B, new_min=1, new_max=rng.choice([1, 5, _log_uniform(rng, 1, 24000 // B)]),
                    past_max=_log_uniform(rng, 1, 4000), strided=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "f16", "f32"]))
    if op == "read":
        B = _log_uniform(rng, 1, 40)
        return dict(base, B=B, past_min=1, past_max=_log_uniform(rng, 1, 48000 // B), pad=rng.choice([0, 1, 300]),
                    dtype=rng.choice(["bf16", "f16", "f32"]))
    kind = rng.choice(["decode", "decode", "verify", "chunk"])
    if kind == "chunk":
        B = _log_uniform(rng, 1, 8)
        new_max = _log_uniform(rng, 16, 2048 // B)
        past_max = _log_uniform(rng, 1, 8000)
    else:
        B = _log_uniform(rng, 1, 64)
        new_max = 1 if kind == "decode" else rng.randint(2, 7)
        past_max = _log_uniform(rng, 10, min(32000, 500000 // B))
    return dict(base, B=B, Hq=heads[0], new_min=1 if B <= 3 or new_max == 1 else 0, new_max=new_max, past_min=0,
                past_max=past_max, causal=rng.random() < 0.85, window=rng.choice([0, 0, 100, 1024]),
                softcap=rng.choice([0.0, 0.0, 30.0]), pad=rng.choice([1, 1, 9]))


# ------------------------------------------------------------------- inputs
def _spread(lo, hi, n):
    """n whole numbers spread evenly over lo .. hi, both ends among them where n allows."""
    return np.clip(np.rint(lo - 0.49 + (hi - lo + 0.98) * (np.arange(n) + 0.5) / n), lo, hi).astype(np.int32)


def _lengths(case, seed):
    """(past, new) of the requests, int32 numpy: even spreads, in an order that the seed gives."""
    rng = np.random.Generator(np.random.PCG64([int(seed), 12]))
    B = case["B"]
    past = rng.permutation(_spread(case.get("past_min", 0), case["past_max"], B))
    new = rng.permutation(_spread(case.get("new_min", 0), case.get("new_max", 0), B))
    return past, new, rng


def _exclusive(x):
    return np.concatenate([[0], np.cumsum(x)]).astype(np.int64)


def _gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _tables(past, new, block, rng, width):
    """Block tables over a scattered pool, as an allocator in use leaves them: (tables [B, width], num_blocks)."""
    held = -(-(past.astype(np.int64) + new) // block)
    num_blocks = int(held.sum()) + 3
    pool, at = rng.permutation(num_blocks).astype(np.int32), _exclusive(held)
    tables = np.full((len(held), width), -1, np.int32)
    for b, n in enumerate(held):
        tables[b, :n] = pool[at[b]:at[b] + n]
    return tables, num_blocks


def _slots(tables, first, count, block):
    """The slots of positions first .. first + count of every request, one request after the other."""
    at = [p + np.arange(n) for p, n in zip(first, count)]
    return np.concatenate([tables[b][pos // block].astype(np.int64) * block + pos % block
                           for b, pos in enumerate(at)] or [np.zeros(0, np.int64)])


def _generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    return gen


def _head_scales(case, gen):
    """Scales of the kv heads, as a calibration leaves them (powers of two), or none."""
    if not case["head_scales"]:
        return None, None
    pow2 = lambda: torch.ldexp(torch.ones(case["Hkv"], device="cuda"), torch.randint(  # noqa: E731
        -3, 3, (case["Hkv"],), generator=gen, device="cuda"))
    return pow2(), pow2()


def _cache(num_blocks, case, heads, gen):
    """A cache of N(0, 1) rows with uneven channels: (bytes, scales)."""
    Hkv, block, D = case["Hkv"], case["block"], case["D"]
    gain = torch.exp(0.3 * torch.randn((1, Hkv, 1, D), generator=gen, device="cuda"))
    made = ([], [])
    for at in range(0, num_blocks, 1 + (1 << 26) // (Hkv * block * D)):
        n = min(num_blocks - at, 1 + (1 << 26) // (Hkv * block * D))
        x = torch.randn((n, Hkv, block, D), generator=gen, device="cuda").mul_(gain)
        code, scale = _encode(x, None if heads is None else heads[:, None])
        made[0].append(code)
        made[1].append(scale)
    return torch.cat(made[0]), torch.cat(made[1])


def _prepare_cache(case, past, new, rng, gen):
    tables, num_blocks = _tables(past, new, case["block"], rng, -(-(case["past_max"] + case.get("new_max", 0))
                                                                 // case["block"]))
    kh, vh = _head_scales(case, gen)
    kc, ks = _cache(num_blocks, case, kh, gen)
    vc, vs = _cache(num_blocks, case, vh, gen)
    return tables, dict(k_cache=kc, v_cache=vc, k_scales=ks, v_scales=vs, k_heads=kh, v_heads=vh, block=case["block"])


def _frequencies(case):
    """Angle a position of every pair, float64, and the factor on the rotated values: 10000^(-2i/rotary), of which the
    slow ones are stretched for a longer context and the fast ones kept, with a ramp between them."""
    R = case["rotary"]
    f = 10000.0 ** (-np.arange(0, R, 2) / R)
    if case["stretch"] == 1.0:
        return f, 1.0
    original = 4096
    turns = original * f / (2 * math.pi)  # over the context that was trained on
    keep = np.clip((np.log2(turns) - 0.0) / 5.0, 0.0, 1.0)  # all of it from 32 turns on, none below one
    return f * (keep + (1 - keep) / case["stretch"]), 0.1 * math.log(case["stretch"]) + 1.0


def _rows(shape, case, gen, wide):
    T, H, D = shape
    x = torch.randn((T, H + wide, D), generator=gen, device="cuda")
    return x.to(DTYPES[case["dtype"]])[:, :H]


def _prepare_rope(case, seed):
    past, new, rng = _lengths(case, seed)
    starts = _exclusive(new)
    T, gen = int(starts[-1]), _generator(seed)
    f, scale = _frequencies(case)
    s = dict(op="rope", q=_rows((T, case["Hq"], case["D"]), case, gen, 2 * case["Hkv"] if case["strided"] else 0),
             k=_rows((T, case["Hkv"], case["D"]), case, gen, case["Hkv"] if case["strided"] else 0),
             freq=_gpu(f), scale=scale, layout=case["layout"], inverse=case["inverse"], positions=None, starts=None,
             totals=None)
    if case["given"] == "positions":
        s["positions"] = _gpu(np.concatenate([p + np.arange(n) for p, n in zip(past, new)]).astype(np.int32))
    else:
        s["starts"], s["totals"] = _gpu(starts.astype(np.int32)), _gpu((past + new).astype(np.int32))
    return s


def _prepare_append(case, seed):
    past, new, rng = _lengths(case, seed)
    gen = _generator(seed)
    tables, s = _prepare_cache(case, past, new, rng, gen)
    slots = _slots(tables, past, new, case["block"])
    shape = (len(slots), case["Hkv"], case["D"])
    wide = 2 * case["Hkv"] if case["strided"] else 0
    k, v = (_rows(shape, case, gen, wide) for _ in range(2))
    loud = torch.exp(0.5 * torch.randn((shape[0], 1, 1), generator=gen, device="cuda")).to(k.dtype)
    for x in (k, v):
        x.mul_(loud)  # louder rows now and then
    return dict(s, op="append", k=k, v=v, slots=_gpu(slots))


def _prepare_read(case, seed):
    past, new, rng = _lengths(case, seed)
    tables, s = _prepare_cache(case, past, new, rng, _generator(seed))
    slots = np.concatenate([_slots(tables, 0 * past, past, case["block"]), np.full(case["pad"], -1, np.int64)])
    return dict(s, op="read", slots=_gpu(slots), dtype=DTYPES[case["dtype"]])


def _prepare_attend(case, seed):
    past, new, rng = _lengths(case, seed)
    gen = _generator(seed)
    tables, s = _prepare_cache(case, past, new, rng, gen)
    starts = _exclusive(new).astype(np.int32)
    shape = (int(starts[-1]) + case["pad"], case["Hq"], case["D"])
    return dict(s, op="attend", q=_rows(shape, case, gen, 0), tables=_gpu(tables), starts=_gpu(starts),
                totals=_gpu((past + new).astype(np.int32)),
                out=torch.zeros(shape, dtype=DTYPES[case["dtype"]], device="cuda"), most_new=max(1, int(new.max())),
                causal=case["causal"], window=case["window"], softcap=case["softcap"])


def prepare(case, seed):
    return {"rope": _prepare_rope, "append": _prepare_append, "read": _prepare_read,
            "attend": _prepare_attend}[case["op"]](case, seed)


# -------------------------------------------------------------- plain forms
def _encode(x, heads):
    """(bytes [..., D/2], scales [..., D/16] e4m3) of 32-bit rows [..., D]; `heads` broadcasts against x without its
    last axis, or is None."""
    x = x.reshape(*x.shape[:-1], -1, GROUP)
    h = torch.ones((), device=x.device) if heads is None else heads[..., None]
    scale = (x.abs().amax(-1) / (6.0 * h)).clamp(max=448.0).to(E4M3).float().clamp(min=2.0 ** -9)
    a = (x / (scale * h)[..., None])
    sign = torch.signbit(a)
    a = a.abs()
    # borders between 0, 1/2, 1, 3/2, 2, 3, 4 and 6; a value on one goes to the even neighbour
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
            + (a >= 3.5).byte() + (a > 5.0).byte() + 8 * sign.byte()).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.to(E4M3)


def _decode(code, scale, heads):
    """32-bit rows [..., D] of bytes and scales."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=code.device)
    x = torch.stack([table[(code & 15).int()], table[(code >> 4).int()]], -1).flatten(-2)
    x = x.reshape(*x.shape[:-1], -1, GROUP) * scale.float()[..., None]
    if heads is not None:
        x = x * heads[..., None, None]
    return x.flatten(-2)


def _plain_rope(s):
    T, f = s["q"].shape[0], s["freq"]
    if s["positions"] is not None:
        pos = s["positions"].long()
    else:
        t = torch.arange(T, device=f.device)
        starts, totals = s["starts"].long(), s["totals"].long()
        b = torch.searchsorted(starts[1:].contiguous(), t, right=True)
        pos = totals[b] - starts[b + 1] + t
    angle = pos[:, None].double() * f  # a far position's angle needs more than 24 bits
    c, n = (torch.cos(angle) * s["scale"]).float()[:, None], (torch.sin(angle) * s["scale"]).float()[:, None]
    if s["inverse"]:
        n = -n
    made, R = [], 2 * f.shape[0]
    for x in (s["q"], s["k"]):
        y = x.float()
        if s["layout"] == "half":
            a, b = y[..., :R // 2], y[..., R // 2:R]
            turned = [a * c - b * n, b * c + a * n]
        else:
            a, b = y[..., 0:R:2], y[..., 1:R:2]
            turned = [torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)]
        made.append(torch.cat(turned + [y[..., R:]], -1).to(x.dtype))
    return tuple(made)


def _plain_append(s):
    blk, off = s["slots"] // s["block"], s["slots"] % s["block"]
    held = []
    for x, cache, scales, heads in ((s["k"], s["k_cache"], s["k_scales"], s["k_heads"]),
                                    (s["v"], s["v_cache"], s["v_scales"], s["v_heads"])):
        code, scale = _encode(x.float(), heads)
        cache[blk, :, off] = code
        scales.view(torch.uint8)[blk, :, off] = scale.view(torch.uint8)
        held.append(_decode(cache[blk, :, off], scales.view(torch.uint8)[blk, :, off].view(E4M3), heads).to(x.dtype))
    return (*held, s["k_scales"], s["v_scales"])


def _plain_read(s):
    there = s["slots"] >= 0
    at = s["slots"].clamp(min=0)
    blk, off = at // s["block"], at % s["block"]
    held = []
    for cache, scales, heads in ((s["k_cache"], s["k_scales"], s["k_heads"]),
                                 (s["v_cache"], s["v_scales"], s["v_heads"])):
        x = _decode(cache[blk, :, off], scales.view(torch.uint8)[blk, :, off].view(E4M3), heads)
        held.append(torch.where(there[:, None, None], x, 0.0).to(s["dtype"]))
    return tuple(held)


def _plain_rows(cache, scales, heads, tables):
    """The cache's rows as 32-bit values, [B, Hkv, width * block, D]."""
    B, width = tables.shape
    N, Hkv, block = cache.shape[:3]
    at = tables.clamp(min=0).long()
    x = _decode(cache[at], scales.view(torch.uint8)[at].view(E4M3), None if heads is None else heads[:, None])
    return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, width * block, -1)


def _plain_attend(s):
    q, tables, starts, totals = s["q"], s["tables"], s["starts"].long(), s["totals"].long()
    T, Hq, D = q.shape
    Hkv, B, n = s["k_cache"].shape[1], tables.shape[0], s["most_new"]
    k = _plain_rows(s["k_cache"], s["k_scales"], s["k_heads"], tables)
    v = _plain_rows(s["v_cache"], s["v_scales"], s["v_heads"], tables)
    S, i = k.shape[2], torch.arange(n, device=q.device)
    news = starts[1:] - starts[:-1]
    row = (starts[:-1, None] + i).clamp(max=T - 1)  # [B, n]
    qb = q[row].float().reshape(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    x = torch.matmul(qb, k.transpose(2, 3)).mul_(1.0 / math.sqrt(D)).reshape(B, Hq, n, S)
    if s["softcap"] > 0:
        x = torch.tanh(x / s["softcap"]) * s["softcap"]
    j = torch.arange(S, device=q.device)
    pos = totals[:, None] - news[:, None] + i  # the row's own position
    seen = j < totals[:, None, None]
    if s["causal"]:
        seen = seen & (j <= pos[..., None])
    if s["window"] > 0:
        seen = seen & (j > pos[..., None] - s["window"])
    x = x.masked_fill_(~seen[:, None], -math.inf)
    m = x.amax(3, keepdim=True)
    p = torch.exp(x.sub_(torch.where(m == -math.inf, 0.0, m)))
    total = p.sum(3, keepdim=True)
    p = p.div_(torch.where(total > 0, total, 1.0))
    v = torch.where((j < totals[:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(p.reshape(B, Hkv, -1, S), v).reshape(B, Hq, n, D).transpose(1, 2)
    # back to packed rows; rows behind the last request stay as they are
    t = torch.arange(T, device=q.device)
    b = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    there = b < B
    b = b.clamp(max=B - 1)
    o = o[b, (t - starts[b]).clamp(0, n - 1)].to(q.dtype)
    return torch.where(there[:, None, None], o, s["out"])


def _own(s):
    import tiled_online_softmax_02_gb300 as attn
    if s["op"] == "rope":
        return attn.attn_rope(s["q"], s["k"], s["freq"], positions=s["positions"], q_starts=s["starts"],
                              total_lengths=s["totals"], layout=s["layout"], inverse=s["inverse"], scale=s["scale"])
    cache = (s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"])
    heads = dict(k_head_scales=s["k_heads"], v_head_scales=s["v_heads"])
    if s["op"] == "append":
        attn.attn_cache_append_fp4(s["k"], s["v"], s["slots"], *cache, **heads)
        return (*attn.attn_cache_read_fp4(*cache, s["slots"], dtype=s["k"].dtype, **heads), s["k_scales"],
                s["v_scales"])
    if s["op"] == "read":
        return attn.attn_cache_read_fp4(*cache, s["slots"], dtype=s["dtype"], **heads)
    return attn.attn_fwd_paged_fp4(s["q"], *cache, s["tables"], s["starts"], s["totals"], causal=s["causal"],
                                   local_window=s["window"], softcap=s["softcap"], out=s["out"], **heads)


def run(s):
    if own:
        return _own(s)
    return {"rope": _plain_rope, "append": _plain_append, "read": _plain_read, "attend": _plain_attend}[s["op"]](s)


# ---------------------------------------------------------------- what it takes
def work(case):
    past = (case.get("past_min", 0) + case["past_max"]) / 2
    new = (case.get("new_min", 0) + case.get("new_max", 0)) / 2
    B, D, Hkv = case["B"], case["D"], case["Hkv"]
    esize = 4 if case["dtype"] == "f32" else 2
    held = D / 2 + D / GROUP  # bytes of a row in the cache
    if case["op"] == "rope":
        rows = B * new * (case["Hq"] + Hkv)
        return dict(bytes=2 * rows * D * esize + 4 * B * new, flops=3 * rows * case["rotary"])
    if case["op"] == "append":  # rows in, into the cache, and out again
        rows = 2 * B * new * Hkv
        return dict(bytes=rows * (2 * D * esize + held) + 8 * B * new, flops=4 * rows * D)
    if case["op"] == "read":
        rows = 2 * B * past * Hkv
        return dict(bytes=rows * (D * esize + held) + 8 * B * past, flops=rows * D)
    # keys that a row sees, on average, and cache rows that some row of the request sees
    seen, rows = past + (new + 1) / 2 if case["causal"] else past + new, past + new
    if case["window"] > 0:
        seen, rows = min(seen, case["window"]), min(rows, case["window"] + new)
    T = B * new
    return dict(bytes=2 * B * rows * Hkv * held + 2 * T * case["Hq"] * D * esize, flops=4 * T * seen * case["Hq"] * D)


# ------------------------------------------------------------------- 64 bits
def _two_to_64(e):
    """2^e for whole e, as 64-bit values, by its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _small_float_64(x, mantissa, least, most):
    """The nearest value with so many mantissa bits, ties to even, subnormal below 2^least, at most `most` in size."""
    a = x.abs().clamp(max=most)
    _, e = torch.frexp(torch.where(a > 0, a, 1.0))
    step = _two_to_64((e - 1).clamp(min=least) - mantissa)
    return torch.round(a / step) * step * torch.sign(x)


def _held_64(x, heads):
    """(values, scales) that the cache holds for rows [T, Hkv, D]."""
    g = x.double().reshape(*x.shape[:2], -1, GROUP)
    h = torch.ones(x.shape[1], dtype=torch.float64, device=x.device) if heads is None else heads.double()
    h = h[None, :, None]
    scale = _small_float_64(g.abs().amax(-1) / 6.0 / h, 3, -6, 448.0).clamp(min=2.0 ** -9)
    unit = (scale * h)[..., None]
    return (_small_float_64(g / unit, 1, 0, 6.0) * unit).reshape(x.shape), scale


def _values_64(code, scales, heads):
    """64-bit rows of bytes [..., D/2] and scales [..., D/16], by the bits of the codes."""
    n = torch.stack([code % 16, code // 16], -1).flatten(-2).long()
    size, sign = n % 8, 1.0 - 2.0 * (n // 8).double()
    e, m = size // 2, (size % 2).double()
    x = sign * torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * _two_to_64(e - 1))
    x = x * scales.view(torch.uint8).view(E4M3).float().double().repeat_interleave(GROUP, -1)
    return x if heads is None else x * heads.double()[..., None]


def _exact_rope(s):
    f = s["freq"].cpu().numpy().astype(np.longdouble)
    if s["positions"] is not None:
        pos = s["positions"].cpu().numpy()
    else:
        starts, totals = s["starts"].tolist(), s["totals"].tolist()
        pos = np.concatenate([np.arange(t - (z - a), t) for a, z, t in zip(starts, starts[1:], totals)])
    turn = 2 * np.longdouble("3.14159265358979323846264338327950288")
    angle = (pos[:, None].astype(np.longdouble) * f) % turn
    w = s["scale"] * np.exp((-1j if s["inverse"] else 1j) * angle.astype(np.float64))
    w = torch.from_numpy(w).to(s["q"].device)[:, None]
    made, R = [], 2 * len(f)
    for x in (s["q"], s["k"]):
        y = x.double().clone()
        z = torch.complex(y[..., :R // 2], y[..., R // 2:R]) if s["layout"] == "half" else \
            torch.view_as_complex(y[..., :R].reshape(*y.shape[:2], -1, 2).contiguous())
        z = z * w
        y[..., :R] = torch.cat([z.real, z.imag], -1) if s["layout"] == "half" else torch.view_as_real(z).flatten(-2)
        made.append(y)
    return tuple(made)


def _exact_append(s):
    held, after = [], []
    for x, scales, heads in ((s["k"], s["k_scales"], s["k_heads"]), (s["v"], s["v_scales"], s["v_heads"])):
        values, scale = _held_64(x, heads)
        all_scales = scales.float().double()
        all_scales[s["slots"] // s["block"], :, s["slots"] % s["block"]] = scale
        held.append(values)
        after.append(all_scales)
    return (*held, *after)


def _exact_read(s):
    made = []
    for cache, scales, heads in ((s["k_cache"], s["k_scales"], s["k_heads"]),
                                 (s["v_cache"], s["v_scales"], s["v_heads"])):
        x = torch.zeros((len(s["slots"]), cache.shape[1], 2 * cache.shape[3]), dtype=torch.float64,
                        device=cache.device)
        at = torch.nonzero(s["slots"] >= 0)[:, 0]
        b, o = s["slots"][at] // s["block"], s["slots"][at] % s["block"]
        x[at] = _values_64(cache[b, :, o], scales.view(torch.uint8)[b, :, o], heads)
        made.append(x)
    return tuple(made)


def _exact_attend(s):
    q, starts, totals = s["q"].double(), s["starts"].tolist(), s["totals"].tolist()
    Hq, D = q.shape[1:]
    Hkv, block = s["k_cache"].shape[1:3]
    out = s["out"].double()
    tables = s["tables"].long()
    for b in range(len(totals)):
        a, z, L = starts[b], starts[b + 1], totals[b]
        if z == a:
            continue
        ids = tables[b, :-(-L // block)]
        kb, vb = (_values_64(s[c][ids].transpose(1, 2), s[g].view(torch.uint8)[ids].transpose(1, 2), s[h])
                  for c, g, h in (("k_cache", "k_scales", "k_heads"), ("v_cache", "v_scales", "v_heads")))
        at = torch.arange(L - (z - a), L, device=q.device)[:, None]
        key = torch.arange(L, device=q.device)[None]
        hide = torch.zeros((z - a, L), dtype=torch.bool, device=q.device)
        if s["causal"]:
            hide |= key > at
        if s["window"] > 0:
            hide |= key <= at - s["window"]
        for h in range(Hq):
            g = h // (Hq // Hkv)
            kh, vh = kb[:, :, g].reshape(-1, D)[:L], vb[:, :, g].reshape(-1, D)[:L]
            score = (q[a:z, h] @ kh.T) / math.sqrt(D)
            if s["softcap"] > 0:
                score = s["softcap"] * torch.tanh(score / s["softcap"])
            score[hide] = -math.inf
            out[a:z, h] = torch.nan_to_num(torch.softmax(score, 1), nan=0.0) @ vh
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "read": _exact_read, "attend": _exact_attend}[s["op"]](s)
