"""The paged 8-bit KV cache: what is measured of it, and the operators' plain forms.

Three operators serve one step of a batch of requests:
  assign   cache blocks for the step's new tokens, block tables, row starts
           and the slot of every new token, from the requests' lengths
  append   the new K / V rows into the cache as e4m3 with one power-of-two
           scale for each (block, kv head)
  attend   attention of the new tokens over the cache
`run` is one pass through one of them: the library's call where `own` is
true, elementary torch operations in 32 bits where it is false.  `exact` is
the definition again in 64 bits.
"""
import math

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
MIN_SCALE_LOG2 = -100  # the smallest scale a block gets (a block of zeros has it)
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one decode step of a full batch: a new token each, now and then a block, some requests just replaced
        dict(name="assign_decode", op="assign", B=64, width=128, block=64, new_max=1, past_max=8000, finished=0.05,
             tokens=64),
        # prompts admitted into half of a batch's rows, in a slot map padded for a captured graph
        dict(name="assign_prompts", op="assign", B=48, width=256, block=32, new_max=2048, past_max=6000, finished=0.5,
             tokens=65536),
        # the same decode step's K / V rows
        dict(name="append_decode", op="append", B=64, Hkv=8, D=128, block=64, dtype="bf16", new_max=1, past_max=8000,
             strided=False),
        # a ragged step, K and V as slices of a fused projection's output, small blocks
        dict(name="append_ragged", op="append", B=13, Hkv=4, D=64, block=16, dtype="f16", new_max=150, past_max=900,
             strided=True),
        # whole prompts
        dict(name="append_prompts", op="append", B=8, Hkv=8, D=128, block=64, dtype="bf16", new_max=4096, past_max=0,
             strided=True),
        # one request's next token: latency
        dict(name="decode_one", op="attend", B=1, Hq=32, Hkv=8, D=128, block=64, dtype="bf16", new_min=1, new_max=1,
             past_min=3000, past_max=4000, causal=True, window=0, softcap=0.0, pad=0),
        # few requests with long contexts (the decode workload of the benchmark, its cache in 8 bits)
        dict(name="decode_long", op="attend", B=8, Hq=32, Hkv=8, D=128, block=64, dtype="bf16", new_min=1, new_max=1,
             past_min=9000, past_max=32700, causal=True, window=0, softcap=0.0, pad=0),
        # a full batch, eight query heads to a kv head, small blocks
        dict(name="decode_batch", op="attend", B=64, Hq=32, Hkv=4, D=128, block=16, dtype="f16", new_min=1, new_max=1,
             past_min=100, past_max=8000, causal=True, window=0, softcap=0.0, pad=0),
        # a few drafted tokens to verify in each request, sliding window and soft-cap
        dict(name="verify_window", op="attend", B=19, Hq=16, Hkv=8, D=64, block=32, dtype="f16", new_min=1, new_max=5,
             past_min=0, past_max=8000, causal=True, window=1024, softcap=50.0, pad=0),
        # chunked prefill over ragged caches (the benchmark's ragged workload), its rows padded for a captured graph
        dict(name="chunk_ragged", op="attend", B=8, Hq=32, Hkv=4, D=128, block=64, dtype="f16", new_min=100,
             new_max=128, past_min=0, past_max=3900, causal=True, window=0, softcap=0.0, pad=107),
        # whole prompts of uneven length (the benchmark's causal prefill)
        dict(name="prompts", op="attend", B=2, Hq=32, Hkv=8, D=128, block=64, dtype="bf16", new_min=3500,
             new_max=4096, past_min=0, past_max=0, causal=True, window=0, softcap=0.0, pad=0),
        # a large chunk far into long contexts
        dict(name="chunk_long", op="attend", B=2, Hq=32, Hkv=8, D=128, block=128, dtype="bf16", new_min=1500,
             new_max=2048, past_min=9000, past_max=14000, causal=True, window=0, softcap=0.0, pad=0),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["assign", "append", "append", "attend", "attend", "attend", "attend"])
    block = rng.choice([16, 32, 64, 128])
    if op == "assign":
        B = _log_uniform(rng, 1, 300)
        new_max = rng.choice([1, _log_uniform(rng, 1, 2048)])
        past_max = _log_uniform(rng, 1, 8000)
        width = -(-(past_max + new_max) // block)
        tokens = min(B * new_max, 65536) + rng.choice([0, 17])
        return dict(op=op, B=B, width=width, block=block, new_max=new_max, past_max=past_max,
                    finished=rng.choice([0.0, 0.1, 0.5]), tokens=tokens)
    heads = rng.choice([(32, 8), (32, 4), (16, 8), (8, 8), (15, 3), (12, 1)])
    base = dict(op=op, Hkv=heads[1], D=rng.choice([64, 128]), block=block, dtype=rng.choice(["bf16", "f16"]))
    if op == "append":
        B = _log_uniform(rng, 1, 100)
        return dict(base, B=B, new_max=rng.choice([1, 5, _log_uniform(rng, 1, 24000 // B)]),
                    past_max=_log_uniform(rng, 1, 4000), strided=rng.random() < 0.5)
    kind = rng.choice(["decode", "decode", "verify", "chunk"])
    if kind == "chunk":
        B = _log_uniform(rng, 1, 8)
        new_max = _log_uniform(rng, 16, 2048 // B)
        past_max = _log_uniform(rng, 1, 8000)
    else:
        B = _log_uniform(rng, 1, 64)
        new_max = 1 if kind == "decode" else rng.randint(2, 7)
        past_max = _log_uniform(rng, 10, min(32000, 500000 // B))
    return dict(base, B=B, Hq=heads[0], new_min=0 if B > 3 else 1, new_max=new_max, past_min=0, past_max=past_max,
                causal=rng.random() < 0.85, window=rng.choice([0, 0, 100, 1024]),
                softcap=rng.choice([0.0, 0.0, 30.0]), pad=rng.choice([1, 1, 9]))


# ------------------------------------------------------------------- inputs
def _spread(lo, hi, n):
    """n whole numbers spread evenly over lo .. hi, both ends among them where n allows."""
    return np.clip(np.rint(lo - 0.49 + (hi - lo + 0.98) * (np.arange(n) + 0.5) / n), lo, hi).astype(np.int32)


def _lengths(case, seed):
    """(past, new) of the requests, int32 numpy: even spreads, in an order that the seed gives."""
    rng = np.random.Generator(np.random.PCG64([int(seed), 11]))
    B = case["B"]
    past = rng.permutation(_spread(case.get("past_min", 0), case["past_max"], B))
    new = rng.permutation(_spread(_least_new(case), case["new_max"], B))
    return past, new, rng


def _least_new(case):
    return 1 if case["new_max"] == 1 else case.get("new_min", 1 if case["op"] == "append" else 0)


def _exclusive(x):
    return np.concatenate([[0], np.cumsum(x)]).astype(np.int64)


def _tables(past, new, block, rng, width):
    """Block tables over a scattered pool, as an allocator in use leaves them: (tables [B, width], num_blocks)."""
    held = -(-(past.astype(np.int64) + new) // block)
    num_blocks = int((-(-past.astype(np.int64) // block) - (-new.astype(np.int64) // block)).sum()) + 3
    pool, at = rng.permutation(num_blocks).astype(np.int32), _exclusive(held)
    tables = np.full((len(held), width), -1, np.int32)
    for b, n in enumerate(held):
        tables[b, :n] = pool[at[b]:at[b] + n]
    return tables, num_blocks


def _width(case):
    return -(-(case["past_max"] + case["new_max"]) // case["block"])


def _cache(num_blocks, Hkv, block, D, gen, dev):
    """An e4m3 cache of N(0, 1) rows with uneven channels, and its power-of-two scales."""
    gain = torch.exp(0.3 * torch.randn((1, Hkv, 1, D), generator=gen, device=dev))
    x = torch.randn((num_blocks, Hkv, block, D), generator=gen, device=dev).mul_(gain)
    scale = _pow2_scale(x.abs().amax((2, 3)))
    return (x / scale[:, :, None, None]).to(E4M3), scale


def _prepare_assign(case, seed):
    past, new, rng = _lengths(case, seed)
    B, width, block = case["B"], case["width"], case["block"]
    finished = rng.random(B) < case["finished"]
    tables, _ = _tables(past, np.zeros_like(new), block, rng, width)
    num_blocks = int((tables >= 0).sum() + (-(-new.astype(np.int64) // block) + 1).sum())
    new[_exclusive(new)[1:] > case["tokens"]] = 0  # admission stops where the slot map ends
    order = rng.permutation(num_blocks).astype(np.int32)
    tables = np.where(tables >= 0, order[np.maximum(tables, 0) % num_blocks], -1)
    taken = np.zeros(num_blocks, bool)
    taken[tables[tables >= 0]] = True
    free = np.flatnonzero(~taken).astype(np.int32)
    rng.shuffle(free)
    stack = np.full(num_blocks, -1, np.int32)
    stack[:len(free)] = free
    gpu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    return dict(op="assign", past=gpu(past), new=gpu(new), tables=gpu(tables.astype(np.int32)), free=gpu(stack),
                count=gpu(np.array([len(free)], np.int32)), finished=gpu(finished), block=block,
                tokens=case["tokens"])


def _slots(tables, past, new, block):
    at = [p + np.arange(n) for p, n in zip(past, new)]
    return np.concatenate([tables[b][pos // block].astype(np.int64) * block + pos % block
                           for b, pos in enumerate(at)] or [np.zeros(0, np.int64)])


def _prepare_append(case, seed):
    past, new, rng = _lengths(case, seed)
    Hkv, D, block = case["Hkv"], case["D"], case["block"]
    tables, num_blocks = _tables(past, new, block, rng, _width(case))
    slots = _slots(tables, past, new, block)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    kc, ks = _cache(num_blocks, Hkv, block, D, gen, dev)
    vc, vs = _cache(num_blocks, Hkv, block, D, gen, dev)
    T, wide = len(slots), 3 if case["strided"] else 1
    dt = DTYPES[case["dtype"]]
    # rows of a fused projection: ever larger ones now and then, so that some scales grow
    k, v = ((torch.randn((T, wide * Hkv, D), generator=gen, device=dev)
             * torch.exp(0.5 * torch.randn((T, 1, 1), generator=gen, device=dev))).to(dt)[:, :Hkv] for _ in range(2))
    return dict(op="append", k=k, v=v, slots=torch.from_numpy(slots).to(dev), k_cache=kc, v_cache=vc, k_scales=ks,
                v_scales=vs, block=block, most_blocks=min(T, case["B"] * (-(-(case["new_max"] - 1) // block) + 1)))


def _prepare_attend(case, seed):
    past, new, rng = _lengths(case, seed)
    Hq, Hkv, D, block = case["Hq"], case["Hkv"], case["D"], case["block"]
    tables, num_blocks = _tables(past, new, block, rng, _width(case))
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    kc, ks = _cache(num_blocks, Hkv, block, D, gen, dev)
    vc, vs = _cache(num_blocks, Hkv, block, D, gen, dev)
    starts = _exclusive(new).astype(np.int32)
    T = int(starts[-1]) + case["pad"]
    dt = DTYPES[case["dtype"]]
    return dict(op="attend", q=torch.randn((T, Hq, D), generator=gen, device=dev).to(dt), k_cache=kc, v_cache=vc,
                k_scales=ks, v_scales=vs, tables=torch.from_numpy(tables).to(dev),
                starts=torch.from_numpy(starts).to(dev),
                totals=torch.from_numpy((past + new).astype(np.int32)).to(dev),
                out=torch.zeros((T, Hq, D), dtype=dt, device=dev), most_new=max(1, int(new.max())), block=block,
                causal=case["causal"], window=case["window"], softcap=case["softcap"])


def prepare(case, seed):
    return {"assign": _prepare_assign, "append": _prepare_append, "attend": _prepare_attend}[case["op"]](case, seed)


# -------------------------------------------------------------- plain forms
def _plain_assign(s):
    past, new, tables, free, block = s["past"].long(), s["new"].long(), s["tables"], s["free"], s["block"]
    B, width = tables.shape
    N, T, dev = free.shape[0], s["tokens"], tables.device
    fin = s["finished"]
    cols = torch.arange(width, device=dev)
    count0 = s["count"][0].long()
    # finished rows give their blocks back, in row order, onto the stack
    given = fin[:, None] & (tables >= 0)
    nth = torch.cumsum(given.reshape(-1), 0).reshape(B, width) - 1
    stack = torch.cat([free, free.new_zeros(1)])
    stack.index_put_((torch.where(given, count0 + nth, N),), tables)
    stack = stack[:N]
    count1 = count0 + given.sum()
    past = torch.where(fin, 0, past)
    held = torch.where(fin[:, None], -1, tables)
    # every entry that a row needs and lacks takes the block on top of the stack, in row order
    need = (past + new + block - 1) // block
    lacks = (cols[None] < need[:, None]) & (held < 0)
    nth = torch.cumsum(lacks.reshape(-1), 0).reshape(B, width) - 1
    taken = stack[(count1 - 1 - nth).clamp(0, N - 1)]
    total = lacks.sum()
    starts = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    bad = torch.where((past < 0).any() | (new < 0).any(), 4, 0)
    bad = torch.where((bad == 0) & (need > width).any(), 2, bad)
    bad = torch.where((bad == 0) & (starts[-1] > T), 3, bad)
    bad = torch.where((bad == 0) & (total > count1), 1, bad)
    fine = bad == 0
    tables.copy_(torch.where(fine, torch.where(lacks, taken, held), tables))
    free.copy_(torch.where(fine, stack, free))
    s["count"].copy_(torch.where(fine, count1 - total, count0)[None])
    starts = torch.where(fine, starts, 0)
    totals = torch.where(fine, past + new, s["past"].long())
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(starts[1:].contiguous(), t, right=True).clamp(max=B - 1)
    pos = (past[b] + t - starts[b]).clamp(0, width * block - 1)
    slot = tables[b, pos // block].long() * block + pos % block
    slot = torch.where(t < starts[-1], slot, -1)
    return starts.int(), totals.int(), slot, bad.int()[None]


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s, from 2^-100 on."""
    m, e = torch.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
    e = torch.where(amax > 0, torch.where(m <= 0.875, e - 9, e - 8), MIN_SCALE_LOG2).clamp(min=MIN_SCALE_LOG2)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)  # 2^e by its bits: a power function rounds


def _plain_append_one(x, slots, cache, scales, block, most):
    x = x.float()
    T, blk, off = x.shape[0], slots // block, slots % block
    # the tokens that begin a block's run, in order; places left over repeat the first
    begins = torch.cat([blk.new_ones(1, dtype=torch.bool), blk[1:] != blk[:-1]])
    nth = torch.cumsum(begins, 0) - 1
    token = torch.zeros(most + 1, dtype=torch.int64, device=x.device)
    token.index_put_((torch.where(begins, nth, most),), torch.arange(T, device=x.device))
    token = token[:most]
    b, first = blk[token], off[token]
    # per (run, head): the scale for the largest new value, and for the block's earlier rows
    amax = torch.zeros((most, x.shape[1]), device=x.device)
    amax.index_reduce_(0, nth, x.abs().amax(2), "amax")
    amax = torch.where((torch.arange(most, device=x.device) <= nth[-1])[:, None], amax, amax[:1])
    old = scales[b]
    grown = torch.maximum(torch.where((first > 0)[:, None], old, 0), _pow2_scale(amax))
    # earlier rows are encoded again where their block's scale grew
    row = torch.arange(block, device=x.device)
    again = ((row < first[:, None])[:, None] & (grown > old)[:, :, None])[..., None]
    held = cache.view(torch.uint8)[b].view(E4M3).float()
    held = torch.where(again, held * old[:, :, None, None] / grown[:, :, None, None], held)
    cache.view(torch.uint8)[b] = held.to(E4M3).view(torch.uint8)
    scales[b] = grown
    cache.view(torch.uint8)[blk, :, off] = (x / grown[nth][:, :, None]).clamp(-448, 448).to(E4M3).view(torch.uint8)


def _plain_append(s):
    _plain_append_one(s["k"], s["slots"], s["k_cache"], s["k_scales"], s["block"], s["most_blocks"])
    _plain_append_one(s["v"], s["slots"], s["v_cache"], s["v_scales"], s["block"], s["most_blocks"])
    return s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]


def _plain_rows(cache, scales, tables):
    """The cache's rows as 32-bit values, [B, Hkv, width * block, D]."""
    N, Hkv, block, D = cache.shape
    B, width = tables.shape
    at = tables.clamp(min=0).long()
    x = cache.view(torch.uint8)[at].view(E4M3).float() * scales[at][..., None, None]  # [B, width, Hkv, block, D]
    return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, width * block, D)


def _plain_attend(s):
    q, tables, starts, totals = s["q"], s["tables"], s["starts"].long(), s["totals"].long()
    T, Hq, D = q.shape
    Hkv, B, n = s["k_cache"].shape[1], tables.shape[0], s["most_new"]
    k = _plain_rows(s["k_cache"], s["k_scales"], tables)
    v = _plain_rows(s["v_cache"], s["v_scales"], tables)
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


def run(s):
    if own:
        import tiled_online_softmax_02_gb300 as attn
        if s["op"] == "assign":
            made = attn.attn_cache_assign(s["past"], s["new"], s["tables"], s["free"], s["count"],
                                          block_size=s["block"], num_tokens=s["tokens"], finished=s["finished"])
            return made + (s["tables"], s["free"], s["count"])
        if s["op"] == "append":
            attn.attn_cache_append_fp8(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scales"],
                                       s["v_scales"])
            return s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]
        return attn.attn_fwd_paged_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["tables"],
                                       s["starts"], s["totals"], causal=s["causal"], local_window=s["window"],
                                       softcap=s["softcap"], out=s["out"])
    if s["op"] == "assign":
        return _plain_assign(s) + (s["tables"], s["free"], s["count"])
    if s["op"] == "append":
        return _plain_append(s)
    return _plain_attend(s)


# ---------------------------------------------------------------- what it takes
def _expected(case):
    past = (case.get("past_min", 0) + case["past_max"]) / 2
    new = (_least_new(case) + case["new_max"]) / 2
    return past, new


def work(case):
    past, new = _expected(case)
    B = case["B"]
    if case["op"] == "assign":
        # lengths in, row starts and totals out, the rows' table entries, a slot for each token
        entries = B * (past + new) / case["block"]
        return dict(bytes=17 * B + 4 * entries + 8 * case["tokens"], flops=0)
    esize, D, Hkv = 2, case["D"], case["Hkv"]
    if case["op"] == "append":
        T = B * new
        return dict(bytes=2 * T * Hkv * D * (esize + 1) + 8 * T, flops=4 * T * Hkv * D)
    # keys that a row sees, on average, and cache rows that some row of the request sees
    before = past + (new + 1) / 2 if case["causal"] else past + new
    seen, rows = before, past + new
    if case["window"] > 0:
        seen, rows = min(seen, case["window"]), min(rows, case["window"] + new)
    T = B * new
    return dict(bytes=2 * B * rows * Hkv * D + 2 * T * case["Hq"] * D * esize,
                flops=4 * T * seen * case["Hq"] * D)


# ------------------------------------------------------------------- 64 bits
def _two_to_64(e):
    """2^e for whole e, as 64-bit values, by its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3_64(x):
    """The e4m3 value nearest to x, ties to even, at most 448 in size (64-bit values)."""
    a = x.abs().clamp(max=448.0)
    _, e = torch.frexp(torch.where(a > 0, a, 1.0))
    step = _two_to_64((e - 1).clamp(min=-6) - 3)
    return torch.round(a / step) * step * torch.sign(x)


def _exact_append(s):
    got = []
    for x, cache, scales in ((s["k"], s["k_cache"], s["k_scales"]), (s["v"], s["v_cache"], s["v_scales"])):
        x, c, sc = x.double(), cache.float().double(), scales.double()
        slots = s["slots"].cpu().numpy()
        blk = slots // s["block"]
        edge = np.flatnonzero(np.diff(blk, prepend=-1, append=-1))  # runs of tokens of one block
        for a, z in zip(edge[:-1], edge[1:]):
            b, o = int(blk[a]), int(slots[a] % s["block"])
            rows = x[a:z]
            top = rows.abs().amax((0, 2))
            e = torch.ceil(torch.log2(top / 448.0)).clamp(min=-100.0)
            e = torch.where(top <= 448.0 * _two_to_64(e - 1), e - 1, e)  # a logarithm next to a whole number
            e = torch.where(top > 448.0 * _two_to_64(e), e + 1, e).clamp(min=-100.0)
            new = torch.maximum(_two_to_64(e), sc[b] if o > 0 else torch.zeros_like(top))
            if o > 0:
                c[b, :, :o] = _e4m3_64(c[b, :, :o] * (sc[b] / new)[:, None, None])
            c[b, :, o:o + z - a] = _e4m3_64(rows / new[:, None]).transpose(0, 1)
            sc[b] = new
        got.append((c, sc))
    return got[0][0], got[1][0], got[0][1], got[1][1]


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
        kb = s["k_cache"].view(torch.uint8)[ids].view(E4M3).float().double() * s["k_scales"][ids].double()[..., None, None]
        vb = s["v_cache"].view(torch.uint8)[ids].view(E4M3).float().double() * s["v_scales"][ids].double()[..., None, None]
        at = torch.arange(L - (z - a), L, device=q.device)[:, None]
        key = torch.arange(L, device=q.device)[None]
        hide = torch.zeros((z - a, L), dtype=torch.bool, device=q.device)
        if s["causal"]:
            hide |= key > at
        if s["window"] > 0:
            hide |= key <= at - s["window"]
        for h in range(Hq):
            g = h // (Hq // Hkv)
            kh, vh = kb[:, g].reshape(-1, D)[:L], vb[:, g].reshape(-1, D)[:L]
            score = (q[a:z, h] @ kh.T) / math.sqrt(D)
            if s["softcap"] > 0:
                score = s["softcap"] * torch.tanh(score / s["softcap"])
            score[hide] = -math.inf
            out[a:z, h] = torch.nan_to_num(torch.softmax(score, 1), nan=0.0) @ vh
    return out


def exact(case, seed):
    if case["op"] == "assign":
        return None  # whole numbers only
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)
