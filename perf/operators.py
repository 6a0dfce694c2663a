"""Timed cases of the serving-step operators around a shared prefix: block
assignment (kvq_assign_blocks), block release (kvq_release_blocks) and decode
attention over a prefix that several sequences share (kvq_prefix_decode).

`own` false computes each operator from elementary torch operations in FP32;
`own` true calls the library.  `exact` restates each operator from its
definition in 64 bits, one sequence at a time.
"""
import math
import random

import numpy as np
import torch

own = False

BS = 16                                   # tokens per cache block
QMAX = {"int8": 127, "int8c": 127, "int4": 7, "int2": 1, "int2c": 1, "fp8": 448}
BITS = {"int8": 8, "int8c": 8, "fp8": 8, "int4": 4, "int2": 2, "int2c": 2}
DTYPE = {"int8": "int8", "int8c": "int8", "fp8": "fp8_e4m3fn", "int4": "int4", "int2": "int2", "int2c": "int2"}
OUTLIER_CHANNELS = (3, 17, 64, 100)       # K channels of the long-context workloads, x20
SIGNS = (0x9E3779B9, 0x7F4A7C15, 0xF39CC060, 0x5CEDC834)  # rotation signs, one bit a channel


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _prefix(name, batch, hq, hkv, d, k, v, prefix, suffix, groups=1, loose=0, rot=False, tail=False, short=False):
    return dict(name=name, op="prefix", batch=batch, hq=hq, hkv=hkv, d=d, k=k, v=v, prefix=prefix, suffix=suffix,
                groups=groups, loose=loose, rot=rot, tail=tail, short=short)


def _pool(name, op, rows, ctx, new, shared=0):
    return dict(name=name, op=op, rows=rows, ctx=ctx, new=new, shared=shared)


def listed():
    return [
        # two requests of a test-sized layer behind one short system prompt: all latency
        _prefix("prefix_tiny_int8", 2, 4, 2, 64, "int8", "int8", 64, 36),
        # an 8B layer, one long document, 27 questions about it
        _prefix("prefix_8b_fp8", 27, 32, 8, 128, "fp8", "fp8", 32003, 1000),
        # a 70B layer, KIVI cache with its full-precision tail, few requests: reading bounds it
        _prefix("prefix_70b_kivi", 8, 64, 8, 128, "int8c", "int4", 65536, 70, tail=True),
        # continuous batching: four system prompts, some rows idle or shorter than the prompt, some without one
        _prefix("prefix_mix_int8", 256, 32, 8, 128, "int8", "int8", 4099, 500, groups=4, loose=16, short=True),
        # long context, mixed precision, 64 samples of one prompt
        _prefix("prefix_long_mixed", 64, 32, 8, 128, "fp8", "int4", 32768, 100),
        # rotated INT4
        _prefix("prefix_8b_int4_rot", 27, 32, 8, 128, "int4", "int4", 32768, 300, rot=True),
        # 2-bit KIVI, many samples of one long prompt: arithmetic bounds it
        _prefix("prefix_70b_kivi2", 100, 64, 8, 128, "int2c", "int2", 65536, 33),
        # a decode step of 256 requests: one token each, every 16th needs a block
        _pool("assign_decode", "assign", 256, 16384, 1),
        # 64 prompts prefilled in one step
        _pool("assign_prefill", "assign", 64, 0, 4097),
        # drafted tokens that the verification rejects: assigned, then given back
        _pool("cycle_draft", "cycle", 256, 16384, 7),
        # 64 requests admitted behind a cached prompt of 2048 blocks, and evicted
        _pool("cycle_admit", "cycle", 64, 0, 300, shared=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "prefix", "assign", "cycle"])
    if op != "prefix":
        shared = _log(rng, 1, 1024) if op == "cycle" and rng.random() < 0.5 else 0
        return dict(op=op, rows=_log(rng, 2, 512), ctx=0 if shared else _log(rng, 1, 8192), new=_log(rng, 1, 500),
                    shared=shared)
    d = rng.choice([64, 128, 128, 128])
    k = rng.choice(["int8", "fp8", "int4", "int8c"] + ["int2c"] * (d == 128))
    v = rng.choice(["int8", "fp8", "int4"] + ["int2"] * (d == 128))
    hkv = rng.choice([1, 2, 3, 4, 7, 8, 8, 8])
    batch = _log(rng, 2, 256)
    groups = min(batch // 2, rng.choice([1, 1, 2, 3, 5]))
    case = dict(op="prefix", batch=batch, hq=hkv * rng.randint(1, 8), hkv=hkv, d=d, k=k, v=v,
                prefix=_log(rng, 16, 65536), suffix=_log(rng, 1, 1000), groups=groups,
                loose=rng.choice([0, 0, min(3, batch - 2 * groups)]), rot=k in ("int8", "fp8", "int4") and rng.random() < 0.2,
                tail=k in ("int8c", "int2c") and rng.random() < 0.5, short=batch > 4 and rng.random() < 0.3)
    while work(case)["flops"] > 2e11:
        case["prefix"] = case["prefix"] * 2 // 3
    return case


def _lengths(case):
    """Shared lengths of the groups, the groups' first sequences (and the end) and the contexts, from the case alone."""
    b, ng = case["batch"], case["groups"]
    grouped = b - case["loose"]
    starts = [grouped * g // ng for g in range(ng + 1)]
    prefixes = [max(BS, case["prefix"] * (ng - g) // ng) for g in range(ng)]
    ctx = [(s * 7919 + 13) % (case["suffix"] + 1) for s in range(b)]
    for g in range(ng):
        for s in range(starts[g], starts[g + 1]):
            ctx[s] += prefixes[g]
    if case["short"]:
        ctx[starts[1] - 1] = prefixes[0] // 3  # a request that is still inside the prompt
        ctx[0] = 0                             # a padded row, first of its group
    return prefixes, starts, ctx


def _token_bytes(case):
    d = case["d"]
    side = lambda f, per_token: d * BITS[f] / 8 + (d * 4 / BS if f.endswith("c") else per_token)  # noqa: E731
    return case["hkv"] * (side(case["k"], 4) + side(case["v"], 4 * (d // 32) if case["v"] in ("int4", "int2") else 4))


def _pool_sizes(case):
    c = [case["ctx"] + (7 * r) % BS if case["ctx"] else 0 for r in range(case["rows"])]
    n = [case["new"] if case["new"] == 1 else 1 + (case["new"] * (r + 1) // 3 + 11 * r) % case["new"] for r in range(case["rows"])]
    return c, n


def work(case):
    if case["op"] == "prefix":
        prefixes, starts, ctx = _lengths(case)
        shared = [0] * case["batch"]
        read = 0
        for g, p in enumerate(prefixes):
            longest = max(ctx[starts[g]:starts[g + 1]])
            whole = min(p, longest) // BS * BS
            read += whole
            for s in range(starts[g], starts[g + 1]):
                shared[s] = whole
        read += sum(max(0, c - w) for c, w in zip(ctx, shared))
        return {"bytes": read * _token_bytes(case) + case["batch"] * case["hq"] * case["d"] * 4,
                "flops": 4.0 * case["d"] * case["hq"] * sum(ctx)}
    c, n = _pool_sizes(case)
    base = case["shared"] * BS
    c = [base] * len(c) if case["shared"] else c
    blocks = sum(-(-(x + y) // BS) - -(-x // BS) for x, y in zip(c, n))
    taken = blocks + case["shared"] * len(c)
    total = len(c) * 16 + sum(n) * 12 + blocks * 12 + case["shared"] * len(c) * 12
    return {"bytes": float(total + (taken * 16 + len(c) * 12 if case["op"] == "cycle" else 0)), "flops": 0.0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _quantize(x, fmt):
    """x [blocks, 16, heads, d] -> (codes uint8, scales FP32) of the cache layout."""
    nb, bs, h, d = x.shape
    if fmt.endswith("c"):
        amax = x.abs().amax(1)                                         # [blocks, heads, d]
        s = amax / QMAX[fmt]
        full = s[:, None]
    elif fmt in ("int4", "int2") and _quantize.grouped:
        amax = x.view(nb, bs, h, d // 32, 32).abs().amax(-1)
        s = amax / QMAX[fmt]
        full = s.repeat_interleave(32, -1)
    else:
        s = x.abs().amax(-1) / QMAX[fmt]
        full = s[..., None]
    y = x / torch.where(full > 0, full, torch.ones_like(full))
    if fmt == "fp8":
        return y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s.contiguous()
    q = y.round().clamp(-QMAX[fmt], QMAX[fmt]).to(torch.int32)
    bits = BITS[fmt]
    per = 8 // bits
    q = (q & ((1 << bits) - 1)).view(nb, bs, h, d // per, per)
    shift = torch.arange(per, device=x.device, dtype=torch.int32) * bits
    return (q << shift).sum(-1).to(torch.uint8), s.contiguous()


_quantize.grouped = False


def _signs(d, device):
    c = torch.arange(d, device=device)
    words = torch.tensor(SIGNS, device=device, dtype=torch.int64)
    return 1.0 - 2.0 * ((words[c // 32] >> (c % 32)) & 1).double()


def _hadamard(d, device):
    i = torch.arange(d, device=device)
    x = i[:, None] & i[None, :]
    for s in (4, 2, 1):
        x = x ^ (x >> s)
    return 1.0 - 2.0 * (x & 1).double()


def _prepare_prefix(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    prefixes, starts, ctx = _lengths(case)
    b, h, d = case["batch"], case["hkv"], case["d"]
    group_of = [-1] * b
    for g in range(case["groups"]):
        for s in range(starts[g], starts[g + 1]):
            group_of[s] = g
    shared = [p // BS for p in prefixes]
    first, count = [], 0
    for g in range(case["groups"]):
        first.append(count)
        count += shared[g]
    heads = sum(shared)
    table = np.full((b, max(1, max(-(-c // BS) for c in ctx))), -1, np.int64)
    for s in range(b):
        n, g = -(-ctx[s] // BS), group_of[s]
        k = min(shared[g], n) if g >= 0 else 0
        if k:
            table[s, :k] = np.arange(first[g], first[g] + k)
        table[s, k:n] = np.arange(count, count + n - k)
        count += n - k
    nb = count + 3
    perm = torch.randperm(nb, generator=gen, device=dev)
    logical = torch.from_numpy(table).to(dev)
    tables = torch.where(logical >= 0, perm[logical.clamp(min=0)], logical).to(torch.int32).contiguous()
    cache = {}
    for w in ("k", "v"):
        fmt = case[w]
        _quantize.grouped = w == "v"
        codes, scales = [], []
        for lo in range(0, nb, 2048):
            n = min(2048, nb - lo)
            x = torch.randn((n, BS, h, d), generator=gen, device=dev)
            if w == "k":
                x[..., [c for c in OUTLIER_CHANNELS if c < d]] *= 20
            if lo == 0 and heads:
                x[0, :4] *= 10                       # the first tokens of the first prompt
            x = x.to(torch.bfloat16).float()
            if case["rot"]:
                x = (x * _signs(d, dev).float()) @ _hadamard(d, dev).float()
            c, s = _quantize(x, fmt)
            codes.append(c)
            scales.append(s)
        at = torch.argsort(perm)
        cache[w + "_cache"] = torch.cat(codes)[at].contiguous()
        cache[w + "_scale"] = torch.cat(scales)[at].contiguous()
    res = None
    if case["tail"]:
        res = {w: torch.randn((b, BS, h, d), generator=gen, device=dev).to(torch.bfloat16) for w in ("k", "v")}
    gran = lambda f, v: "block_channel" if f.endswith("c") else "token_group" if v and f in ("int4", "int2") else "token_head"  # noqa: E731
    fmt = dict(k_dtype=DTYPE[case["k"]], v_dtype=DTYPE[case["v"]], k_gran=gran(case["k"], False),
               v_gran=gran(case["v"], True), num_kv_heads=h, head_dim=d, num_blocks=nb,
               v_group=32 if case["v"] in ("int4", "int2") else 0, rotation_signs=SIGNS if case["rot"] else None)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    return dict(case=case, fmt=fmt, cache=cache, tables=tables, ctx=i32(ctx), max_ctx=max(ctx), starts=i32(starts),
                prefixes=i32(prefixes), max_prefix=max(prefixes), residual=res,
                most=max(starts[g + 1] - starts[g] for g in range(case["groups"])),
                q=torch.randn((b, case["hq"], d), generator=gen, device=dev).to(torch.bfloat16))


def _prepare_pool(case, seed):
    dev = "cuda"
    c, n = _pool_sizes(case)
    rows, shared = len(c), case["shared"]
    held = [-(-x // BS) for x in c]
    grown = [-(-(x + shared * BS + y) // BS) for x, y in zip(c, n)]
    extra = 1 if shared else 0               # the row that keeps the cached prompt
    width = max(grown)
    nb = sum(grown) - shared * rows + shared + 37
    order = torch.randperm(nb, generator=torch.Generator(device=dev).manual_seed(seed), device=dev).to(torch.int32)
    table = np.full((rows + extra, width), -1, np.int64)
    used = 0
    for r in range(rows):
        table[r, :held[r]] = np.arange(used, used + held[r])
        used += held[r]
    if shared:
        table[rows, :shared] = np.arange(used, used + shared)
        used += shared
        c, n = c + [shared * BS], n + [0]
    logical = torch.from_numpy(table).to(dev)
    tables = torch.where(logical >= 0, order[logical.clamp(min=0)].long(), logical).to(torch.int32).contiguous()
    refs = torch.zeros(nb, dtype=torch.int32, device=dev)
    refs[order[:used].long()] = 1
    free = torch.zeros(nb, dtype=torch.int32, device=dev)
    free[:nb - used] = order[used:]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    start = i32(c + [nb - used])             # contexts and the pool's free count, restored by one copy
    live = start.clone()
    st = dict(case=case, tables=tables, start=start, live=live, ctx=live[:-1], new=i32(n), capacity=sum(n) + 5,
              pool=dict(free_list=free, free_count=live[-1:], ref_counts=refs), blocks=sum(grown),
              prefix_rows=None, prefix_blocks=None)
    if case["op"] == "cycle":
        st["keep"] = i32([0 if shared else x for x in c[:rows]] + [1 << 30] * extra)
    if shared:
        st["prefix_rows"] = i32([rows] * rows + [-1])
        st["prefix_blocks"] = i32([shared] * rows + [0])
    return st


def prepare(case, seed):
    with torch.no_grad():
        return _prepare_prefix(case, seed) if case["op"] == "prefix" else _prepare_pool(case, seed)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _values(cache, w, fmt, blocks):
    """Dequantized FP32 rows of the given physical blocks: [..., 16, heads, d]."""
    codes, scales = cache[w + "_cache"][blocks], cache[w + "_scale"][blocks]
    if fmt == "fp8":
        x = codes.view(torch.float8_e4m3fn).float()
    elif BITS[fmt] == 8:
        x = codes.view(torch.int8).float()
    else:
        bits = BITS[fmt]
        shift = torch.arange(8 // bits, device=codes.device, dtype=torch.uint8) * bits
        half = 1 << (bits - 1)
        x = ((codes[..., None] >> shift) & (2 * half - 1)).flatten(-2)
        x = (x ^ half).float() - half
    if fmt.endswith("c"):
        return x * scales.unsqueeze(-3)
    if scales.dim() == x.dim():
        return (x.unflatten(-1, (scales.shape[-1], -1)) * scales[..., None]).flatten(-2)
    return x * scales[..., None]


def _plain_prefix(st):
    case, cache, q = st["case"], st["cache"], st["q"].float()
    b, hq, d = q.shape
    h = case["hkv"]
    g = hq // h
    ng = case["groups"]
    if case["rot"]:
        turn = _hadamard(d, q.device).float() * _signs(d, q.device).float()[:, None]
        q = (q @ turn) / d
    q = q.view(b, h, g, d) / math.sqrt(d)
    ctx, starts = st["ctx"].long(), st["starts"].long()
    cached = ctx // BS * BS if case["tail"] else ctx
    # the groups' sequences, padded to the largest group
    seq = starts[:-1, None] + torch.arange(st["most"], device=q.device)
    member = seq < starts[1:, None]
    seq = seq.clamp(max=b - 1)
    longest = torch.where(member, ctx[seq], -1)
    lead = seq.gather(1, longest.argmax(1, keepdim=True))[:, 0]
    whole = torch.minimum(st["prefixes"].long(), longest.amax(1)) // BS * BS
    wide = st["max_prefix"] // BS
    width = st["tables"].shape[1]
    # prefix: every row of a group against the leader's blocks
    blocks = st["tables"][lead][:, :min(wide, width)].long().clamp(min=0)
    k = _values(cache, "k", case["k"], blocks).flatten(1, 2).permute(0, 2, 3, 1)       # [ng, h, d, t]
    v = _values(cache, "v", case["v"], blocks).flatten(1, 2).transpose(1, 2)           # [ng, h, t, d]
    rows = q[seq].permute(0, 2, 1, 3, 4).reshape(ng, h, -1, d)
    s = rows @ k
    limit = torch.minimum(cached[seq], whole[:, None])
    t = torch.arange(s.shape[-1], device=q.device)
    seen = (t < limit[..., None]).repeat_interleave(g, 1)[:, None]
    s.masked_fill_(~seen, -math.inf)
    m1 = s.amax(-1, keepdim=True)
    m1c = m1.clamp(min=-1e30)
    p = s.sub_(m1c).exp_()
    l1, o1 = p.sum(-1, keepdim=True), p @ v
    del s, p, k, v
    at = seq[member]
    back = lambda x: x.view(ng, h, -1, g, x.shape[-1]).permute(0, 2, 1, 3, 4)[member]  # noqa: E731
    m = torch.full((b, h, g, 1), -1e30, device=q.device)
    l = torch.zeros_like(m)
    o = torch.zeros((b, h, g, d), device=q.device)
    m[at], l[at], o[at] = back(m1c), back(l1), back(o1)
    # suffix: each sequence's own blocks, padded to the longest
    skip = torch.zeros(b, dtype=torch.long, device=q.device)
    skip[at] = whole[:, None].expand_as(seq)[member]
    most = max(1, -(-(case["suffix"] + 2 * BS) // BS))
    j = skip[:, None] // BS + torch.arange(most, device=q.device)
    blocks = st["tables"].long().gather(1, j.clamp(max=width - 1)).clamp(min=0)
    k = _values(cache, "k", case["k"], blocks).flatten(1, 2).transpose(1, 2)           # [b, h, t, d]
    v = _values(cache, "v", case["v"], blocks).flatten(1, 2).transpose(1, 2)
    pos = (j * BS)[..., None] + torch.arange(BS, device=q.device)
    seen = pos.flatten(1) < cached[:, None]
    if case["tail"]:
        k = torch.cat([k, st["residual"]["k"].float().transpose(1, 2)], 2)
        v = torch.cat([v, st["residual"]["v"].float().transpose(1, 2)], 2)
        seen = torch.cat([seen, torch.arange(BS, device=q.device) < (ctx % BS)[:, None]], 1)
    s = (q @ k.transpose(2, 3)).masked_fill_(~seen[:, None, None], -math.inf)
    both = torch.maximum(m, s.amax(-1, keepdim=True))
    keep = (m - both).exp()
    p = s.sub_(both).exp_()
    l = l * keep + p.sum(-1, keepdim=True)
    o = (o * keep + p @ v.masked_fill(~seen[:, None, :, None], 0.0)) / torch.where(l > 0, l, torch.ones_like(l))
    o = o.view(b, hq, d)
    if case["rot"]:
        o = (o @ turn.t()) / d
    return o.to(torch.bfloat16)


def _plain_assign(st):
    c, n, table, pool = st["ctx"].long(), st["new"].long(), st["tables"], st["pool"]
    rows, width = table.shape
    if st["prefix_rows"] is not None:
        src, k = st["prefix_rows"].long(), st["prefix_blocks"].long()
        mine = (torch.arange(width, device=c.device) < k[:, None]) & (src >= 0)[:, None]
        table.copy_(torch.where(mine, table[src.clamp(min=0)], table))
        pool["ref_counts"].scatter_add_(0, table.long().clamp(min=0).flatten(), mine.to(torch.int32).flatten())
        c = torch.where(src >= 0, k * BS, c)
    have, want = (c + BS - 1) // BS, (c + n + BS - 1) // BS
    free = pool["free_count"].long()
    ends = (want - have).cumsum(0)
    # new blocks, over a bound of their number
    i = torch.arange(st["blocks"], device=c.device)
    r = torch.searchsorted(ends, i, right=True)
    ok = r < rows
    r = r.clamp(max=rows - 1)
    col = have[r] + i - (ends - want + have)[r]
    block = pool["free_list"][(free - 1 - i).clamp(min=0)]
    spill = torch.cat([table.flatten(), table.new_zeros(1)])
    spill.scatter_(0, torch.where(ok, r * width + col, rows * width), block)
    table.copy_(spill[:-1].view(rows, width))
    refs = torch.cat([pool["ref_counts"], pool["ref_counts"].new_zeros(1)])
    refs.scatter_(0, torch.where(ok, block.long(), refs.numel() - 1), torch.ones_like(block))
    pool["ref_counts"].copy_(refs[:-1])
    # tokens
    offsets = torch.cat([n.new_zeros(1), n.cumsum(0)])
    t = torch.arange(st["capacity"], device=c.device)
    r = torch.searchsorted(offsets[1:], t, right=True)
    ok = r < rows
    r = r.clamp(max=rows - 1)
    pos = c[r] + t - offsets[r]
    slot = table.flatten()[(r * width + (pos // BS).clamp(max=width - 1))].long() * BS + pos % BS
    st["ctx"].copy_(c + n)
    pool["free_count"].sub_(ends[-1:].int())
    minus = torch.full_like(slot, -1)
    return offsets.int(), torch.where(ok, slot, minus), torch.where(ok, pos, minus).int()


def _plain_release(st):
    c, keep, table, pool = st["ctx"].long(), st["keep"].long(), st["tables"], st["pool"]
    rows, width = table.shape
    col = torch.arange(width, device=c.device)
    gone = (col >= ((keep + BS - 1) // BS)[:, None]) & (col < ((c + BS - 1) // BS)[:, None])
    block = torch.where(gone, table, 0).long().flatten()
    gone = gone.flatten()
    refs = pool["ref_counts"]
    refs.scatter_add_(0, block, -gone.to(torch.int32))
    i = torch.arange(block.numel(), device=c.device)
    far = block.numel()
    first = torch.full((refs.numel(),), far, device=c.device).scatter_reduce_(0, block, torch.where(gone, i, far), "amin")
    push = gone & (refs[block] == 0) & (first[block] == i)
    ends = push.cumsum(0)
    free = pool["free_count"].long()
    nb = refs.numel()
    stack = torch.cat([pool["free_list"], pool["free_list"].new_zeros(1)])
    stack.scatter_(0, torch.where(push, free + ends[-1] - ends, nb), block.int())
    pool["free_list"].copy_(stack[:-1])
    pool["free_count"].add_(ends[-1:].int())
    table.masked_fill_(gone.view(rows, width), -1)
    st["ctx"].copy_(torch.minimum(c, keep))


def run(state):
    case, pool = state["case"], state.get("pool")
    if own:
        import quantized_paged_kv_write_gb300 as kvq
    if case["op"] == "prefix":
        if own:
            return kvq.kvq_prefix_decode(state["q"], kvq.CacheFormat(**state["fmt"]), state["cache"], state["tables"],
                                         state["ctx"], state["max_ctx"], state["starts"], state["prefixes"],
                                         state["max_prefix"], residual=state["residual"])
        return _plain_prefix(state)
    if case["op"] == "assign":               # a step's lengths come from the request list
        state["live"].copy_(state["start"])
    if own:
        out = kvq.kvq_assign_blocks(state["new"], state["ctx"], state["tables"], pool, state["capacity"],
                                    prefix_rows=state["prefix_rows"], prefix_blocks=state["prefix_blocks"])
    else:
        out = _plain_assign(state)
    if case["op"] == "cycle":
        if own:
            kvq.kvq_release_blocks(state["keep"], state["ctx"], state["tables"], pool)
        else:
            _plain_release(state)
    return dict(offsets=out[0], slots=out[1], positions=out[2], contexts=state["ctx"], tables=state["tables"], **pool)


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_rows(st, w, table, n):
    """Dequantized float64 rows of positions [0, n) of one sequence: [n, heads, d]."""
    fmt, ids = st["case"][w], table[: -(-n // BS)].long()
    codes, s = st["cache"][w + "_cache"][ids], st["cache"][w + "_scale"][ids].double()
    nb, bs, h, _ = codes.shape
    d = st["case"]["d"]
    if fmt == "fp8":
        e, f = ((codes >> 3) & 15).double(), (codes & 7).double()
        x = torch.where(e > 0, (1 + f / 8) * torch.exp2(e - 7), f / 8 * 2.0 ** -6) * (1 - 2 * (codes >> 7).double())
    elif BITS[fmt] == 8:
        x = codes.double() - 256.0 * (codes > 127).double()
    else:
        per, top = 8 // BITS[fmt], 1 << BITS[fmt]
        parts = [torch.div(codes.int(), top ** i, rounding_mode="floor") % top for i in range(per)]
        x = torch.stack(parts, -1).reshape(nb, bs, h, d).double()
        x = x - top * (x >= top // 2).double()
    if fmt.endswith("c"):
        x = x * s[:, None]
    elif s.dim() == 4:
        x = x * s.repeat_interleave(32, -1)
    else:
        x = x * s[..., None]
    return x.reshape(nb * bs, h, d)[:n]


def _exact_prefix(st):
    case = st["case"]
    d, h = case["d"], case["hkv"]
    out = torch.zeros((case["batch"], case["hq"], d), dtype=torch.float64, device="cuda")
    for s, n in enumerate(st["ctx"].tolist()):
        if n == 0:
            continue
        part = n // BS * BS if case["tail"] else n
        k, v = (_exact_rows(st, w, st["tables"][s], part) for w in ("k", "v"))
        if case["tail"]:
            k, v = (torch.cat([x, st["residual"][w][s, : n - part].double()]) for x, w in ((k, "k"), (v, "v")))
        q = st["q"][s].double()
        if case["rot"]:
            q = (q * _signs(d, "cuda")) @ _hadamard(d, "cuda") / d
        z = torch.einsum("hgd,thd->hgt", q.view(h, -1, d), k) / math.sqrt(d)
        o = torch.einsum("hgt,thd->hgd", torch.softmax(z, -1), v).reshape(-1, d)
        out[s] = (o @ _hadamard(d, "cuda")) * _signs(d, "cuda") / d if case["rot"] else o
    return out


def _exact_pool(st):
    case = st["case"]
    c, n, table = st["start"][:-1].tolist(), st["new"].tolist(), st["tables"].tolist()
    free = st["pool"]["free_list"].tolist()
    refs, count = st["pool"]["ref_counts"].tolist(), int(st["start"][-1])
    offsets, slots, positions = [0], [], []
    for r in range(len(c)):
        if st["prefix_rows"] is not None and int(st["prefix_rows"][r]) >= 0:
            src, k = int(st["prefix_rows"][r]), int(st["prefix_blocks"][r])
            for i in range(k):
                table[r][i] = table[src][i]
                refs[table[r][i]] += 1
            c[r] = k * BS
        for p in range(c[r], c[r] + n[r]):
            if p % BS == 0:
                count -= 1
                table[r][p // BS] = free[count]
                refs[free[count]] = 1
            slots.append(table[r][p // BS] * BS + p % BS)
            positions.append(p)
        c[r] += n[r]
        offsets.append(len(slots))
    if case["op"] == "cycle":
        keep = st["keep"].tolist()
        for r in reversed(range(len(c))):
            for i in reversed(range(-(-min(keep[r], c[r]) // BS), -(-c[r] // BS))):
                block, table[r][i] = table[r][i], -1
                refs[block] -= 1
                if refs[block] == 0:
                    free[count] = block
                    count += 1
            c[r] = min(c[r], keep[r])
    pad = [-1] * (st["capacity"] - len(slots))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return dict(offsets=i32(offsets), slots=torch.tensor(slots + pad), positions=i32(positions + pad), contexts=i32(c),
                tables=i32(table), free_list=i32(free), free_count=i32([count]), ref_counts=i32(refs))


def exact(case, seed):
    if case["op"] == "prefix" and sum(_lengths(case)[2]) * case["hkv"] * case["d"] > 1.2e10:
        return None
    st = prepare(case, seed)
    return _exact_prefix(st) if case["op"] == "prefix" else _exact_pool(st)


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(s)) for s in range(6)]:
        print(c, work(c))
