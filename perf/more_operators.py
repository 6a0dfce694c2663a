"""Timed cases of what a serving step does before and after its decode: causal
attention over packed prompts (kvq_prompt_attention), a decode that adds up how
much attention each cached token gets (kvq_weigh_decode), and eviction of the
tokens that got least (kvq_evict_tokens).

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
QMAX = {"int8": 127, "int4": 7, "fp8": 448}
BITS = {"int8": 8, "fp8": 8, "int4": 4}
DTYPE = {"int8": "int8", "int4": "int4", "fp8": "fp8_e4m3fn"}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _prompt(name, hq, hkv, d, seqs, longest, fixed=False, fused=False, pad=0):
    return dict(name=name, op="prompt", hq=hq, hkv=hkv, d=d, seqs=seqs, longest=longest, fixed=fixed, fused=fused, pad=pad)


def _weigh(name, batch, hq, hkv, d, k, v, ctx, fixed=False):
    return dict(name=name, op="weigh", batch=batch, hq=hq, hkv=hkv, d=d, k=k, v=v, ctx=ctx, fixed=fixed)


def _evict(name, batch, hkv, d, k, v, ctx, keep, recent, pinned=0, fixed=False):
    return dict(name=name, op="evict", batch=batch, hkv=hkv, d=d, k=k, v=v, ctx=ctx, keep=keep, recent=recent,
                pinned=pinned, fixed=fixed)


def listed():
    return [
        # two requests of a test-sized layer: all latency
        _prompt("prompt_tiny", 4, 2, 64, 2, 100, pad=3),
        # an 8B layer, a step that admits requests of many lengths, Q, K and V as parts of one projection
        _prompt("prompt_8b_mix", 32, 8, 128, 23, 2049, fused=True, pad=11),
        # an 8B layer, one long document
        _prompt("prompt_8b_long", 32, 8, 128, 1, 16384, fixed=True),
        # a 70B layer, a few requests
        _prompt("prompt_70b", 64, 8, 128, 4, 4097),
        # head dimension 64, three query heads a kv head
        _prompt("prompt_d64", 24, 8, 64, 3, 5003),
        # two requests of a test-sized layer
        _weigh("weigh_tiny_int8", 2, 4, 2, 64, "int8", "int8", 100),
        # an 8B layer at the long-context batch
        _weigh("weigh_8b_fp8", 27, 32, 8, 128, "fp8", "fp8", 32768, fixed=True),
        # a 70B layer's heads, mixed precision, requests of all lengths
        _weigh("weigh_70b_mixed", 33, 64, 8, 128, "int8", "int4", 16384),
        # two requests of a test-sized layer, down to a few tokens
        _evict("evict_tiny_int8", 2, 2, 64, "int8", "int8", 100, 32, 8, 2),
        # an 8B layer: the long-context batch cut to half
        _evict("evict_8b_fp8", 27, 8, 128, "fp8", "fp8", 32768, 16384, 512, 4, fixed=True),
        # a budget that is held: every request is a few blocks over it
        _evict("evict_steady_int8", 256, 8, 128, "int8", "int8", 4160, 4096, 256, 4),
        # long documents in 4 bits cut to an eighth behind their prompt
        _evict("evict_8b_int4", 8, 8, 128, "int4", "int4", 65536, 8192, 1024, 1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "weigh", "evict"])
    d = rng.choice([64, 128, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 7, 8, 8, 8])
    fixed = rng.random() < 0.25
    if op == "prompt":
        case = dict(op=op, hq=hkv * rng.randint(1, 8), hkv=hkv, d=d, seqs=_log(rng, 1, 64), longest=_log(rng, 1, 16384),
                    fixed=fixed, fused=rng.random() < 0.4, pad=rng.choice([0, 1, 7, 130]))
        while work(case)["flops"] > 1.2e12 or sum(_lengths(case)) > 65536 or case["seqs"] * case["hq"] * case["longest"] ** 2 > 8e9:
            case["longest"] = max(1, case["longest"] * 2 // 3)
            case["seqs"] = max(1, case["seqs"] * 4 // 5)
        return case
    k, v = rng.choice(["int8", "fp8", "int4"]), rng.choice(["int8", "fp8", "int4"])
    case = dict(op=op, batch=_log(rng, 1, 256), hkv=hkv, d=d, k=k, v=v, ctx=_log(rng, 1, 65536), fixed=fixed)
    while case["batch"] * case["ctx"] * hkv * d > 6e8:
        case["ctx"] = case["ctx"] * 2 // 3
    if op == "weigh":
        return dict(case, hq=hkv * rng.randint(1, 8))
    keep = max(1, int(case["ctx"] * rng.choice([0.1, 0.5, 0.9, 0.98])))
    return dict(case, keep=keep, recent=rng.choice([0, 1, keep // 9, keep // 2]), pinned=rng.choice([0, 4, keep // 5]))


def _lengths(case):
    """Tokens of each sequence, from the case alone."""
    n, most = case.get("seqs", case.get("batch")), case.get("longest", case.get("ctx"))
    if case["fixed"]:
        return [most] * n
    if case["op"] == "evict" and case["keep"] * 20 > most * 19:
        got = [max(0, most - (5 * r) % (most - case["keep"] + 9)) for r in range(n)]   # all near the budget
    else:
        got = [most - (r * 7919 * most // 10007 + r) % most for r in range(n)]
    if n > 2 and case["op"] != "prompt":
        got[1] = 0                                          # a padded row
    return got


def _row_bytes(case):
    """Bytes of one token's codes and scales, K and V."""
    return case["hkv"] * (case["d"] * (BITS[case["k"]] + BITS[case["v"]]) // 8 + 4 + 4 * _groups(case))


def _groups(case):
    return case["d"] // 32 if case["v"] == "int4" else 1


def work(case):
    n = _lengths(case)
    if case["op"] == "prompt":
        return {"bytes": 4.0 * sum(n) * (case["hq"] + case["hkv"]) * case["d"] + 4.0 * sum(n) * case["hq"],
                "flops": 2.0 * case["d"] * case["hq"] * sum(x * (x + 1) for x in n)}
    if case["op"] == "weigh":
        return {"bytes": float(sum(n) * (_row_bytes(case) + 8 * case["hkv"]) + case["batch"] * case["hq"] * case["d"] * 6),
                "flops": 4.0 * case["d"] * case["hq"] * sum(n)}
    # weights of every token read; half of what is kept past the kept places' share moves, as do the last ones
    total = 0.0
    for x in n:
        k = case["keep"]
        if x <= k:
            continue
        w = min(case["recent"], k)
        p = min(case["pinned"], k - w)
        old, free = x - w - p, k - w - p
        moved = free * (old - free) / old + w    # expected, for weights in no order
        total += 4.0 * case["hkv"] * (x + (x - k)) + 2.0 * moved * (_row_bytes(case) + 4 * case["hkv"])
    return {"bytes": total + 12.0 * len(n), "flops": 0.0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _prepare_prompt(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    n = _lengths(case)
    total, hq, h, d = sum(n) + case["pad"], case["hq"], case["hkv"], case["d"]
    make = lambda heads: torch.randn((total, heads, d), generator=gen, device=dev).to(torch.bfloat16)  # noqa: E731
    if case["fused"]:
        q, k, v = make(hq + 2 * h).split((hq, h, h), 1)     # parts of one projection's output
    else:
        q, k, v = make(hq), make(h), make(h)
    if case["pad"]:                                         # rows behind the last sequence hold anything
        for x in (q, k, v):
            x[sum(n):] = math.nan
    return dict(case=case, q=q, k=k, v=v, longest=max(n),
                offsets=torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=dev),
                out=torch.zeros((total, hq, d), dtype=torch.bfloat16, device=dev),
                lse=torch.zeros((total, hq), dtype=torch.float32, device=dev))


def _codes(case, w, nb, gen):
    """Codes and scales of nb blocks, as a quantizer of normal values leaves them."""
    fmt, h, d, dev = case[w], case["hkv"], case["d"], "cuda"
    groups = _groups(case) if w == "v" else 1
    codes, scales = [], []
    for lo in range(0, nb, 4096):
        x = torch.randn((min(4096, nb - lo), BS, h, groups, d // groups), generator=gen, device=dev).to(torch.bfloat16).float()
        s = x.abs().amax(-1, keepdim=True) / QMAX[fmt]
        y = (x / s).flatten(-2)
        scales.append(s[..., 0] if groups > 1 else s[..., 0, 0])
        if fmt == "fp8":
            codes.append(y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        elif fmt == "int8":
            codes.append(y.round().to(torch.int8).view(torch.uint8))
        else:
            z = y.round().to(torch.int32).view(*y.shape[:-1], d // 2, 2) & 15
            codes.append((z[..., 0] | z[..., 1] << 4).to(torch.uint8))
    return torch.cat(codes), torch.cat(scales).contiguous()


def _prepare_cache(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    n = _lengths(case)
    held = [-(-x // BS) for x in n]
    nb = sum(held) + 3
    order = torch.randperm(nb - 1, generator=gen, device=dev)   # (block nb - 1 is in no table)
    table = np.full((len(n), max(held)), -1, np.int64)
    used = 0
    for r, x in enumerate(held):
        table[r, :x] = np.arange(used, used + x)
        used += x
    logical = torch.from_numpy(table).to(dev)
    st = dict(case=case, tables=torch.where(logical >= 0, order[logical.clamp(min=0)], logical).to(torch.int32).contiguous(),
              ctx=torch.tensor(n, dtype=torch.int32, device=dev), longest=max(n), cache={})
    for w in ("k", "v"):
        st["cache"][w + "_cache"], st["cache"][w + "_scale"] = _codes(case, w, nb, gen)
    st["fmt"] = dict(k_dtype=DTYPE[case["k"]], v_dtype=DTYPE[case["v"]], k_gran="token_head",
                     v_gran="token_group" if case["v"] == "int4" else "token_head", num_kv_heads=case["hkv"],
                     head_dim=case["d"], num_blocks=nb, v_group=32 if case["v"] == "int4" else 0)
    shape = (len(n), case["hkv"], max(held) * BS)
    if case["op"] == "weigh":
        st["weights"] = torch.rand(shape, generator=gen, device=dev)
        st["q"] = torch.randn((len(n), case["hq"], case["d"]), generator=gen, device=dev).to(torch.bfloat16)
        return st
    # sums of weights: few large ones, many small ones, some that nothing ever attended to
    w = torch.rand(shape, generator=gen, device=dev)
    st["start"] = torch.where(w < 0.05, 0.0, w ** 9)
    st["weights"] = st["start"].clone()
    i32 = lambda x: torch.full((len(n),), x, dtype=torch.int32, device=dev)  # noqa: E731
    st["keep"], st["recent"], st["pinned"] = i32(case["keep"]), i32(case["recent"]), i32(case["pinned"])
    refs = torch.zeros(nb, dtype=torch.int32, device=dev)
    refs[order[:used]] = 1
    free = torch.zeros(nb, dtype=torch.int32, device=dev)
    free[:nb - 1 - used] = order[used:].to(torch.int32)
    st["pool"] = dict(free_list=free, free_count=torch.tensor([nb - 1 - used], dtype=torch.int32, device=dev), ref_counts=refs)
    return st


def prepare(case, seed):
    with torch.no_grad():
        return _prepare_prompt(case, seed) if case["op"] == "prompt" else _prepare_cache(case, seed)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_prompt(st):
    """All sequences padded to the longest."""
    h, longest, dev = st["case"]["hkv"], st["longest"], st["q"].device
    n = st["offsets"].diff()
    t = torch.arange(longest, device=dev)
    inside = t < n[:, None]
    rows = torch.where(inside, st["offsets"][:-1, None] + t, 0).long()
    q = st["q"][rows].float()
    seqs, _, hq, d = q.shape
    g = hq // h
    q = q.view(seqs, longest, h, g, d).permute(0, 2, 3, 1, 4).reshape(seqs, h, g * longest, d)
    k = st["k"][rows].float().permute(0, 2, 3, 1)
    v = torch.where(inside[..., None, None], st["v"][rows].float(), 0.0).transpose(1, 2)
    s = (q @ k).mul_(1 / math.sqrt(d)).view(seqs, h, g, longest, longest)
    s.masked_fill_(t > t[:, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    s.sub_(m).exp_()
    l = s.sum(-1, keepdim=True)
    o = (s.view(seqs, h, g * longest, longest) @ v).view(seqs, h, g, longest, d) / l
    lse = (m + l.log())[..., 0]
    at = torch.where(inside, st["offsets"][:-1, None] + t, st["q"].shape[0]).flatten().long()   # past the end: a row to spare
    for name, x in (("out", o.permute(0, 3, 1, 2, 4).reshape(-1, hq, d)), ("lse", lse.permute(0, 3, 1, 2).reshape(-1, hq))):
        y = torch.cat([st[name], st[name][:1]])
        y[at] = x.to(y.dtype)
        st[name].copy_(y[:-1])
    return st["out"], st["lse"]


def _values(cache, w, fmt, blocks):
    """Dequantized FP32 rows of the given physical blocks: [..., 16, heads, d]."""
    codes, scales = cache[w + "_cache"][blocks], cache[w + "_scale"][blocks]
    if fmt == "fp8":
        x = codes.view(torch.float8_e4m3fn).float()
    elif fmt == "int8":
        x = codes.view(torch.int8).float()
    else:
        x = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
        x = (x ^ 8).float() - 8
    if scales.dim() == x.dim():
        return (x.unflatten(-1, (scales.shape[-1], -1)) * scales[..., None]).flatten(-2)
    return x * scales[..., None]


def _plain_weigh(st):
    case, cache, q = st["case"], st["cache"], st["q"].float()
    b, hq, d = q.shape
    h = case["hkv"]
    blocks = st["tables"].long().clamp(min=0)
    k = _values(cache, "k", case["k"], blocks).flatten(1, 2).permute(0, 2, 3, 1)      # [b, h, d, t]
    s = (q.view(b, h, hq // h, d) / math.sqrt(d)) @ k
    del k
    seen = torch.arange(s.shape[-1], device=q.device) < st["ctx"][:, None]
    s.masked_fill_(~seen[:, None, None], -math.inf)
    s.sub_(s.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    l = s.sum(-1, keepdim=True)
    p = s.div_(torch.where(l > 0, l, torch.ones_like(l)))
    v = _values(cache, "v", case["v"], blocks).flatten(1, 2).transpose(1, 2)          # [b, h, t, d]
    out = (p @ v.masked_fill_(~seen[:, None, :, None], 0.0)).view(b, hq, d)
    st["weights"].add_(p.sum(2))
    return out, st["weights"]


def _plain_evict(st):
    n, k = st["ctx"].long()[:, None, None], st["keep"].long()[:, None, None]
    weights, tables = st["weights"], st["tables"].long()
    rows, h, length = weights.shape
    pos = torch.arange(length, device=n.device).expand(rows, h, length)
    w = torch.minimum(st["recent"].long()[:, None, None], k)
    p = torch.minimum(st["pinned"].long()[:, None, None], k - w)
    over = n > k
    # the heaviest of [p, n - w), ties to the lower position
    open_ = (pos >= p) & (pos < n - w)
    order = torch.where(open_, weights, -math.inf).sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(open_).scatter_(2, order, pos < k - w - p)
    # freed places below k - w, in order, for the kept ones past it
    hole = (pos >= p) & (pos < k - w) & ~kept
    late = kept & (pos >= k - w)
    places = torch.full((rows, h, length + 1), length, device=n.device)
    places.scatter_(2, torch.where(hole, hole.cumsum(2) - 1, length), pos)
    source = torch.arange(length + 1, device=n.device).repeat(rows, h, 1)
    to = places.gather(2, (late.cumsum(2) - 1).clamp(min=0))
    source.scatter_(2, torch.where(late, to, length), pos)
    last = (pos >= k - w) & (pos < k)
    source = torch.where(last, pos + (n - k), source[..., :length])
    source = torch.where(over & (pos < k), source, pos)
    moved = torch.where(over & (pos >= k) & (pos < n), 0.0, weights.gather(2, source))
    weights.copy_(torch.where(pos < n, moved, weights))
    # the rows of codes and scales; places past a row's end repeat its first one, an empty row the spare block
    at = torch.where(pos < n, pos, 0)
    source = source.gather(2, at)
    spare = st["cache"]["k_cache"].shape[0] - 1
    block = torch.where(tables >= 0, tables, spare)[:, None].expand(rows, h, -1)
    slot = lambda x: block.gather(2, x // BS) * BS + x % BS  # noqa: E731
    to, source = slot(at), slot(source)
    head = torch.arange(h, device=n.device)[:, None]
    for x in st["cache"].values():
        flat = x.view(-1, *x.shape[2:])
        flat[to, head] = flat[source, head]
    return torch.minimum(n, k)[:, 0, 0].int()


def run(state):
    case = state["case"]
    if own:
        import quantized_paged_kv_write_gb300 as kvq
    if case["op"] == "prompt":
        if own:
            kvq.kvq_prompt_attention(state["q"], state["k"], state["v"], state["offsets"], state["longest"],
                                     out=state["out"], lse=state["lse"])
            return state["out"], state["lse"]
        return _plain_prompt(state)
    if case["op"] == "weigh":
        if own:
            out = kvq.kvq_weigh_decode(state["q"], kvq.CacheFormat(**state["fmt"]), state["cache"], state["tables"],
                                       state["ctx"], state["longest"], state["weights"])
            return out, state["weights"]
        return _plain_weigh(state)
    state["weights"].copy_(state["start"])    # what the steps since the last eviction have added up
    if own:
        kept = kvq.kvq_evict_tokens(state["keep"], state["ctx"], state["tables"], kvq.CacheFormat(**state["fmt"]),
                                    state["cache"], state["weights"], recent_lens=state["recent"],
                                    pinned_lens=state["pinned"], pool=state["pool"])
    else:
        kept = _plain_evict(state)
    # (codes only move: their bytes say all)
    return dict(kept=kept, weights=state["weights"], **state["cache"])


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_prompt(st):
    hq, h, d = st["case"]["hq"], st["case"]["hkv"], st["case"]["d"]
    out, lse = st["out"].double(), st["lse"].double()
    ends = st["offsets"].tolist()
    for a, b in zip(ends, ends[1:]):
        k, v = (st[x][a:b].double().transpose(0, 1) for x in ("k", "v"))
        for lo in range(a, b, 1024):
            hi = min(b, lo + 1024)
            q = st["q"][lo:hi].double().view(hi - lo, h, hq // h, d)
            z = torch.einsum("thgd,hjd->hgtj", q, k[:, :hi - a]) / math.sqrt(d)
            ahead = torch.arange(hi - a, device="cuda") > torch.arange(lo - a, hi - a, device="cuda")[:, None]
            z[..., ahead] = -math.inf
            lse[lo:hi] = torch.logsumexp(z, -1).permute(2, 0, 1).reshape(hi - lo, hq)
            out[lo:hi] = torch.einsum("hgtj,hjd->thgd", torch.softmax(z, -1), v[:, :hi - a]).reshape(hi - lo, hq, d)
    return out, lse


def _exact_rows(st, w, table, n):
    """Dequantized float64 rows of positions [0, n) of one sequence: [n, heads, d]."""
    fmt, ids = st["case"][w], table[: -(-n // BS)].long()
    codes, s = st["cache"][w + "_cache"][ids], st["cache"][w + "_scale"][ids].double()
    nb, _, h, _ = codes.shape
    if fmt == "fp8":
        e, f = ((codes >> 3) & 15).double(), (codes & 7).double()
        x = torch.where(e > 0, (1 + f / 8) * torch.exp2(e - 7), f / 8 * 2.0 ** -6) * (1 - 2 * (codes >> 7).double())
    elif fmt == "int8":
        x = codes.double() - 256.0 * (codes > 127).double()
    else:
        x = torch.stack([codes % 16, codes // 16], -1).reshape(nb, BS, h, -1).double()
        x = x - 16 * (x >= 8).double()
    x = x * (s.repeat_interleave(32, -1) if s.dim() == 4 else s[..., None])
    return x.reshape(nb * BS, h, -1)[:n]


def _exact_weigh(st):
    case = st["case"]
    d, h = case["d"], case["hkv"]
    out = torch.zeros((case["batch"], case["hq"], d), dtype=torch.float64, device="cuda")
    weights = st["weights"].double()
    for s, n in enumerate(st["ctx"].tolist()):
        if n == 0:
            continue
        k, v = (_exact_rows(st, w, st["tables"][s], n) for w in ("k", "v"))
        p = torch.softmax(torch.einsum("hgd,thd->hgt", st["q"][s].double().view(h, -1, d), k) / math.sqrt(d), -1)
        out[s] = torch.einsum("hgt,thd->hgd", p, v).reshape(-1, d)
        weights[s, :, :n] += p.sum(1)
    return out, weights


def _exact_evict(st):
    weights, tables = st["start"].cpu().numpy().copy(), st["tables"].cpu().numpy()
    n, keep, recent, pinned = (st[x].tolist() for x in ("ctx", "keep", "recent", "pinned"))
    to, source, heads = [], [], []
    for r in range(len(n)):
        if n[r] <= keep[r]:
            continue
        w = min(recent[r], keep[r])
        p = min(pinned[r], keep[r] - w)
        end = keep[r] - w
        for h in range(weights.shape[1]):
            x = weights[r, h]
            best = p + np.argsort(-x[p:n[r] - w], kind="stable")[:end - p]
            late = np.sort(best[best >= end])
            places = np.setdiff1d(np.arange(p, end), best)
            a, b = (np.concatenate([y, np.arange(z, z + w)]) for y, z in ((places, end), (late, n[r] - w)))
            x[a] = x[b].copy()
            x[keep[r]:n[r]] = 0
            to.append(tables[r][a // BS].astype(np.int64) * BS + a % BS)
            source.append(tables[r][b // BS].astype(np.int64) * BS + b % BS)
            heads.append(np.full(len(a), h))
    got = dict(kept=np.minimum(n, keep).astype(np.int32), weights=weights.astype(np.float64))
    cat = lambda x: torch.from_numpy(np.concatenate(x + [np.zeros(0, np.int64)])).cuda()  # noqa: E731
    to, source, heads = cat(to), cat(source), cat(heads)
    for name, x in st["cache"].items():
        flat = x.view(-1, *x.shape[2:])
        flat[to, heads] = flat[source, heads]
        got[name] = x.double() if x.dtype == torch.float32 else x
    return got


def exact(case, seed):
    with torch.no_grad():
        return {"prompt": _exact_prompt, "weigh": _exact_weigh, "evict": _exact_evict}[case["op"]](prepare(case, seed))


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(s)) for s in range(12)]:
        print(c, work(c))
