"""kvq_prefix_decode against float64 attention over the whole contexts.

Tolerance.  A rounding is off by at most half a step: 2^-11 of the value in
f16, 2^-8 in BF16.  With A = sum_t p_t |v_t| (per channel, p the softmax) and
Z = max_t sum_c |q_c k_tc| / sqrt(d):
  output            2^-8 |out|
  probabilities and scaled V codes, one rounding each: 2^-11 A + 2^-11 A
  scaled K codes (one rounding) and rotated queries move a score by at most
                    2^-11 Z each; a softmax whose scores move by e moves its
                    output by at most (e^(2 e) - 1) A
  f16 subnormals    an absolute 2^-25: of a probability that is at least 2^8 at
                    the row's largest, and of V codes that are at least 2^4 at
                    the largest (scales of 2^4 and more, codes of 1 and more):
                    less than 2^-28 of the largest |v| per token
  FP32 sums         2^-17 A for up to a few thousand terms
With the rotation, errors are taken in the rotated basis and the worst of
them is summed over the d channels by the way back, (1/d) sum_c.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import workloads as wl
from tests import _helpers as H

pytestmark = pytest.mark.gpu

kvq = None


@pytest.fixture(scope="module", autouse=True)
def _lib():
    global kvq
    from quantized_paged_kv_write_gb300 import build
    build.build()
    import quantized_paged_kv_write_gb300 as m
    m.load_library()
    kvq = m
    yield


INT8 = wl.CacheFormat(wl.INT8, wl.PER_TOKEN_HEAD)
FP8 = wl.CacheFormat(wl.FP8, wl.PER_TOKEN_HEAD)
INT4T = wl.CacheFormat(wl.INT4, wl.PER_TOKEN_HEAD)
INT8C = wl.CacheFormat(wl.INT8, wl.PER_BLOCK_CHANNEL)
INT2C = wl.CacheFormat(wl.INT2, wl.PER_BLOCK_CHANNEL)
INT4G = wl.CacheFormat(wl.INT4, wl.PER_TOKEN_GROUP, 32)
INT2G = wl.CacheFormat(wl.INT2, wl.PER_TOKEN_GROUP, 32)
KS = {"int8": INT8, "fp8": FP8, "int4": INT4T, "int8c": INT8C, "int2c": INT2C}
VS = {"int8": INT8, "fp8": FP8, "int4g": INT4G, "int2g": INT2G}
WORDS = (0x12345678, 0x9ABCDEF0, 0x0F1E2D3C, 0x4B5A6978)


class Batch:
    """groups: [(prefix_len, [context, ...])]; `loose`: contexts of sequences
    in no group.  Prefix blocks are shared physically; unused positions and
    blocks hold NaN codes and scales."""

    def __init__(self, k="fp8", v="fp8", hq=8, hkv=2, d=128, groups=(), loose=(), rot=False, tail=False, seed=0,
                 outliers=True, v_spread=1.0):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.hq, self.hkv, self.d, self.tail = hq, hkv, d, tail
        self.ctx = np.array([c for _, cs in groups for c in cs] + list(loose), dtype=np.int64)
        b = len(self.ctx)
        self.starts = np.cumsum([0] + [len(cs) for _, cs in groups])
        self.prefix = np.array([p for p, _ in groups], dtype=np.int64)
        cached = self.ctx // 16 * 16 if tail else self.ctx
        rows, width, used = [], int(max(1, (-(-cached // 16)).max(initial=0))), 0
        s = 0
        for p, cs in list(groups) + [(0, [c]) for c in loose]:
            shared = p // 16
            own = list(range(used, used + shared))
            used += shared
            for _ in cs:
                n = -(-int(cached[s]) // 16)
                row = own[:min(n, shared)]
                row += list(range(used, used + n - len(row)))
                used += max(0, n - shared)
                rows.append(row)
                s += 1
        nb = used + 3
        perm = rng.permutation(nb)
        self.table = np.full((b, width), -1, np.int32)
        for s, row in enumerate(rows):
            self.table[s, :len(row)] = perm[row]
        self.fmt = kvq.cache_format(KS[k], VS[v], hkv, d, nb, rotation_signs=WORDS if rot else None)
        self.cache = kvq.allocate_cache(self.fmt)
        for w in ("k", "v"):
            self.cache[w + "_cache"].fill_(0x7F)
            self.cache[w + "_scale"].fill_(float("nan"))
        # every block's tokens that some sequence holds, one write per block row
        slots = sorted({int(self.table[s, t // 16]) * 16 + t % 16 for s in range(b) for t in range(int(cached[s]))})
        x = {}
        for w in ("k", "v"):
            y = torch.randn((len(slots), hkv, d), generator=gen, device="cuda")
            if outliers and w == "k":
                y[..., [3, 17]] *= 8
            if outliers and len(slots):
                y[:2] *= 6
            if w == "v" and v_spread != 1.0:
                y *= v_spread ** torch.rand((len(slots), 1, 1), generator=gen, device="cuda")
            x[w] = y.to(torch.bfloat16)
        if slots:
            kvq.kvq_quantize_write(x["k"], x["v"], torch.tensor(slots, dtype=torch.int64, device="cuda"), self.fmt,
                                   self.cache)
        self.res = None
        if tail:
            self.res = {w: torch.randn((b, 16, hkv, d), generator=gen, device="cuda").to(torch.bfloat16) for w in "kv"}
            for s in range(b):
                for w in "kv":
                    self.res[w][s, int(self.ctx[s]) % 16:] = float("nan")
        self.q = torch.randn((b, hq, d), generator=gen, device="cuda").to(torch.bfloat16)
        self.oc = oracle.OracleCache(nb, 16, hkv, d, KS[k], VS[v],
                                     rotation_signs=oracle.signs_from_words(WORDS, d) if rot else None)
        torch.cuda.synchronize()
        for w in ("k", "v"):
            self.oc.codes[w] = self.cache[w + "_cache"].cpu().numpy()
            self.oc.scales[w] = self.cache[w + "_scale"].cpu().numpy()

    def args(self, ctx=None, starts=None, prefix=None, table=None):
        i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
        prefix = self.prefix if prefix is None else np.asarray(prefix)
        ctx = self.ctx if ctx is None else np.asarray(ctx)
        return (self.q, self.fmt, self.cache, i32(self.table if table is None else table), i32(ctx),
                int(max(ctx.max(initial=0), 0)), i32(self.starts if starts is None else starts), i32(prefix),
                int(max(prefix.max(initial=0), 0)))

    def run(self, **kw):
        out = kvq.kvq_prefix_decode(*self.args(**kw), residual=self.res)
        torch.cuda.synchronize()
        return out

    def reference(self, ctx=None, skip=()):
        """(output, tolerance) in float64; `skip`: physical blocks left out."""
        ctx = self.ctx if ctx is None else np.asarray(ctx)
        d, g = self.d, self.hq // self.hkv
        ref = np.zeros((len(ctx), self.hq, d))
        tol = np.zeros_like(ref)
        rot = self.oc.rotation
        for s, n in enumerate(ctx):
            n = int(n)
            part = n // 16 * 16 if self.tail else n
            t = np.arange(part)
            t = t[~np.isin(self.table[s][t // 16], list(skip))] if len(skip) else t
            blk, off = self.table[s][t // 16], t % 16
            k, v = (oracle.dequantize_cache_rows(self.oc, w, blk, off) for w in ("k", "v"))
            if self.tail and n > part:
                f = lambda w: oracle.bf16_bits_to_f32(H.bits(self.res[w][s, :n - part])).astype(np.float64)  # noqa: E731
                k, v = np.concatenate([k, f("k")]), np.concatenate([v, f("v")])
            if not len(k):
                continue
            q = oracle.bf16_bits_to_f32(H.bits(self.q[s])).astype(np.float64)
            if rot is not None:
                q = oracle.rotate_query_fp64(q, rot)
            k, v = np.repeat(k, g, axis=1), np.repeat(v, g, axis=1)
            z = np.einsum("hd,thd->ht", q, k) / np.sqrt(d)
            reach = (np.einsum("hd,thd->ht", np.abs(q), np.abs(k)) / np.sqrt(d)).max(1)
            p = np.exp(z - z.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            o = np.einsum("ht,thd->hd", p, v)
            a = np.einsum("ht,thd->hd", p, np.abs(v))
            move = 2.0 ** -11 * (1 + int(rot is not None)) + 2.0 ** -20
            err = a * (2.0 ** -11 * 2 + 2.0 ** -17 + np.expm1(2 * move * reach)[:, None])
            err = err + 2.0 ** -28 * len(v) * np.abs(v).max((0, 2))[:, None]
            if rot is not None:
                o = oracle.unrotate_output_fp64(o, rot)
                err = np.broadcast_to(err.sum(-1, keepdims=True) / d, err.shape)
            ref[s], tol[s] = o, err + 2.0 ** -8 * (np.abs(o) + err)
        return ref, tol

    def check(self, out, **kw):
        ref, tol = self.reference(**kw)
        got = out.float().cpu().numpy().astype(np.float64)
        assert np.isfinite(got).all()
        worst = np.max(np.abs(got - ref) / np.maximum(tol, 1e-30)) if got.size else 0.0
        print(f"[prefix] error / bound {worst:.3f}, relative 2-norm "
              f"{np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30):.2e}")
        assert worst <= 1.0
        assert (got[(self.ctx if kw.get("ctx") is None else np.asarray(kw["ctx"])) == 0] == 0).all()


FORMATS = [(k, v, 128) for k in KS for v in VS] + [(k, v, 64) for k in ("int8", "fp8", "int4", "int8c")
                                                   for v in ("int8", "fp8", "int4g")]


@pytest.mark.parametrize("k,v,d", FORMATS)
def test_formats(k, v, d):
    s = Batch(k, v, hq=12, hkv=3, d=d, groups=[(150, [190, 144, 151, 163, 160])], seed=1)
    s.check(s.run())
    assert kvq.kvq_device_errors() == 0


@pytest.mark.parametrize("k,v,d,hq,hkv", [("int4", "int4g", 128, 32, 8), ("int4", "int4g", 64, 3, 3),
                                          ("int8", "int8", 64, 16, 2), ("fp8", "int2g", 128, 6, 1),
                                          ("int8", "int4g", 128, 14, 7)])
def test_rotated(k, v, d, hq, hkv):
    s = Batch(k, v, hq=hq, hkv=hkv, d=d, groups=[(300, [330, 301, 350])], loose=[40], rot=True, seed=2)
    s.check(s.run())
    assert kvq.kvq_device_errors() == 0


@pytest.mark.parametrize("k,v,d,hq,hkv", [("int8c", "int4g", 128, 16, 2), ("int8c", "int8", 64, 4, 4),
                                          ("int2c", "int2g", 128, 24, 8), ("int2c", "fp8", 128, 5, 1)])
def test_tail(k, v, d, hq, hkv):
    s = Batch(k, v, hq=hq, hkv=hkv, d=d, groups=[(200, [207, 240, 193, 16, 15, 0, 7])], loose=[3, 33], tail=True, seed=3)
    s.check(s.run())
    assert kvq.kvq_device_errors() == 0


CASES = {
    "two_sequences": dict(groups=[(64, [64, 80])]),
    "one_block": dict(groups=[(16, [16, 17])]),
    "prefix_below_a_block": dict(groups=[(15, [20, 30])]),
    "prefix_not_in_whole_blocks": dict(groups=[(143, [143, 150, 200])]),
    "tile_ends": dict(groups=[(128, [128, 129]), (256, [256, 300]), (112, [112, 113]), (144, [144, 145])]),
    "suffix_empty_everywhere": dict(groups=[(320, [320, 320, 320])]),
    "rows_end_inside_the_prefix": dict(groups=[(400, [401, 0, 1, 15, 16, 17, 127, 128, 129, 399, 400])]),
    "first_row_is_empty": dict(groups=[(200, [0, 210, 0, 222])]),
    "all_rows_short": dict(groups=[(500, [40, 33, 7])]),
    "all_rows_empty": dict(groups=[(500, [0, 0])], loose=[5]),
    "nothing_at_all": dict(groups=[(16, [0, 0])], loose=[0]),
    "a_group_of_one": dict(groups=[(100, [130]), (90, [95, 99]), (0, [50, 60])]),
    "empty_groups": dict(groups=[(50, []), (80, [90, 85]), (70, [])], loose=[10, 700]),
    "no_group": dict(groups=[], loose=[100, 33, 0]),
    "many_groups": dict(groups=[(16 * (i % 9) + i, [16 * (i % 9) + i + 5, 16 * (i % 9) + i + 33]) for i in range(40)],
                        hkv=1, hq=2),
    "rows_128": dict(groups=[(300, [301 + i for i in range(16)])], hq=16),
    "rows_129_of_256": dict(groups=[(300, [300 + i for i in range(43)])], hq=6),
    "rows_256": dict(groups=[(270, [270 + i for i in range(32)])], hq=16),
    "rows_257_cut_in_two": dict(groups=[(270, [270 + i % 40 for i in range(257)])], hq=2),
    "rows_600": dict(groups=[(190, [190 + i % 20 for i in range(75)])], hq=16),
    "g1": dict(groups=[(500, [510, 520, 533])], hq=2),
    "g3_h1": dict(groups=[(500, [510, 520, 533])], hq=3, hkv=1),
    "g7_h8": dict(groups=[(500, [510, 520, 533])], hq=56, hkv=8),
    "long": dict(groups=[(5003, [5003, 5100, 5040])], hq=4),
    "long_many_rows": dict(groups=[(2900, [2900 + i for i in range(40)])], hq=8, hkv=1),
    "d64": dict(groups=[(700, [700 + 3 * i for i in range(30)])], d=64, k="int8", v="int8"),
    "d64_rows": dict(groups=[(700, [700 + 3 * i for i in range(50)])], d=64, k="int8", v="int4g", hq=16),
    "wide_v_scales": dict(groups=[(600, [610, 633, 700])], v_spread=1e-3),
    "wide_v_group_scales": dict(groups=[(600, [610, 633, 700])], v="int4g", v_spread=1e3),
}


@pytest.mark.parametrize("name", list(CASES))
def test_shapes(name):
    s = Batch(**CASES[name], seed=4)
    s.check(s.run())
    assert kvq.kvq_device_errors() == 0


def test_twice_the_same_bits_and_the_paged_decode():
    s = Batch("fp8", "int4g", hq=32, hkv=8, groups=[(1000, [1000 + 7 * i for i in range(20)]), (300, [310] * 9)],
              loose=[77], seed=5)
    a, b = s.run(), s.run()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    q, fmt, cache, bt, cl, mx = s.args()[:6]
    plain = kvq.kvq_paged_decode(q, fmt, cache, bt, cl, mx).cpu().numpy()
    ref, tol = s.reference()
    assert (np.abs(plain - ref) <= tol).all() and (np.abs(a.float().cpu().numpy() - plain) <= 2 * tol).all()


def test_masked_scores_of_extreme_rows():
    # rows of huge and of zero queries: no overflow on the way to f16, no NaN
    s = Batch("int8", "int8", groups=[(200, [201, 230, 210])], seed=6)
    s.q[0] *= 2.0 ** 60
    s.q[1] = 0
    s.q[2] *= 2.0 ** -70
    out = s.run()
    ref, tol = s.reference()
    got = out.float().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got[1:] - ref[1:]) <= tol[1:]).all()
    # 2^60: the softmax is one-hot, and the row it picks is a cached V row: its
    # scaled codes are rounded to f16 (2^-11), then the output to BF16 (2^-8 of
    # what that left)
    assert (np.abs(got[0] - ref[0]) <= (2.0 ** -11 + 2.0 ** -8 * (1 + 2.0 ** -11)) * np.abs(ref[0]) + 1e-6).all()


def test_zero_scales():
    s = Batch("int8", "int8", groups=[(160, [161, 170])], seed=7)
    s.cache["v_scale"].nan_to_num_(0.0).zero_()
    assert (s.run() == 0).all()
    assert kvq.kvq_device_errors() == 0


def test_a_bad_block_is_skipped():
    s = Batch(groups=[(300, [310, 333, 301])], loose=[20], seed=8)
    for bad in (-1, int(s.fmt.num_blocks), 2 ** 31 - 1):
        table, gone = s.table.copy(), int(s.table[0, 9])
        table[:3, 9] = bad
        out = s.run(table=table)
        assert kvq.kvq_device_errors() == kvq.DEVERR_BLOCK_RANGE
        s.check(out, skip=[gone])


def test_invalid_groups_and_lengths_share_nothing():
    s = Batch(groups=[(100, [110, 120, 130]), (80, [90, 85])], loose=[40], seed=9)
    for starts, prefix, bit in [([0, 3, 2], None, kvq.DEVERR_GROUP_RANGE), ([-1, 3, 5], None, kvq.DEVERR_GROUP_RANGE),
                                ([0, 3, 7], None, kvq.DEVERR_GROUP_RANGE), (None, [-5, 80], kvq.DEVERR_CONTEXT_RANGE)]:
        s.check(s.run(starts=starts, prefix=prefix))
        assert kvq.kvq_device_errors() == bit, (starts, prefix)
    a = list(s.args())
    a[8] = 90                                          # the first prefix is longer than the stated bound
    out = kvq.kvq_prefix_decode(*a)
    s.check(out)
    assert kvq.kvq_device_errors() == kvq.DEVERR_CONTEXT_RANGE


def test_overlapping_groups_stay_right():
    # starts out of order name sequences twice: nobody is counted twice
    s = Batch(groups=[(96, [110, 120, 130, 140, 99, 101])], seed=10)
    for starts in ([0, 4, 1, 6], [2, 6, 0, 5], [0, 6, 0, 6]):
        s.check(s.run(starts=starts, prefix=[96, 96, 96]))
        kvq.kvq_device_errors()


def test_invalid_contexts_give_zero():
    s = Batch(groups=[(100, [110, 120, 130])], loose=[40], seed=11)
    for bad in (-3, 2 ** 30):
        ctx = s.ctx.copy()
        ctx[0] = bad
        a = list(s.args(ctx=ctx))
        a[5] = 130
        out = kvq.kvq_prefix_decode(*a)
        assert kvq.kvq_device_errors() == kvq.DEVERR_CONTEXT_RANGE
        ctx[0] = 0
        s.check(out, ctx=ctx)


def test_streams_and_captured_graphs():
    s = Batch("int8", "int4g", hq=16, hkv=4, groups=[(500, [501 + i for i in range(6)])], seed=12)
    t = Batch("int8", "int4g", hq=16, hkv=4, groups=[(700, [701 + 9 * i for i in range(6)])], seed=13)
    want = [s.run().clone(), t.run().clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = kvq.kvq_prefix_decode(*s.args(), stream=side)
    side.synchronize()
    assert torch.equal(out, want[0])
    graphs, outs = [], []
    args = [s.args(), t.args()]
    for a in args:                                       # each graph owns its workspace
        o = torch.empty_like(a[0])
        ws = torch.empty(kvq.kvq_prefix_decode_workspace_size(a[1], 6, 16, a[5], 1), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kvq.kvq_prefix_decode(*a, out=o, workspace=ws)
        graphs.append(g)
        outs.append((o, ws))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for o, _w in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for (o, _w), w in zip(outs, want):
            assert torch.equal(o, w)
    # the captured call follows the device's lengths
    args[0][4].sub_(3)
    graphs[0].replay()
    torch.cuda.synchronize()
    s.check(outs[0][0], ctx=s.ctx - 3)


def test_calls_in_a_row_share_a_workspace():
    """The kernels of a call overlap; calls of a stream do not, nor the kernels
    around them that change lengths and read outputs."""
    a = Batch("fp8", "int8", hq=16, hkv=4, groups=[(2000, [2000 + 7 * i for i in range(40)])], seed=16)
    b = Batch("fp8", "int8", hq=16, hkv=4, loose=[40 + 13 * i for i in range(40)], seed=17)  # no group at all
    c = Batch("fp8", "int8", hq=16, hkv=4, groups=[(90, [100, 95, 3]), (640, [650] * 37)], seed=18)
    args = [a.args(), b.args(), c.args()]
    size = max(kvq.kvq_prefix_decode_workspace_size(x[1], 40, 16, x[5], int(x[7].shape[0])) for x in args)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    start = [x[4].clone() for x in args]
    want = {}
    for less in range(4):
        for i, x in enumerate(args):
            torch.sub(start[i], less, out=x[4])
            torch.cuda.synchronize()
            want[i, less] = kvq.kvq_prefix_decode(*x)
            torch.cuda.synchronize()
    ws.fill_(0xFF)
    got = []
    for n in range(48):
        i, less = n % 3, n % 4
        torch.sub(start[i], less, out=args[i][4])
        out = kvq.kvq_prefix_decode(*args[i], workspace=ws)
        got.append((i, less, out.clone()))
        out.fill_(float("nan"))
    torch.cuda.synchronize()
    for i, less, out in got:
        assert torch.equal(out, want[i, less]), (i, less)
    a.check(want[0, 3], ctx=a.ctx - 3)


def test_a_call_allocates_on_its_own_stream(monkeypatch):
    """Outputs and workspaces that a call makes belong to the stream it runs on
    (given as a Stream or a raw handle)."""
    s = Batch(groups=[(300, [310, 320, 333])], seed=20)
    want, args = s.run(), s.args()
    side, plain, where = torch.cuda.Stream(), torch.empty, []

    def empty(*a, **k):
        where.append(torch.cuda.current_stream().cuda_stream)
        return plain(*a, **k)
    i32 = args[4].clone()
    pool, tables = kvq.allocate_pool(40), torch.full((3, 9), -1, dtype=torch.int32, device="cuda")
    ctx, one = torch.zeros_like(i32), torch.ones_like(i32)
    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "empty", empty)
    for stream in (side, side.cuda_stream):
        out = kvq.kvq_prefix_decode(*args, stream=stream)
        got = kvq.kvq_assign_blocks(one, ctx, tables, pool, 3, stream=stream)
        side.synchronize()
        assert torch.equal(out, want) and int(got[0][-1]) == 3
        torch.cuda.synchronize()
    assert len(where) == 10 and set(where) == {side.cuda_stream}


def test_more_tiles_than_counted_are_refused():
    s = Batch(groups=[(100, [110, 120])], seed=19)
    q, fmt, cache, tables, ctx, _, starts, prefix, _ = s.args()
    lib, cf = kvq.load_library(), s.fmt.as_c()
    caches, scales = kvq._caches(cache)

    def call(batch, width, longest):
        return lib.kvq_prefix_decode(q.data_ptr(), batch, 8, ctypes.byref(cf), caches, scales, tables.data_ptr(), width,
                                     ctx.data_ptr(), 120, starts.data_ptr(), prefix.data_ptr(), 1, longest, None, None,
                                     q.data_ptr(), ctx.data_ptr() // 256 * 256, 0, None)
    assert call(8192, 1 << 18, 16) == kvq.KVQ_ERR_UNSUPPORTED        # 2^31 table entries
    # sequences * kv heads * tiles (2^15 for 2^18 blocks): 2^31 with 8 heads; fewer go on to the next check
    assert call(8192, (1 << 18) - 1, 0x7FFFFFFF) == kvq.KVQ_ERR_WORKSPACE
    cf.num_kv_heads = 8
    assert call(8191, (1 << 18) - 8, 0x7FFFFFFF) == kvq.KVQ_ERR_WORKSPACE
    assert call(8192, (1 << 18) - 1, 0x7FFFFFFF) == kvq.KVQ_ERR_UNSUPPORTED


def test_refusals():
    s = Batch(groups=[(100, [110, 120])], seed=14)
    a = s.args()
    ws = kvq.kvq_prefix_decode_workspace_size(s.fmt, 2, 8, 120, 1)
    with pytest.raises(kvq.KvqError) as e:
        kvq.kvq_prefix_decode(*a, workspace=torch.empty(ws - 256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == kvq.KVQ_ERR_WORKSPACE
    with pytest.raises(kvq.KvqError) as e:               # no tail without per-channel K
        kvq.kvq_prefix_decode(*a, residual=kvq.allocate_residual(s.fmt, 2))
    assert e.value.status == kvq.KVQ_ERR_UNSUPPORTED
    with pytest.raises(TypeError):
        kvq.kvq_prefix_decode(*a, out=torch.empty(a[0].shape, dtype=torch.float32, device="cuda"))
    with pytest.raises(ValueError):
        kvq.kvq_prefix_decode(*a[:6], a[6][:1], *a[7:])


def test_serving_steps_together():
    """assign -> quantize-write -> prefix decode -> release, as a serving loop
    uses them: a prompt kept by row 0, readers that join, grow and leave."""
    k = v = FP8
    hq, hkv, d, rows, width, nb = 8, 2, 128, 6, 20, 70
    fmt = kvq.cache_format(k, v, hkv, d, nb)
    cache, pool = kvq.allocate_cache(fmt), kvq.allocate_pool(nb)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ctx, tables = i32([0] * rows), torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(15)
    content = {}                                          # (row, position) -> (k, v) bits

    def write(n, prefix_rows=None, prefix_blocks=None):
        cap = sum(n)
        off, slots, pos = kvq.kvq_assign_blocks(i32(n), ctx, tables, pool, cap, prefix_rows=prefix_rows,
                                                prefix_blocks=prefix_blocks)
        x = torch.randn((2, cap, hkv, d), generator=gen, device="cuda").to(torch.bfloat16)
        kvq.kvq_quantize_write(x[0], x[1], slots, fmt, cache)
        o = off.tolist()
        for r in range(rows):
            for j in range(o[r], o[r + 1]):
                content[r, int(pos[j])] = (H.bits(x[0, j]), H.bits(x[1, j]))

    prompt = 150
    write([prompt, 0, 0, 0, 0, 0])
    whole = prompt // 16
    write([0, 20, 13, 1, 0, 0], i32([-1, 0, 0, 0, -1, -1]), i32([0, whole, whole, whole, 0, 0]))
    for r in (1, 2, 3):
        for p in range(16 * whole):
            content[r, p] = content[0, p]
    for step in range(6):
        live = [0, step < 5, 1, 1, step > 2, step > 3]    # row 1 has left after step 4
        if step == 3:                                     # row 4 joins, sharing from row 1
            write([0, 0, 0, 0, 5, 0], i32([-1, -1, -1, -1, 1, -1]), i32([0, 0, 0, 0, whole, 0]))
            for p in range(16 * whole):
                content[4, p] = content[1, p]
        write([int(x) for x in live])
        q = torch.randn((rows, hq, d), generator=gen, device="cuda").to(torch.bfloat16)
        out = kvq.kvq_prefix_decode(q, fmt, cache, tables, ctx, width * 16, i32([0, 5]), i32([prompt]), prompt)
        torch.cuda.synchronize()
        assert kvq.kvq_device_errors() == 0
        # the oracle quantizes the same rows into a cache of its own, row by row
        oc = oracle.OracleCache(rows * width, 16, hkv, d, k, v)
        lens = ctx.tolist()
        own = np.arange(rows * width).reshape(rows, width)
        for r in range(rows):
            if lens[r]:
                kb, vb = (np.stack([content[r, p][w] for p in range(lens[r])]) for w in (0, 1))
                oracle.quantize_write(oc, kb, vb, own[r, 0] * 16 + np.arange(lens[r]))
        ref = oracle.paged_decode_fp64(oc, H.bits(q), own, lens)
        err = np.abs(out.float().cpu().numpy() - ref)
        assert (err <= 2.0 ** -8 * np.abs(ref) + 2e-3).all(), (step, err.max())
        if step == 4:
            kvq.kvq_release_blocks(i32([10_000, 0, 10_000, 10_000, 10_000, 10_000]), ctx, tables, pool)
    kvq.kvq_release_blocks(i32([0] * rows), ctx, tables, pool)
    assert int(pool["free_count"]) == nb and int(pool["ref_counts"].sum()) == 0
    assert sorted(pool["free_list"].tolist()) == list(range(nb))
