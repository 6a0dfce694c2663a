"""Host-side argument checks of kvq_prompt_attention, kvq_weigh_decode and
kvq_evict_tokens that need no GPU: each refusal before anything is enqueued."""
import ctypes

import pytest
import torch

import quantized_paged_kv_write_gb300 as kvq
from quantized_paged_kv_write_gb300 import build as kbuild

A = 1 << 20                                                  # some aligned address, never read here


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kvq.load_library()


def _fmt(**kw):
    base = dict(k_dtype=0, v_dtype=0, k_gran=0, v_gran=0, k_group=0, v_group=0, num_kv_heads=8, head_dim=128,
                block_size=16, rotation=0, num_blocks=10)
    base.update(kw)
    return kvq._Format(**base)


def prompt(lib, **kw):
    x = dict(q=A, qs=4096, k=A, ks=1024, v=A, vs=1024, offsets=A, seqs=3, tokens=50, longest=20, hq=32, hkv=8, d=128, out=A,
             lse=A, ws=A, bytes=1 << 20)
    x.update(kw)
    return lib.kvq_prompt_attention(*x.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(seqs=0), 0), (dict(tokens=0), 0), (dict(longest=0), 0), (dict(seqs=0, q=None, out=None), 0),
    (dict(seqs=-1), -1), (dict(tokens=-1), -1), (dict(longest=-1), -1), (dict(hq=0), -1), (dict(hkv=0), -1), (dict(hq=33), -1),
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(offsets=None), -1), (dict(out=None), -1), (dict(ws=None), -1),
    (dict(q=A + 8), -1), (dict(k=A + 2), -1), (dict(v=A + 4), -1), (dict(offsets=A + 2), -1), (dict(out=A + 16), -1),
    (dict(lse=A + 1), -1), (dict(ws=A + 128), -1), (dict(qs=4088), -1), (dict(ks=1020), -1), (dict(vs=1025), -1), (dict(qs=4100), -1),
    (dict(d=96), -2), (dict(hq=72), -2), (dict(hkv=16), -2), (dict(seqs=8193), -2), (dict(tokens=(1 << 24) + 1), -2),
    (dict(longest=(1 << 24) + 1), -2), (dict(qs=1 << 25), -2), (dict(bytes=64), -3)])
def test_prompt_attention_refusals(lib, kw, status):
    assert prompt(lib, **kw) == status


def test_prompt_workspace_grows_with_sequences_and_lengths(lib):
    size = kvq.kvq_prompt_attention_workspace_size
    assert size(0, 0, 8, 8) > 0 and size(8192, 1 << 24, 64, 8) > size(8192, 100, 64, 8) > size(1, 100, 64, 8)
    assert prompt(lib, bytes=size(3, 20, 32, 8) - 1) == kvq.KVQ_ERR_WORKSPACE
    for bad in ((-1, 5, 8, 8), (1, -1, 8, 8), (1, 5, 9, 8)):
        with pytest.raises(kvq.KvqError, match="invalid"):
            size(*bad)
    with pytest.raises(kvq.KvqError, match="unsupported"):
        size(1, 5, 72, 8)
    assert lib.kvq_prompt_attention_workspace_size(1, 1, 8, 8, None) == kvq.KVQ_ERR_INVALID_ARG


def weigh(lib, fmt=None, **kw):
    c, s = kvq._Caches(A, A), kvq._Scales(A, A)
    x = dict(q=A, batch=2, hq=32, fmt=ctypes.byref(fmt or _fmt()), c=c, s=s, tables=A, width=4, ctx=A, longest=60, weights=A,
             stride=60, out=A, ws=A, bytes=0)
    x.update(kw)
    return lib.kvq_weigh_decode(*x.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(weights=None), -1), (dict(weights=A + 2), -1), (dict(stride=59), -1), (dict(batch=0), 0), (dict(batch=-1), -1),
    (dict(hq=33), -1), (dict(hq=72), -2), (dict(q=None), -1), (dict(out=None), -1), (dict(ws=None), -1), (dict(tables=None), -1),
    (dict(width=0), -1), (dict(width=1 << 27), -2)])
def test_weigh_decode_refusals(lib, kw, status):
    assert weigh(lib, **kw) == status


@pytest.mark.parametrize("bad", [dict(k_gran=2), dict(k_dtype=3, k_gran=2), dict(head_dim=96), dict(num_kv_heads=9)])
def test_weigh_decode_formats(lib, bad):
    assert weigh(lib, _fmt(**bad)) == kvq.KVQ_ERR_UNSUPPORTED


def evict(lib, fmt=None, **kw):
    c, s = kvq._Caches(A, A), kvq._Scales(A, A)
    x = dict(keep=A, recent=A, pinned=None, rows=2, ctx=A, tables=A, width=4, fmt=ctypes.byref(fmt or _fmt()), c=c, s=s, refs=None,
             weights=A, positions=60, kept=A + 4096, ws=A, bytes=0)
    x.update(kw)
    return lib.kvq_evict_tokens(*x.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), 0), (dict(rows=0, keep=None, ws=None), 0), (dict(rows=-1), -1), (dict(positions=-1), -1), (dict(width=0), -1),
    (dict(keep=None), -1), (dict(recent=None), -1), (dict(ctx=None), -1), (dict(tables=None), -1), (dict(weights=None), -1),
    (dict(kept=None), -1), (dict(ws=None), -1), (dict(keep=A + 1), -1), (dict(recent=A + 2), -1), (dict(pinned=A + 3), -1),
    (dict(kept=A), -1), (dict(kept=A + 4, ctx=A), -1), (dict(kept=A + 8, ctx=A, bytes=1 << 20, ws=None), -1),
    (dict(kept=A + 16, recent=A + 20), -1), (dict(kept=A + 16, pinned=A + 12), -1), (dict(kept=A + 16, keep=A + 16), -1),
    (dict(refs=A + 1), -1), (dict(weights=A + 2), -1), (dict(kept=A + 2), -1), (dict(ws=A + 16), -1), (dict(rows=8193, kept=A + (1 << 20)), -2),
    (dict(width=1 << 27), -2), (dict(positions=(1 << 30) + 1), -2), (dict(), -3)])
def test_evict_refusals(lib, kw, status):
    assert evict(lib, **kw) == status


@pytest.mark.parametrize("bad", [dict(k_gran=2), dict(k_dtype=3, k_gran=2), dict(head_dim=96), dict(num_blocks=1 << 31),
                                 dict(block_size=32)])
def test_evict_formats(lib, bad):
    assert evict(lib, _fmt(**bad)) == kvq.KVQ_ERR_UNSUPPORTED


def test_evict_workspace_holds_two_lists_of_half_the_positions(lib):
    size = kvq.kvq_evict_workspace_size
    lists = lambda r, h, n: r * h * 2 * (n // 2) * 4  # noqa: E731
    for x in ((3, 8, 101), (0, 8, 101), (5, 1, 1), (8192, 8, 1 << 30)):   # (the last counts in 64 bits)
        assert lists(*x) <= size(*x) <= lists(*x) + x[0] * x[1] * 16 + 256
    with pytest.raises(kvq.KvqError, match="invalid"):
        size(1, 0, 5)
    with pytest.raises(kvq.KvqError, match="unsupported"):
        size(1, 9, 5)


def test_the_binding_refuses_shapes():
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    fmt = kvq.CacheFormat("int8", "int8", "token_head", "token_head", 2, 64, 4)
    i = lambda *s: z(*s, t=torch.int32)  # noqa: E731
    f = lambda *s: z(*s, t=torch.float32)  # noqa: E731
    for q, k, v in ((z(5, 4, 64), z(5, 2, 64), z(5, 1, 64)), (z(5, 4, 64), z(4, 2, 64), z(4, 2, 64)),
                    (z(5, 4, 64), z(5, 2, 128), z(5, 2, 128)), (z(5, 256), z(5, 2, 64), z(5, 2, 64))):
        with pytest.raises(ValueError):
            kvq.kvq_prompt_attention(q, k, v, i(2), 5)
    q, k = z(5, 4, 64), z(5, 2, 64)
    for kw in (dict(out=z(5, 4, 63)), dict(lse=f(5, 3)), dict(lse=f(4, 4))):
        with pytest.raises(ValueError):
            kvq.kvq_prompt_attention(q, k, k, i(2), 5, **{"out": q, "workspace": z(9), **kw})
    with pytest.raises(ValueError):
        kvq.kvq_prompt_attention(q, k, k, i(0), 5)
    with pytest.raises(ValueError, match="CUDA"):
        kvq.kvq_prompt_attention(q, k, k, i(2), 5, out=q, workspace=z(9))
    wide = z(5, 4, 128)[..., :64]
    with pytest.raises(ValueError, match="contiguous"):
        kvq.kvq_prompt_attention(wide, k, k, i(2), 5, out=q, workspace=z(9))
    for w in (f(2, 2), f(3, 2, 64), f(2, 1, 64)):
        with pytest.raises(ValueError):
            kvq.kvq_weigh_decode(z(2, 4, 64), fmt, {}, i(2, 4), i(2), 64, w)
        with pytest.raises(ValueError):
            kvq.kvq_evict_tokens(i(2), i(2), i(2, 4), fmt, {}, w, i(2))
    with pytest.raises(ValueError):
        kvq.kvq_weigh_decode(z(2, 4, 64), fmt, {}, i(2, 4), i(2), 64, f(2, 2, 64), out=f(2, 4, 63))
    for kw in (dict(recent_lens=i(3)), dict(recent_lens=i(2), pinned_lens=i(1)), dict(recent_lens=i(2), kept_lens=i(3)),
               dict(recent_lens=i(2), pool=dict(ref_counts=i(5)))):
        with pytest.raises(ValueError):
            kvq.kvq_evict_tokens(i(2), i(2), i(2, 4), fmt, {}, f(2, 2, 64), **kw)


def test_arrays_without_entries_may_be_null(lib):
    assert weigh(lib, weights=None, batch=0) == 0
    assert weigh(lib, weights=None, stride=0, longest=0) in (kvq.KVQ_ERR_CUDA, kvq.KVQ_ERR_WORKSPACE)   # without, with a GPU
    assert weigh(lib, stride=-1, longest=-1) == kvq.KVQ_ERR_INVALID_ARG
    assert weigh(lib, weights=None, stride=1, longest=0) == kvq.KVQ_ERR_INVALID_ARG
    assert evict(lib, weights=None, positions=0) == kvq.KVQ_ERR_WORKSPACE
    assert weigh(lib, _fmt(k_gran=2), stride=0, longest=0) == kvq.KVQ_ERR_UNSUPPORTED
