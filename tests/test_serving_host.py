"""Host-side argument checks of the serving-step calls (block pool and
shared-prefix decode) that need no GPU."""
import ctypes

import pytest

import quantized_paged_kv_write_gb300 as kvq
from quantized_paged_kv_write_gb300 import build as kbuild

BUF = ctypes.c_void_p(4096)  # never dereferenced: every call returns before any device work
ODD = ctypes.c_void_p(4098)


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kvq.load_library()


def _pool(nb=8, fl=BUF, fc=BUF, rc=BUF):
    return kvq._BlockPool(fl, fc, rc, nb)


def _assign(lib, rows=2, lens=BUF, ctx=BUF, tables=BUF, width=4, pool=None, pr=None, pb=None, cap=8, off=BUF, slots=BUF,
            pos=BUF):
    return lib.kvq_assign_blocks(lens, rows, ctx, tables, width, pool or _pool(), pr, pb, cap, off, slots, pos, None)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(width=0), dict(lens=None), dict(ctx=None), dict(tables=None), dict(cap=-1), dict(off=None),
    dict(slots=None), dict(pr=BUF), dict(pb=BUF), dict(lens=ODD), dict(ctx=ODD), dict(tables=ODD), dict(off=ODD),
    dict(slots=ctypes.c_void_p(4100)), dict(pos=ODD), dict(pool=_pool(-1)), dict(pool=_pool(fl=None)),
    dict(pool=_pool(fc=None)), dict(pool=_pool(rc=None)), dict(pool=_pool(fc=ODD))])
def test_assign_refuses(lib, bad):
    assert _assign(lib, **bad) == kvq.KVQ_ERR_INVALID_ARG


@pytest.mark.parametrize("big", [dict(rows=8193), dict(rows=8192, width=1 << 18), dict(pool=_pool(1 << 31))])
def test_assign_refuses_what_is_too_large(lib, big):
    assert _assign(lib, **big) == kvq.KVQ_ERR_UNSUPPORTED


def test_release_checks(lib):
    call = lambda rows=2, keep=BUF, ctx=BUF, tb=BUF, width=4, pool=None: lib.kvq_release_blocks(  # noqa: E731
        keep, rows, ctx, tb, width, pool or _pool(), None)
    assert call(rows=0, keep=None, ctx=None, tb=None) == kvq.KVQ_OK
    for bad in (dict(rows=-1), dict(keep=None), dict(ctx=None), dict(tb=None), dict(width=0), dict(keep=ODD),
                dict(pool=_pool(fc=None))):
        assert call(**bad) == kvq.KVQ_ERR_INVALID_ARG, bad
    assert call(rows=9000) == kvq.KVQ_ERR_UNSUPPORTED


def _fmt(**kw):
    base = dict(k_dtype=0, v_dtype=0, k_gran=0, v_gran=0, k_group=0, v_group=0, num_kv_heads=8, head_dim=128,
                block_size=16, rotation=0, num_blocks=10)
    base.update(kw)
    return kvq._Format(**base)


def _decode(lib, fmt=None, batch=0, hq=32, width=1, max_ctx=0, groups=0, max_prefix=0, rk=None, rv=None):
    f = fmt or _fmt()
    return lib.kvq_prefix_decode(None, batch, hq, ctypes.byref(f), kvq._Caches(None, None), kvq._Scales(None, None),
                                 None, width, None, max_ctx, None, None, groups, max_prefix, rk, rv, None, None, 0, None)


def test_prefix_decode_checks(lib):
    assert _decode(lib) == kvq.KVQ_OK                                              # empty batch
    for bad in (dict(batch=-1), dict(hq=12), dict(groups=-1), dict(max_ctx=-1), dict(max_prefix=-1), dict(width=0),
                dict(fmt=_fmt(k_gran=2), rk=BUF), dict(fmt=_fmt(k_gran=2), rk=BUF, rv=ODD)):
        assert _decode(lib, **bad) == kvq.KVQ_ERR_INVALID_ARG, bad
    for bad in (dict(hq=128), dict(batch=8193), dict(fmt=_fmt(head_dim=96)), dict(groups=8193), dict(rk=BUF, rv=BUF)):
        assert _decode(lib, **bad) == kvq.KVQ_ERR_UNSUPPORTED, bad


def test_pool_and_lengths_must_agree_in_the_binding():
    torch = pytest.importorskip("torch")
    i = torch.zeros(3, dtype=torch.int32)
    t = torch.zeros((3, 2), dtype=torch.int32)
    pool = kvq.allocate_pool(4, device="cpu")
    with pytest.raises(ValueError):
        kvq.kvq_assign_blocks(i, i[:2], t, pool, 4)
    with pytest.raises(ValueError):
        kvq.kvq_assign_blocks(i, i, t, pool, 4, prefix_rows=i[:2])
    with pytest.raises(ValueError):
        kvq.kvq_release_blocks(i, i, t[:2], pool)
    with pytest.raises(ValueError):                                                 # not CUDA tensors
        kvq.kvq_release_blocks(i, i, t, pool)


@pytest.mark.parametrize("rows,width", [(1, 1 << 27), (1, (1 << 31) - 1), (15, 1 << 27), (16, (1 << 27) - 1),
                                        (8192, (1 << 18) - 7)])
def test_tables_whose_positions_pass_32_bits_are_refused(lib, rows, width):
    assert _assign(lib, rows=rows, width=width) == kvq.KVQ_ERR_UNSUPPORTED
    assert lib.kvq_release_blocks(BUF, rows, BUF, BUF, width, _pool(), None) == kvq.KVQ_ERR_UNSUPPORTED


def test_lengths_of_two_columns_are_refused_by_the_binding():
    torch = pytest.importorskip("torch")
    i, t = torch.zeros(3, dtype=torch.int32), torch.zeros((3, 2), dtype=torch.int32)
    pool = kvq.allocate_pool(4, device="cpu")
    with pytest.raises(ValueError, match=r"new_lens and context_lens must be \[R\]"):
        kvq.kvq_assign_blocks(t, i, t, pool, 4)
    with pytest.raises(ValueError, match=r"keep_lens and context_lens must be \[R\]"):
        kvq.kvq_release_blocks(t, i, t, pool)


def test_decodes_refuse_tables_whose_positions_pass_32_bits(lib):
    c, s = kvq._Caches(BUF, BUF), kvq._Scales(BUF, BUF)
    f, g = _fmt(), _fmt(k_gran=2)
    for width in (1 << 27, (1 << 28) + 5, (1 << 31) - 1):
        assert _decode(lib, batch=1, width=width) == kvq.KVQ_ERR_UNSUPPORTED
        assert lib.kvq_paged_decode(BUF, 1, 32, ctypes.byref(f), c, s, BUF, width, BUF, 64, BUF, BUF, 1 << 20,
                                    None) == kvq.KVQ_ERR_UNSUPPORTED
        assert lib.kvq_kivi_decode(BUF, 1, 32, ctypes.byref(g), c, s, BUF, width, BUF, 64, BUF, BUF, BUF, BUF, 1 << 20,
                                   None) == kvq.KVQ_ERR_UNSUPPORTED
        assert lib.kvq_kivi_append(BUF, BUF, 1, ctypes.byref(g), c, s, BUF, width, BUF, BUF, BUF,
                                   None) == kvq.KVQ_ERR_UNSUPPORTED
