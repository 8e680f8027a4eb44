"""Host-side refusals of the decode loop's entry points (no GPU needed)."""
import ctypes

import pytest
import torch

from gemm_decode_register_gb300 import build as b
from gemm_decode_register_gb300 import ops

A = 1 << 20  # an aligned fake address: validation fails before it is used
Z = 1 << 40


@pytest.fixture(scope="module")
def lib():
    b.build()
    return ops.load()


def beam_args(**kw):
    d = dict(logits=A, dtype=0, row_stride=1000, scores=A, mask=A, mask_stride=32, B=2, W=4, V=1000, k=8, eos=-1, score=A,
             parent=A, token=A, next_score=A, next_parent=A, next_token=A, ws=A, ws_bytes=Z)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,want", [
    (dict(logits=0), -1), (dict(scores=0), -1), (dict(score=0), -1), (dict(parent=0), -1), (dict(token=0), -1),
    (dict(B=0), -1), (dict(W=0), -1), (dict(V=0), -1), (dict(k=0), -1), (dict(next_score=0), -1), (dict(next_token=0), -1),
    (dict(dtype=2), -2), (dict(W=65), -2), (dict(k=129), -2), (dict(V=(1 << 20) + 1, row_stride=1 << 21, mask_stride=1 << 16), -2),
    (dict(B=4097), -2), (dict(B=4096, W=16), -2), (dict(row_stride=999), -1), (dict(mask_stride=31), -1),
    (dict(ws_bytes=255), -1), (dict(ws=None), -1),  # (a size without a workspace)
    (dict(logits=A + 1), -3), (dict(logits=A + 2, dtype=1), -3), (dict(scores=A + 2), -3), (dict(mask=A + 1), -3),
    (dict(token=A + 2), -3), (dict(next_parent=A + 1), -3), (dict(ws=A + 16), -3)])
def test_beam_rejects(lib, kw, want):
    assert lib.mx_beam_select(*beam_args(**kw)) == want


def test_beam_workspace_sizes(lib):
    f = lib.mx_beam_select_workspace_size
    assert 0 < f(1, 4, 32000, 8) <= 16 << 20 and f(1, 4, 32000, 8) % 256 == 0
    for bad in ((0, 4, 100, 8), (1, 0, 100, 8), (1, 4, 0, 8), (1, 4, 100, 0), (1, 65, 100, 8), (1, 4, 100, 129),
                (1, 4, (1 << 20) + 1, 8), (4096, 16, 100, 8)):
        assert f(*bad) == 0
    big = (1100, 32, 1000, 128)
    assert f(*big) > 16 << 20
    assert lib.mx_beam_select(*beam_args(B=1100, W=32, V=1000, mask=0, k=128, ws=None, ws_bytes=0)) == -1


def pool(**kw):
    d = dict(count=A, refs=A, free_pages=A, work=A, num_pages=100)
    d.update(kw)
    return ctypes.byref(ops._PagePool(*d.values()))


POOL_FAULTS = [(dict(count=0), -1), (dict(refs=0), -1), (dict(free_pages=0), -1), (dict(work=0), -1), (dict(num_pages=0), -1),
               (dict(num_pages=(1 << 24) + 1), -2), (dict(refs=A + 2), -3), (dict(work=A + 128), -3)]


def remap_args(p=None, **kw):
    d = dict(pool=p or pool(), page_size=16, table_in=A, in_stride=8, in_pages=8, kv_len_in=2 * A, S_in=4, table_out=3 * A,
             out_stride=8, out_pages=8, kv_len_out=4 * A, S_out=4, parent=A, keep=A, add=A, add_all=0, copies=A)
    d.update(kw)
    return list(d.values())


def compact_args(p=None, **kw):
    d = dict(pool=p or pool(), page_size=16, table=A, stride=8, pages=8, kv_len=A, S=4, copies=A)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,want", POOL_FAULTS)
def test_pool_rejects(lib, kw, want):
    assert lib.mx_kv_remap(*remap_args(pool(**kw))) == want
    assert lib.mx_kv_compact(*compact_args(pool(**kw))) == want


@pytest.mark.parametrize("kw,want", [
    (dict(pool=None), -1), (dict(page_size=0), -1), (dict(table_in=0), -1), (dict(in_pages=0), -1), (dict(in_stride=7), -1),
    (dict(kv_len_in=0), -1), (dict(S_in=0), -1), (dict(table_out=0), -1), (dict(out_pages=0), -1), (dict(out_stride=7), -1),
    (dict(kv_len_out=0), -1), (dict(S_out=0), -1), (dict(parent=0), -1), (dict(copies=0), -1), (dict(add_all=-1), -1),
    (dict(S_in=4097), -2), (dict(S_out=4097), -2), (dict(table_in=A + 2), -3), (dict(parent=A + 1), -3), (dict(keep=A + 2), -3),
    (dict(add=A + 2), -3), (dict(copies=A + 4), -3),
    (dict(table_out=A), -1), (dict(table_out=A + 4 * 31), -1), (dict(kv_len_out=2 * A + 12), -1)])  # in place
def test_remap_rejects(lib, kw, want):
    assert lib.mx_kv_remap(*remap_args(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(pool=None), -1), (dict(page_size=0), -1), (dict(table=0), -1), (dict(pages=0), -1), (dict(stride=7), -1),
    (dict(kv_len=0), -1), (dict(S=0), -1), (dict(S=4097), -2), (dict(copies=0), -1), (dict(copies=A + 8), -3),
    (dict(kv_len=A + 2), -3)])
def test_compact_rejects(lib, kw, want):
    assert lib.mx_kv_compact(*compact_args(**kw)) == want


def test_pool_work_sizes(lib):
    f = lib.mx_page_pool_work_size
    assert f(1) > 0 and f(1000) % 256 == 0 and f(1 << 24) > f(1000)
    assert f(0) == f(-1) == f((1 << 24) + 1) == 0


def cache(**kw):
    d = dict(k=A, v=A, k_scales=None, v_scales=None, block_table=None, page_stride=2 * 16 * 128, head_stride=16 * 128,
             token_stride=128, scale_page_stride=0, scale_head_stride=0, scale_token_stride=0, kv_fmt=0, num_pages=4,
             page_size=16, Hkv=2, D=128, table_stride=0, table_pages=0)
    d.update(kw)
    c = ops._PagedKV()
    for name, v in d.items():
        setattr(c, name, v)
    return c


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(num_pages=0), -1), (dict(page_size=0), -1), (dict(Hkv=0), -1),
    (dict(D=0), -1), (dict(page_stride=0), -1), (dict(head_stride=-128), -1), (dict(token_stride=0), -1), (dict(kv_fmt=2), -2),
    (dict(D=264), -2), (dict(D=100), -2), (dict(Hkv=4097), -2), (dict(Hkv=4096, page_size=8192), -2), (dict(kv_fmt=1), -1),
    (dict(kv_fmt=1, k_scales=A, v_scales=A), -1), (dict(k=A + 8), -3), (dict(token_stride=132), -3)])
def test_copy_rejects_caches(lib, kw, want):
    for caches in ([cache(**kw)], [cache(), cache(**kw)]):
        assert lib.mx_kv_copy_pages((ops._PagedKV * len(caches))(*caches), len(caches), A, 4) == want


@pytest.mark.parametrize("kw", [dict(num_pages=5), dict(page_size=8), dict(Hkv=1), dict(D=64), dict(page_stride=8192),
                                dict(head_stride=4096), dict(token_stride=256)])
def test_copy_rejects_caches_that_differ(lib, kw):
    assert lib.mx_kv_copy_pages((ops._PagedKV * 2)(cache(), cache(**kw)), 2, A, 4) == -1


def test_copy_rejects_lists(lib):
    c = (ops._PagedKV * 1)(cache())
    assert lib.mx_kv_copy_pages(None, 1, A, 4) == -1
    assert lib.mx_kv_copy_pages(c, 0, A, 4) == -1
    assert lib.mx_kv_copy_pages(c, 257, A, 4) == -2
    assert lib.mx_kv_copy_pages(c, 1, None, 4) == -1
    assert lib.mx_kv_copy_pages(c, 1, A, 0) == -1
    assert lib.mx_kv_copy_pages(c, 1, A, (1 << 24) + 1) == -2
    assert lib.mx_kv_copy_pages(c, 1, A + 8, 4) == -3


@pytest.mark.parametrize("args,want", [
    ((A, 2, A, A, 4, 64), -2), ((0, 0, A, A, 4, 64), -1), ((A, 0, 0, A, 4, 64), -1), ((A, 0, A, 0, 4, 64), -1),
    ((A, 0, A, A, 0, 64), -1), ((A, 0, A, A, 4, 0), -1), ((A, 0, A, A, 4, 72), -1), ((A + 8, 0, A, A, 4, 64), -3),
    ((A, 0, A + 4, A, 4, 64), -3), ((A, 0, A, A + 2, 4, 64), -3)])
def test_i8_quantize_rejects(lib, args, want):
    assert lib.mx_i8_quantize(*args) == want


def i8_args(**kw):
    d = dict(x=A, xdtype=2, sx=A, w=A, sw=A, y=A, ydtype=0, M=4, N=100, K=64, ws=A, ws_bytes=Z)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,want", [
    (dict(xdtype=3), -2), (dict(ydtype=2), -2), (dict(x=0), -1), (dict(w=0), -1), (dict(sw=0), -1), (dict(y=0), -1),
    (dict(sx=0), -1), (dict(xdtype=0), -1),  # int8 without scales, bf16 with them
    (dict(M=0), -1), (dict(N=0), -1), (dict(K=0), -1), (dict(K=72), -1), (dict(K=131072), -2), (dict(ws_bytes=255), -1),
    (dict(ws=None), -1), (dict(ws=None, ws_bytes=0, M=4096, K=8192), -1), (dict(x=A + 8), -3), (dict(w=A + 4), -3),
    (dict(y=A + 8), -3), (dict(sx=A + 1), -3), (dict(sw=A + 2), -3), (dict(ws=A + 64), -3)])
def test_i8_mm_rejects(lib, kw, want):
    assert lib.mx_i8_mm(*i8_args(**kw)) == want


def test_i8_workspace_sizes(lib):
    f = lib.mx_i8_mm_workspace_size
    assert f(1, 16) > 0 and f(4096, 8192) >= 4096 * 8192 * 2 and f(3, 8192) % 256 == 0
    assert f(0, 16) == f(1, 0) == f(1, 24) == f(1, 131072) == 0


def test_bindings_refuse_host_tensors(lib):
    x, c = torch.zeros((4, 10)), torch.zeros((2, 2))
    with pytest.raises(ValueError):
        ops.beam_select(x, c)
    with pytest.raises(ValueError):
        ops.beam_select(x.double(), c)
    with pytest.raises(ValueError):
        ops.PagePool(10, device="cpu")
    w, s = torch.zeros((4, 32), dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError):
        ops.i8_quantize(torch.zeros((2, 32)))
    with pytest.raises(ValueError):
        ops.i8_mm(torch.zeros((2, 32)), w, s)
    with pytest.raises(ValueError):
        ops.i8_mm(w, w, s)  # codes without scales
    with pytest.raises(ValueError):
        ops.i8_mm(torch.zeros((2, 16)), w, s)
