"""Host-side refusals of the attention-side entry points (no GPU needed)."""
import ctypes

import pytest

from gemm_decode_register_gb300 import build as b
from gemm_decode_register_gb300 import ops

A = 1 << 20  # an aligned fake address: validation fails before it is used


@pytest.fixture(scope="module")
def lib():
    b.build()
    return ops.load()


def kv(**kw):
    d = dict(k=A, v=A, k_scales=None, v_scales=None, block_table=A, page_stride=2 * 16 * 128, head_stride=16 * 128,
             token_stride=128, scale_page_stride=0, scale_head_stride=0, scale_token_stride=0, kv_fmt=0, num_pages=4,
             page_size=16, Hkv=2, D=128, table_stride=8)
    d.update(kw)
    c = ops._PagedKV()
    for name, v in d.items():
        setattr(c, name, v)
    return c


KV_FAULTS = [
    (dict(k=None), -1), (dict(v=None), -1), (dict(block_table=None), -1), (dict(num_pages=0), -1),
    (dict(page_size=0), -1), (dict(Hkv=0), -1), (dict(D=0), -1), (dict(table_stride=0), -1),
    (dict(page_stride=0), -1), (dict(head_stride=-128), -1), (dict(token_stride=0), -1),
    (dict(kv_fmt=2), -2), (dict(D=264), -2), (dict(D=100), -2), (dict(Hkv=5000), -2),
    (dict(kv_fmt=1), -1),  # no scales
    (dict(kv_fmt=1, k_scales=A, v_scales=A), -1),  # no scale strides
    (dict(kv_fmt=1, k_scales=A, v_scales=A, scale_page_stride=128, scale_head_stride=64, scale_token_stride=4, D=80), -2),
    (dict(k=A + 8), -3), (dict(v=A + 2), -3), (dict(token_stride=132), -3), (dict(block_table=A + 2), -3),
]


@pytest.mark.parametrize("kw,want", KV_FAULTS)
def test_cache_rejects(lib, kw, want):
    c = ctypes.byref(kv(**kw))
    assert lib.mx_kv_append(c, A, 0, 2048, A, A, A, 64, 128, A, 4, 2, 8, 0) == want
    assert lib.mx_paged_attn(c, A, 1024, 128, A, A, 0.1, 1, 0, None, A, None, 4, 2, 8, A, 1 << 40) == want


@pytest.mark.parametrize("i,value,want", [
    (1, 0, -1), (2, 5, -2), (3, 100, -1), (3, 2052, -3), (4, 0, -1), (5, 0, -1), (6, 0, -1), (8, 63, -1),
    (8, 130, -1), (9, 0, -1), (10, 0, -1), (11, 0, -1), (12, -1, -1), (12, 5000, -2), (13, 2, -1), (1, A + 4, -3),
    (9, A + 8, -3), (4, A + 1, -3), (11, 1 << 21, -2), (6, A + 4, -3)])
def test_append_rejects(lib, i, value, want):
    c = kv()
    args = [ctypes.byref(c), A, 0, 2048, A, A, A, 64, 128, A, 4, 2, 8, 0]
    args[i] = value
    assert lib.mx_kv_append(*args) == want


@pytest.mark.parametrize("i,value,want", [
    (1, 0, -1), (2, 0, -1), (3, -8, -1), (4, 0, -1), (5, 0, -1), (6, float("nan"), -1), (7, 2, -1), (8, -1, -1),
    (10, 0, -1), (12, 0, -1), (13, 0, -1), (14, 0, -1), (14, 7, -1), (14, 512, -2), (15, 0, -1), (16, 255, -1),
    (1, A + 8, -3), (2, 1028, -3), (10, A + 4, -3), (15, A + 128, -3), (9, A + 2, -3), (11, A + 1, -3)])
def test_attn_rejects(lib, i, value, want):
    c = kv()
    args = [ctypes.byref(c), A, 1024, 128, A, A, 0.1, 1, 0, None, A, None, 4, 2, 8, A, 1 << 40]
    args[i] = value
    assert lib.mx_paged_attn(*args) == want


def test_attn_null_workspace(lib):
    """Only where the stream's slot (16 MiB) is large enough, and with no size."""
    c = kv()
    assert lib.mx_paged_attn_workspace_size(4, 2, 8, 2, 128) <= 16 << 20 < lib.mx_paged_attn_workspace_size(4096, 1, 64, 2, 128)
    args = [ctypes.byref(c), A, 8192, 128, A, A, 0.1, 1, 0, None, A, None, 4096, 1, 64, None, 0]
    assert lib.mx_paged_attn(*args) == -1


@pytest.mark.parametrize("i,value,want", [
    (0, 0, -1), (1, 0, -1), (2, 2, -2), (3, 0, -1), (4, 0, -1), (6, 0, -1), (7, 0, -1), (8, 0, -1), (9, 63, -1),
    (9, 130, -1), (10, -1, -1), (12, 0, -1), (14, 4, -1), (0, A + 1, -3), (3, A + 2, -3), (4, A + 8, -3)])
def test_rope_rejects(lib, i, value, want):
    args = [A, A, 0, A, A, 64, 4, 8, 128, 128, 1024, 128, 1024, 128, 0]
    args[i] = value
    assert lib.mx_rope(*args) == want


@pytest.mark.parametrize("args,want", [((0, 1.0, A, 0, 4, 8), -1), ((A, 1.0, 0, 0, 4, 8), -1),
                                       ((A, 1.0, A, -1, 4, 8), -1), ((A, 1.0, A, 0, 0, 8), -1),
                                       ((A, 1.0, A, 0, 4, 0), -1), ((A + 4, 1.0, A, 0, 4, 8), -3)])
def test_rope_table_rejects(lib, args, want):
    assert lib.mx_rope_table(*args) == want


def test_attn_workspace_sizes(lib):
    f = lib.mx_paged_attn_workspace_size
    assert f(1, 1, 8, 8, 128) > 0 and f(1, 1, 8, 8, 128) % 256 == 0
    for bad in ((0, 1, 8, 8, 128), (1, 0, 8, 8, 128), (1, 1, 0, 8, 128), (1, 1, 7, 2, 128), (1, 1, 8, 8, 300),
                (1, 1, 256, 1, 128)):
        assert f(*bad) == 0


def test_frequencies():
    f, m = ops.rope_frequencies(8, 10000.0)
    assert f.tolist() == [1.0, 0.1, 0.01, 0.001] and m == 1.0
    with pytest.raises(ValueError):
        ops.rope_frequencies(7)
    with pytest.raises(ValueError):
        ops.rope_frequencies(8, scaling="other")
    y, my = ops.rope_frequencies(128, 10000.0, "yarn", factor=16.0, original_len=4096, low=1.0, high=32.0)
    p, _ = ops.rope_frequencies(128, 10000.0)
    assert y[0] == p[0] and abs(float(p[-1] / y[-1]) - 16) < 1e-9 and abs(my - 1.27725887) < 1e-7
    assert (y[:-1] > y[1:]).all()


def test_an_empty_rotation_table_is_refused(lib):
    """Its row 0 would be read for positions that are out of range; without a rotation there is no table."""
    c = kv()
    rope = [A, A, 0, A, A, 0, 4, 8, 128, 128, 1024, 128, 1024, 128, 0]
    append = [ctypes.byref(c), A, 0, 2048, A, A, A, 0, 128, A, 4, 2, 8, 0]
    assert lib.mx_rope(*rope) == -1
    assert lib.mx_kv_append(*append) == -1


@pytest.mark.parametrize("pages", [-1, 9])
def test_table_pages_within_a_row(lib, pages):
    c = ctypes.byref(kv(table_pages=pages))
    assert lib.mx_kv_append(c, A, 0, 2048, A, A, A, 64, 128, A, 4, 2, 8, 0) == -1
    assert lib.mx_paged_attn(c, A, 1024, 128, A, A, 0.1, 1, 0, None, A, None, 4, 2, 8, A, 1 << 40) == -1


def test_published_bands_are_the_defaults():
    """Left out, the band's upper end is each scaling's own: 4 turns (banded), 32 (YaRN)."""
    for scaling, high in (("yarn", 32.0), ("banded", 4.0)):
        kw = dict(factor=8.0, original_len=4096)
        f, m = ops.rope_frequencies(128, 10000.0, scaling, **kw)
        g, n = ops.rope_frequencies(128, 10000.0, scaling, low=1.0, high=high, **kw)
        h, _ = ops.rope_frequencies(128, 10000.0, scaling, low=1.0, high=36.0 - high, **kw)
        assert f.tolist() == g.tolist() and m == n and f.tolist() != h.tolist()
