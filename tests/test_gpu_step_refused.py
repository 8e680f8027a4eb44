"""A step that the pool cannot supply, with the append and the attention right behind it: they read the lengths as soon as they
start, so the remap's -1 have to be there by then."""
import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page,D,S", [(16, 64, 4), (32, 128, 40), (7, 40, 5)])
def test_a_refused_step_touches_no_cache(page, D, S):
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    i32 = dict(dtype=torch.int32, device="cuda")
    P, Hkv, Hq = 3 * S, 2, 4
    pool = ops.PagePool(P)
    tables = [torch.zeros((S, 5), **i32) for _ in range(2)]
    none, ident = torch.full((S,), -1, **i32), torch.arange(S, **i32)
    one_each, rows = torch.arange(S + 1, **i32), torch.randn((S, (Hq + 2 * Hkv) * D), device="cuda").bfloat16()
    kvs = [ops.PagedKV.empty(P, Hkv, page, D, t) for t in tables]
    kv = kvs[0]
    kvs[1] = ops.PagedKV(kv.k, kv.v, tables[1])
    kv.k.normal_()
    kv.v.normal_()
    n0, _ = ops.kv_remap(pool, page, tables[1], none, none, tables[0], torch.full((S,), 2 * page, **i32))
    big = torch.full((S,), 2 * page, **i32)  # two pages more for each: S are left
    for fits in (False, True, False):
        old = kv.k.clone(), kv.v.clone()
        # (the same tensor held good lengths just before)
        n1, _ = ops.kv_remap(pool, page, tables[0], n0, ident, tables[1], 0)
        n1, _ = ops.kv_remap(pool, page, tables[0], n0, ident, tables[1], 1 if fits else big, kv_len_out=n1)
        q = ops.kv_append(kvs[1], rows, one_each, n1, Hq, None)
        out = ops.paged_attn(kvs[1], q, one_each, n1)
        error = ops.device_error()
        if fits:
            assert error == 0 and (n1 == 2 * page + 1).all() and out.isfinite().all()
            n1, _ = ops.kv_remap(pool, page, tables[1], n1, ident, tables[0], 0, keep=n0)  # back again
            assert torch.equal(n1, n0) and int(pool.count) == S
        else:
            assert error == 0x10 | 0x8 and (n1 == -1).all()
            assert torch.equal(kv.k, old[0]) and torch.equal(kv.v, old[1])
            assert q.isnan().all() and (out == 0).all()
