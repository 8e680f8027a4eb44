"""kv_remap's parent as beams come: [B][W], and a part of wider rows, which is flattened into a tensor of its own."""
import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,W,wide", [(2, 3, 3), (2, 3, 6), (5, 64, 128)])
def test_parents_in_rows(B, W, wide, monkeypatch):
    """The same step as with parents in a row, and no output lies where the parents are read."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    i32 = dict(dtype=torch.int32, device="cuda")
    S, page = B * W, 4
    g = torch.Generator(device="cuda").manual_seed(W)
    full = torch.randint(0, S, (B, wide), generator=g, **i32)
    parent, lib, seen = full[:, :W], ops.load(), []

    class Lib:
        def __getattr__(self, name):
            f = getattr(lib, name)
            return f if name != "mx_kv_remap" else lambda *a: (seen.append(a), f(*a))[1]

    results = []
    for p in (parent, parent.flatten().clone()):
        pool, tables = ops.PagePool(20 * S), [torch.zeros((S, 8), **i32) for _ in range(2)]
        n, _ = ops.kv_remap(pool, page, tables[1], torch.full((S,), -1, **i32), torch.full((S,), -1, **i32), tables[0],
                            torch.arange(S, **i32) % 17)
        with monkeypatch.context() as m:
            m.setattr(ops, "load", Lib)
            n, copies = ops.kv_remap(pool, page, tables[0], n, p, tables[1], 1)
        k = int(copies[0, 0])
        results.append([n.tolist(), tables[1].tolist(), pool.state.tolist(), copies[:1 + k].tolist()])
        args = seen[-1]
        kv_len_out, at, listed = args[10], args[12], args[16]
        for out, size in ((kv_len_out, 4 * S), (listed, 16 * (1 + S))):
            assert out + size <= at or at + 4 * S <= out
    assert results[0] == results[1] and ops.device_error() == 0
