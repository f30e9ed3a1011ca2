"""Decode over trees with starts that fall: whatever is computed stays within the buffers."""
import pytest
import torch

from paged_kv_cache_255_gb300 import pagedattn as pa
from test_gpu_tree import Batch

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _lib(pa_lib):
    return pa_lib


@pytest.fixture(autouse=True)
def _no_error_left():
    pa.take_device_error()
    yield
    pa.take_device_error()


def guarded(n, dtype, fill, around=1 << 16):
    """n elements in the middle of a larger buffer, and what checks its other elements."""
    big = torch.full((n + 2 * around,), fill, dtype=dtype, device="cuda")

    def untouched():
        return bool((big[:around] == fill).all() and (big[around + n:] == fill).all())
    return big[around:around + n], untouched


# Every second sequence has all rows of the batch: 256 units over 131072 key tiles each. Their
# places pass 2^31, to a negative number in 32 bits or to a small one: nothing is computed.
@pytest.mark.parametrize("S", [160, 256])
def test_places_past_32_bits(S):
    T, Hq, bs, blocks = 4096, 16, 256, 1 << 16
    full = S // 2
    assert full * 256 * (blocks * bs // 128 + 3) >= 2 ** 31
    i32 = dict(device="cuda", dtype=torch.int32)
    q = torch.randn(T, Hq, D, device="cuda").bfloat16()
    k, v = (torch.randn(3, bs, 1, D, device="cuda").bfloat16() for _ in range(2))
    tables = torch.ones(S, blocks, **i32)
    lens = torch.full((S,), blocks * bs, **i32)
    starts = (torch.arange(S + 1, **i32) % 2) * T
    mask = torch.ones(T, 1, device="cuda", dtype=torch.int64)
    out, out_same = guarded(q.numel(), torch.bfloat16, 77.0)
    ws, ws_same = guarded(pa.decode_tree_workspace_size(Hq, 1), torch.uint8, 3)
    pa.decode_tree(q, k, v, tables, lens, starts, mask, 0.1, out=out.view(q.shape), workspace=ws)
    assert pa.take_device_error() == 0
    assert out_same() and ws_same() and (out == 77.0).all()
    # the same buffers again, with starts in order
    few = [0, 5, 5, 40]
    pa.decode_tree(q[:40], k, v, tables[:3, :2].contiguous(), lens[:3], torch.tensor(few, **i32), mask[:40], 0.1,
                   out=out.view(q.shape)[:40], workspace=ws)
    assert pa.take_device_error() == 0 and out_same() and ws_same()
    assert (out.view(q.shape)[:40] != 77.0).any(2).all() and (out.view(q.shape)[40:] == 77.0).all()


def test_padded_starts_are_empty_sequences():
    """Starts padded with zeros behind the last sequence's: those sequences have no rows."""
    b = Batch([300, 40, 0, 0, 0], [9, 33, 0, 0, 0], 16, 4)
    want = b.check().clone()
    b.starts[3:] = 0
    out = torch.full_like(b.q, 77.0)
    b.run(out=out)
    assert pa.take_device_error() == 0 and torch.equal(out, want)


@pytest.mark.parametrize("starts", [[0, 7, 3, 18], [18, 3, 0, -4], [-5, 3, 7, 900], [5, 5, 5, 5], [0, 18, 0, 18],
                                    [2 ** 31 - 1, -(2 ** 31), 2 ** 31 - 1, 0]])
@pytest.mark.parametrize("Hq,Hkv,hm", [(8, 2, False), (33, 3, True)])
def test_starts_of_any_kind_change_nothing_around_the_buffers(starts, Hq, Hkv, hm):
    b = Batch([30, 300, 20], [5, 9, 4], Hq, Hkv, hm=hm)
    out, out_same = guarded(b.q.numel(), torch.bfloat16, 77.0)
    ws, ws_same = guarded(pa.decode_tree_workspace_size(Hq, Hkv), torch.uint8, 255)
    inputs = [x.clone() for x in (b.tables, b.lens, b.mask)]
    kv = [x.view(torch.int16).clone() for x in (b.q, b.k, b.v)]
    b.starts.copy_(torch.tensor(starts, dtype=torch.int32))
    for _ in range(2):      # also over what a call has left in the workspace
        b.run(out=out.view(b.q.shape), workspace=ws)
        assert pa.take_device_error() in (0, 4)
        assert out_same() and ws_same()
    assert all(torch.equal(x, y) for x, y in zip((b.tables, b.lens, b.mask), inputs))
    assert all(torch.equal(x.view(torch.int16), y) for x, y in zip((b.q, b.k, b.v), kv))


@pytest.mark.parametrize("hm", [False, True])
def test_a_chain_is_prefill(hm):
    """A chain's rows see what a prompt's last rows see."""
    b = Batch([300, 1, 64, 0], [4, 20, 130, 33], 16, 8, hm=hm, masks=lambda r, n: [(2 << i) - 1 for i in range(n)])
    b.check()
    b.check(pa.prefill(b.q, b.k, b.v, b.tables, b.lens, b.starts, b.scale, head_major=hm))
