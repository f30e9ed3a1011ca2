"""Rotation of heads, and appends with it, against 64 bits (rotary_ref.py)."""
import math

import pytest
import torch

import rotary_ref as ref
from paged_kv_cache_255_gb300 import pagedattn as pa

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


def randn(*shape, seed=0, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def close(got, x, positions, theta, inter, **kw):
    want, slack = ref.rotated(x, positions, theta, inter, **kw)
    err = (got.double() - want).abs()
    assert got.dtype == torch.bfloat16 and got.shape == x.shape and torch.isfinite(got).all()
    assert (err <= ref.bound(want, slack)).all(), (err - ref.bound(want, slack)).max()


def positions_of(T, far=1 << 20, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randint(0, far, (T,), generator=gen, device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot_dim", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("norm", [False, True])
def test_rotation(rot_dim, inter, norm):
    T = 37
    q, k, pos = randn(T, 12, D), randn(T, 3, D, seed=1), positions_of(T)
    qw, kw = (randn(D, seed=2), randn(D, seed=3)) if norm else (None, None)
    R = pa.Rotary(rot_dim, interleaved=inter)
    before = q.clone(), k.clone()
    qo, ko = pa.rotate(q, k, pos, R, q_weight=qw, k_weight=kw)
    theta = ref.frequencies(rot_dim)
    close(qo, q, pos, theta, inter, weight=qw)
    close(ko, k, pos, theta, inter, weight=kw)
    assert torch.equal(q, before[0]) and torch.equal(k, before[1])
    if not norm:        # dims that are not rotated are the same bits
        assert torch.equal(qo[..., rot_dim:].view(torch.int16), q[..., rot_dim:].view(torch.int16))


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 0), (1, 0, 1), (1, 1, 1), (2, 5, 2), (3, 7, 1), (1, 64, 8), (997, 33, 3),
                                      (4096, 16, 8), (20000, 10, 2), (1, 1000, 7)])
def test_sizes(T, Hq, Hkv):
    q, k = (randn(T, Hq, D) if Hq else None), (randn(T, Hkv, D, seed=1) if Hkv else None)
    pos, w = positions_of(T), randn(D, seed=2)
    R = pa.Rotary(64)
    qo, ko = pa.rotate(q, k, pos, R, q_weight=w)
    theta = ref.frequencies(64)
    for x, o, wt in ((q, qo, w), (k, ko, None)):
        if x is None:
            assert o is None
        else:
            close(o, x, pos, theta, False, weight=wt)


@pytest.mark.parametrize("scaling,kw", [("linear", {}), ("ntk", {}), ("yarn", {}), ("banded", {}),
                                        ("yarn", dict(low=2.0, high=16.0)), ("banded", dict(low=0.5, high=9.0))])
@pytest.mark.parametrize("factor", [1.0, 8.0, 40.0])
def test_scalings(scaling, kw, factor):
    T = 64
    q, pos = randn(T, 4, D), positions_of(T)
    R = pa.Rotary(128, base=500000.0, scaling=scaling, factor=factor, original_context=8192, **kw)
    theta = ref.frequencies(128, 500000.0, scaling, factor, 8192.0, **kw)
    amp = 0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0
    assert abs(R.amplitude - amp) < 1e-6
    qo, _ = pa.rotate(q, None, pos, R)
    close(qo, q, pos, theta, False, amplitude=amp)


def test_given_frequencies_and_amplitude():
    theta = [0.0, 1.0, math.pi, 6.5, -0.25, 1e-12, 1000.125, 2.0 ** -30]
    q, pos = randn(9, 3, D), positions_of(9, 1 << 30)
    R = pa.Rotary(16, interleaved=True, frequencies=theta, amplitude=-0.75)
    qo, _ = pa.rotate(q, None, pos, R)
    close(qo, q, pos, theta, True, amplitude=-0.75)


def test_extreme_positions():
    pos = torch.tensor([0, 1, -1, 2**31 - 1, -2**31, 2**24 + 1, 1 << 20], device="cuda", dtype=torch.int32)
    q = randn(7, 8, D)
    for inter in (False, True):
        qo, _ = pa.rotate(q, None, pos, pa.Rotary(128, interleaved=inter))
        close(qo, q, pos, ref.frequencies(128), inter)
    assert torch.equal(qo[0], q[0])     # position 0 turns nothing


def test_rotation_by_position_is_relative():
    # q at p and k at p + d: the product depends on d alone
    q, k = randn(1, 1, D), randn(1, 1, D, seed=1)
    R = pa.Rotary(128)
    dots = []
    for p in (0, 1000, 10 ** 6, 2 * 10 ** 9):
        pos = torch.tensor([p], device="cuda", dtype=torch.int32)
        a, b = pa.rotate(q, None, pos, R)[0], pa.rotate(None, k, pos + 5, R)[1]
        dots.append((a.double() * b.double()).sum().item())
    # 128 products of values rounded to bf16: 2^-8 of each twice, |a| |b| at most
    slack = 2 * 2 ** -8 * q.double().norm().item() * k.double().norm().item() * 1.01
    assert max(dots) - min(dots) <= 2 * slack


def test_norm_alone_and_nothing():
    q, k, w = randn(50, 6, D), randn(50, 2, D, seed=1), randn(D, seed=2)
    qo, ko = pa.rotate(q, k, None, None, q_weight=w, eps=1e-2)
    close(qo, q, None, None, False, weight=w, eps=1e-2)
    assert torch.equal(ko, k)
    # every bit pattern passes, NaN and infinities among them
    bits = torch.arange(1 << 16, device="cuda", dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(64, 8, D)
    qo, _ = pa.rotate(bits, None, None, None)
    assert torch.equal(qo.view(torch.int16), bits.view(torch.int16))


def test_rows_do_not_reach_each_other():
    q, pos = randn(5, 6, D), positions_of(5)
    bad = q.clone()
    bad[2, 3, 7] = float("nan")
    bad[1, 0] = float("inf")
    R, w = pa.Rotary(96), randn(D, seed=2)
    want, got = pa.rotate(q, None, pos, R, q_weight=w)[0], pa.rotate(bad, None, pos, R, q_weight=w)[0]
    same = torch.ones(5, 6, dtype=torch.bool, device="cuda")
    same[2, 3] = same[1, 0] = False
    assert torch.equal(got[same], want[same]) and got[2, 3].isnan().all() and got[1, 0].isnan().all()


def test_zero_rows():
    q, pos = torch.zeros(3, 2, D, device="cuda", dtype=torch.bfloat16), positions_of(3)
    qo, _ = pa.rotate(q, None, pos, pa.Rotary(128), q_weight=randn(D))
    assert (qo == 0).all()
    # eps 0: 0 / 0, as the formula
    assert pa.rotate(q, None, pos, pa.Rotary(128), q_weight=randn(D), eps=0.0)[0].isnan().all()


def test_strides_and_in_place():
    T, Hq, Hkv = 33, 8, 2
    pos, R, w = positions_of(T), pa.Rotary(64, interleaved=True), randn(D, seed=2)
    qkv = randn(T, Hq + 2 * Hkv, D)
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    want_q, want_k = pa.rotate(q.contiguous(), k.contiguous(), pos, R, q_weight=w)
    # parts of a projection
    got = pa.rotate(q, k, pos, R, q_weight=w)
    assert torch.equal(got[0], want_q) and torch.equal(got[1], want_k)
    # per KV head: g query heads, then its key and value head
    per = torch.cat([q.view(T, Hkv, -1, D), k[:, :, None], v[:, :, None]], 2)
    pk = per[:, :, -2]
    assert pk.stride(1) == 6 * D
    assert torch.equal(pa.rotate(None, pk, pos, R)[1], want_k)
    # heads outermost, a broadcast row
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(pa.rotate(qt, None, pos, R, q_weight=w)[0], want_q)
    one = q[:, :1].expand(T, Hq, D)
    assert torch.equal(pa.rotate(one, None, pos, R, q_weight=w)[0][:, 5], want_q[:, 0])
    # strided outputs, in place
    keep = qkv.clone()
    out = torch.full((Hq, T, 2 * D), 3.0, device="cuda", dtype=torch.bfloat16)
    pa.rotate(q, None, pos, R, q_weight=w, q_out=out[..., :D].transpose(0, 1))
    assert torch.equal(out[..., :D].transpose(0, 1), want_q) and (out[..., D:] == 3).all()
    assert pa.rotate(q, k, pos, R, q_weight=w, q_out=q, k_out=k)[0] is q
    assert torch.equal(q, want_q) and torch.equal(k, want_k) and torch.equal(v, keep[:, Hq + Hkv:])


def test_stream_graph_and_threads():
    T = 300
    q, k, pos, R = randn(T, 8, D), randn(T, 2, D, seed=1), positions_of(T), pa.Rotary(128)
    want = pa.rotate(q, k, pos, R)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pa.rotate(q, k, pos, R, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    outs = torch.empty_like(q), torch.empty_like(k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.rotate(q, k, pos, R, q_out=outs[0], k_out=outs[1])
    q.copy_(randn(T, 8, D, seed=9))
    pos.add_(77)
    g.replay()
    want = pa.rotate(q, k, pos, R)
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_offsets_past_32_bits():
    # 2.2e9 elements between the first and the last token
    T, ts = 4, 1 << 29
    big = torch.empty((T - 1) * ts + 3 * D, device="cuda", dtype=torch.bfloat16)
    q = big.as_strided((T, 3, D), (ts, D, 1))
    x, pos, R = randn(T, 3, D), positions_of(T), pa.Rotary(128)
    q.copy_(x)
    pa.rotate(q, None, pos, R, q_out=q)
    assert torch.equal(q, pa.rotate(x, None, pos, R)[0])


# -- append ------------------------------------------------------------------------

def pools(NB, bs, Hkv, hm, fill=5.0):
    shape = (NB, Hkv, bs, D) if hm else (NB, bs, Hkv, D)
    return [torch.full(shape, fill + i, device="cuda", dtype=torch.bfloat16) for i in range(2)]


@pytest.mark.parametrize("hm", [False, True])
@pytest.mark.parametrize("bs,T,Hq,Hkv,rot,inter,norm", [
    (16, 1, 16, 8, 128, False, True), (16, 60, 16, 8, 128, False, False), (64, 333, 12, 3, 96, True, True),
    (256, 77, 1, 1, 16, True, False), (32, 5000, 8, 2, 64, False, True), (128, 9, 0, 5, 128, False, True)])
def test_append(bs, T, Hq, Hkv, rot, inter, norm, hm):
    NB = 2 + -(-T // bs) * 2
    kc, vc = pools(NB, bs, Hkv, hm)
    qkv, pos = randn(T, Hq + 2 * Hkv, D), positions_of(T)
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    # values of any kind are copied bit by bit
    v[::3] = torch.randint(-32768, 32768, v[::3].shape, device="cuda").to(torch.int16).view(torch.bfloat16)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    slots = torch.randperm(NB * bs, generator=gen, device="cuda")[:T].contiguous()
    if T > 4:
        slots[::5] = -1
    qw, kw = (randn(D, seed=2), randn(D, seed=3)) if norm else (None, None)
    R = pa.Rotary(rot, interleaved=inter)
    got = pa.append_kvcache(q if Hq else None, k, v, kc, vc, slots, pos, R, q_weight=qw, k_weight=kw, head_major=hm)
    want_q, want_k = pa.rotate(q if Hq else None, k, pos, R, q_weight=qw, k_weight=kw)
    close(want_k, k, pos, ref.frequencies(rot), inter, weight=kw)
    assert (got is None) == (Hq == 0) and (Hq == 0 or torch.equal(got, want_q))
    kc2, vc2 = pools(NB, bs, Hkv, hm)
    pa.store_kvcache(want_k.contiguous(), v.contiguous(), kc2, vc2, slots, head_major=hm)
    assert torch.equal(kc.view(torch.int16), kc2.view(torch.int16))
    assert torch.equal(vc.view(torch.int16), vc2.view(torch.int16))
    assert pa.take_device_error() == 0


def test_append_bad_slots_are_skipped_and_recorded():
    kc, vc = pools(4, 16, 2, False)
    q, k, v = randn(4, 4, D), randn(4, 2, D, seed=1), randn(4, 2, D, seed=2)
    slots = torch.tensor([64, -2, 2**40, 63], device="cuda")
    R, pos = pa.Rotary(128), positions_of(4)
    out = pa.append_kvcache(q, k, v, kc, vc, slots, pos, R)
    assert pa.take_device_error() == 3
    assert torch.equal(out, pa.rotate(q, None, pos, R)[0])
    assert torch.equal(vc[3, 15], v[3]) and (vc.view(64, 2, D)[:63] == 6).all() and (kc.view(64, 2, D)[:63] == 5).all()


def test_append_without_rotation_is_the_store():
    kc, vc = pools(9, 16, 2, True)
    kc2, vc2 = pools(9, 16, 2, True)
    k, v = randn(50, 2, D), randn(50, 2, D, seed=1)
    slots = torch.randperm(144, device="cuda")[:50].contiguous()
    assert pa.append_kvcache(None, k, v, kc, vc, slots, None, None, head_major=True) is None
    pa.store_kvcache(k, v, kc2, vc2, slots, head_major=True)
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_append_past_32_bits():
    # 4.6 GB a pool; rows at both ends
    NB, bs, Hkv = 140001, 16, 8
    for hm in (False, True):
        kc, vc = (torch.zeros((NB, Hkv, bs, D) if hm else (NB, bs, Hkv, D), device="cuda", dtype=torch.bfloat16)
                  for _ in range(2))
        k, v, pos = randn(3, Hkv, D), randn(3, Hkv, D, seed=1), positions_of(3)
        slots = torch.tensor([16, NB * bs - 1, NB * bs - 17], device="cuda")
        pa.append_kvcache(None, k, v, kc, vc, slots, pos, pa.Rotary(128), head_major=hm)
        want = pa.rotate(None, k, pos, pa.Rotary(128))[1]
        for i, (b, r) in enumerate([(1, 0), (NB - 1, 15), (NB - 2, 15)]):
            at = (b, slice(None), r) if hm else (b, r)
            assert torch.equal(kc[at], want[i]) and torch.equal(vc[at], v[i])
        assert kc.count_nonzero() <= 3 * Hkv * D and pa.take_device_error() == 0
        del kc, vc


def test_empty_batches():
    e = torch.empty(0, 4, D, device="cuda", dtype=torch.bfloat16)
    none = torch.empty(0, device="cuda", dtype=torch.int32)
    qo, ko = pa.rotate(e, e[:, :2], none, pa.Rotary(128))
    assert qo.shape == (0, 4, D) and ko.shape == (0, 2, D)
    kc, vc = pools(3, 16, 2, False)
    pa.append_kvcache(e, e[:, :2], e[:, :2], kc, vc, none.long(), none, pa.Rotary(128))
    assert (kc == 5).all() and (vc == 6).all()
