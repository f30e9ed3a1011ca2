"""Rotations by high frequencies at the ends of 32-bit positions, against angles in exact
fractions (rotary_exact)."""
import math
from fractions import Fraction

import pytest
import torch

import rotary_exact as exact
import rotary_ref as ref
from paged_kv_cache_255_gb300 import pagedattn as pa

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _lib(pa_lib):
    return pa_lib


@pytest.mark.parametrize("inter", [False, True])
def test_given_frequencies_at_the_ends_of_the_positions(inter):
    f = [2.0 ** 20, -(2.0 ** 20) + 0.7, 12345.678, 1.0, -math.pi, 1e-4, 2.0 ** -31, 333333.25]
    positions = [2 ** 31 - 1, -(2 ** 31), 2 ** 31 - 12345, -1, 1, 0, 2 ** 24 + 1, -987654321]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    q = torch.randn(len(positions), 8, D, generator=gen, device="cuda").bfloat16()
    got, _ = pa.rotate(q, None, torch.tensor(positions, device="cuda", dtype=torch.int32),
                       pa.Rotary(16, interleaved=inter, frequencies=f))
    # angles to 2^-53 turns; bound() counts the roundings of what the kernel does
    angle = torch.tensor([[2 * math.pi * float(exact.turns(x, Fraction(p))) for x in f] for p in positions],
                         dtype=torch.float64, device="cuda")[:, None]
    i = torch.arange(8, device="cuda")
    ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + 8)
    want, slack = q.double(), q.double().abs()
    a, b = want[..., ia].clone(), want[..., ib].clone()
    want[..., ia], want[..., ib] = a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()
    slack[..., ia] = slack[..., ib] = a.abs() + b.abs()
    err = (got.double() - want).abs()
    assert (err <= ref.bound(want, slack)).all(), (err - ref.bound(want, slack)).max()
    assert torch.equal(got[..., 16:], q[..., 16:])
