"""The bounds of tile_codes on the CPU: a right computation with its roundings
stays within them, and one that loses, doubles or swaps 16 keys does not. The
mistakes are planted here, in the model."""
import pytest
import torch

import tile_codes as tc

SCALE = 128 ** -0.5


def rounded(q, k, v, scale, keep=None):
    """Attention with its weights and output rounded to bf16, over the rows `keep`
    (any list of row numbers) of k and v."""
    if keep is not None:
        k, v = k[keep], v[keep]
    s = q.double() @ k.double().T * scale
    p = torch.exp(s - s.max(-1, keepdim=True).values)
    return ((p.bfloat16().double() @ v.double()) / p.sum(-1, keepdim=True)).bfloat16()


def mistakes(t):
    """Row lists with 16 keys lost, twice, or replaced by those a ring of 2 or 3
    tiles of 128 before, near both ends and inside."""
    for at in (0, 16 * (t // 16 // 2) + 16, t - 16):
        rows = torch.arange(t)
        yield torch.cat([rows[:at], rows[at + 16:]])
        yield torch.cat([rows, rows[at:at + 16]])
        for back in (256, 384):
            if at >= back:
                stale = rows.clone()
                stale[at:at + 16] -= back
                yield stale


@pytest.mark.parametrize("tokens", [2032, 9000, 48000])
def test_coded_keys_show_every_mistake(tokens):
    tokens -= tokens % 16
    k, v = tc.coded_rows(tokens)
    q = torch.zeros(tc.K_PERIOD + 1, 128, dtype=torch.bfloat16)
    q[torch.arange(tc.K_PERIOD), torch.arange(tc.K_PERIOD)] = 400.0         # the last row stays 0
    o, A = tc.attend(q, k, v, SCALE)
    bound = tc.element_bound(o, A)
    assert ((rounded(q, k, v, SCALE).double() - o).abs() <= bound).all()
    for keep in mistakes(tokens):
        off = (rounded(q, k, v, SCALE, keep).double() - o).abs()
        assert (off > 2 * bound).any()


@pytest.mark.parametrize("tokens", [4000, 16000, 48000])
def test_the_row_bound_shows_every_mistake(tokens):
    gen = torch.Generator()
    gen.manual_seed(tokens)
    k, v = (torch.randn(tokens, 128, generator=gen).bfloat16() for _ in range(2))
    q = torch.randn(8, 128, generator=gen).bfloat16()
    o, _ = tc.attend(q, k, v, SCALE)
    assert (tc.row_error(rounded(q, k, v, SCALE), o) <= tc.ROW_REL).all()
    for keep in mistakes(tokens):
        assert (tc.row_error(rounded(q, k, v, SCALE, keep), o) > tc.ROW_REL).any()
