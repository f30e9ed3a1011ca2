"""Inputs for which every group of 16 keys shows in attention's output, at any
length, and a bound on the relative error of a row.

Coded keys. The keys of group g (tokens 16 g .. 16 g + 15) are the unit vector of
dim g mod 127, the values that of dim 5 g mod 113. A query of weight w on dim j
scores w on the groups g = j mod 127 and 0 on the others; with w so large that
the others' weights vanish the output is, on each dim d, the share of those
groups whose values stand there. Of 24 groups (48,000 tokens) a lost, doubled or
stale one moves a share by 1/24 or more, where rounding moves it by 3 * 2^-8
at most. With w = 0 every key counts the same and the output is the histogram of
the values alone. Values are positive, so nothing cancels in a bound on the sum.

Relative error of a row, for random values. A weight and the output are each
rounded to bf16: a relative error of at most 2^-8, uniform within its step, with
a root mean square of 2^-8 / sqrt(3) times the mean of 1 / m over a mantissa in
[1, 2), which is ln 2: 0.00156. Over many keys with independent values the
weights' errors give a vector of that length relative to the output's, the output's
own rounding another: 0.0022 together. Over the 128 dims of a row the length
spreads by 1/16 of itself; 8 times that above is 0.0034, and the bound is 0.004.
Losing 16 keys of 48,000 moves a row by sqrt(16 / 48000) = 0.018."""
import torch

K_PERIOD, V_PERIOD, V_STEP = 127, 113, 5
ROW_REL = 0.004


def k_dim(group):
    return group % K_PERIOD


def v_dim(group):
    return V_STEP * group % V_PERIOD


def coded_rows(tokens, device="cpu"):
    """(k, v) of every token, [tokens, 128] in bf16."""
    g = torch.arange(tokens, device=device) // 16
    k, v = (torch.zeros(tokens, 128, dtype=torch.bfloat16, device=device) for _ in range(2))
    k.scatter_(1, k_dim(g)[:, None], 1)
    v.scatter_(1, v_dim(g)[:, None], 1)
    return k, v


def attend(q, k, v, scale):
    """(o, sum p |v|) in 64 bits for rows q [n, 128] over k, v [t, 128]."""
    p = torch.softmax(q.double() @ k.double().T * scale, -1)
    return p @ v.double(), p @ v.double().abs()


def element_bound(o, A):
    """Weights rounded to bf16 (2^-8 of A), their sum taken of the rounded or the
    exact ones and the output rounded (2^-8 |o| each), and a tenth for what is computed
    in 32 bits."""
    return 1.1 * 2 ** -8 * (A + 2 * o.abs())


def row_error(got, o):
    """Relative L2 error of each row (last axis)."""
    return (got.double() - o).norm(dim=-1) / o.norm(dim=-1)
