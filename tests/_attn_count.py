"""Cases of the attention in which every token counts the same, so that one that is lost or taken twice shows.

A token's score is a whole number `level` (in powers of two), its value 2^-level in one column and 0 in the others: the column
gets 1 / sum of all 2^level from it, whatever its score.  Columns are shared by at most 64 tokens, so that a token is 1/64 of one,
four times the half step of a bf16 output."""
import torch

SHARED = 64  # tokens that a column counts


def level(t, spread):
    """Levels -spread .. spread that change within units, and over them."""
    return (t * 7 // 37 + t // 501) % (2 * spread + 1) - spread


def chunk(D):
    return SHARED * D


def column(t, head, D):
    return (t + 17 * head) % D


def counts(n, window, at, head, D, spread, lost=None):
    """What the columns of a sequence of n tokens get, of which those of [at, at + chunk) have values: float64 [D], and the sum
    of all weights.  `lost`: a token that is left out."""
    t = torch.arange(max(0, n - window) if window else 0, n)
    if lost is not None:
        t = t[t != lost]
    total = torch.pow(2.0, level(t, spread).double()).sum()
    t = t[(t >= at) & (t < at + chunk(D))]
    return torch.zeros(D, dtype=torch.float64).index_add_(0, column(t, head, D), torch.ones(len(t), dtype=torch.float64)) / total, total


# Of an output, relative: its rounding, and 2^-12 for all else.  Weights are off by 2^-20 (a score times a factor of 1 + 2^-23, up to
# 8 of it; an exponential's 2^-22) and by 2^-17 of their operands, powers of two as halves exactly; no chain of a sum in 32 bits is longer
# than a thousand additions of positive terms (a lane's of the units that its warp takes, then those of warps and CTAs): 2^-14, for the
# weighted sum and for the sum of weights.
def bound(want):
    return want * (torch.finfo(torch.bfloat16).eps / 2 + 2.0 ** -12)
