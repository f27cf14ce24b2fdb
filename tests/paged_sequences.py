"""Whole sequences for tests of the paged calls together: the tokens' q, k and v,
and attention over a sequence laid out plainly, with its bounds (paged_cases.py)."""

import numpy as np
import torch

import oracle
from paged_cases import attention_bounds

LENGTHS = [75, 20, 133]
STEPS = [[50, 20, 100], [25, 0, 31], [0, 0, 1], [0, 0, 1]]  # tokens of each request in each step
DECODE_ROWS = [(2, 131), (2, 132)]  # (request, position) of the steps of one token


def sequences(Hq, Hkv, D, seed):
    """bf16 [tokens, Hq + 2 Hkv, D] of each request."""
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn((n, Hq + 2 * Hkv, D), generator=gen).to(torch.bfloat16) for n in LENGTHS]


def bf16(x):
    return torch.tensor(x).to(torch.bfloat16).double().numpy()


def turned(x, Hq, Hkv, turns):
    """q and k of a sequence in 64 bits, turned."""
    y = x.double().numpy()
    pos = np.arange(len(y))
    return (oracle.rope_rotate(y[:, :Hq], pos, turns, False, 1.0),
            oracle.rope_rotate(y[:, Hq:Hq + Hkv], pos, turns, False, 1.0))


def attend(q, k, v):
    """out and lse of a sequence's causal attention, and their bounds: of numbers as they are in the cache."""
    n, _, D = q.shape
    out, lse, A, S, count, _ = oracle.paged_attention(q, k[None], v[None], np.zeros((1, 1), int), [0, n], [n],
                                                      D ** -0.5, 0)
    tol, lse_tol = attention_bounds(out, lse, A, S, count, D)
    return out, lse, tol, lse_tol
