"""64-bit attention under any mask, with the error bounds of attention_reference.py."""
import torch

from attention_reference import HALF_STEP


def masked64(q, k, v, scale, keep, weights):
    """q [rows, d], k, v [keys, d], keep [rows, keys] bool.  Returns (out, lse, tol_out, tol_lse) in float64; a row
    that keeps nothing: zeros and -inf.  What is masked may hold anything."""
    q, k, v = q.double(), k.double(), v.double()
    zero = torch.zeros((), dtype=torch.float64, device=q.device)
    minus = zero - float("inf")
    s = torch.where(keep, (q @ k.T) * scale, minus)
    lse = torch.logsumexp(s, 1)
    some = keep.any(1)
    p = torch.where(keep, torch.exp(s - torch.where(some, lse, zero)[:, None]), zero)
    seen = keep.any(0)  # rows of v that nobody keeps would make NaN of 0 * NaN
    v = torch.where(seen[:, None], v, zero)
    out, spread = p @ v, p @ v.abs()
    big = torch.where(keep, q.abs() @ k.abs().T, zero).amax(1) if k.shape[0] else torch.zeros_like(lse)
    d = 2.0 ** -20 * (1.0 + abs(scale) * big)
    tol = 2.0 ** -8 * out.abs() + 2.0 * (2.0 * d[:, None] + HALF_STEP[weights]) * spread
    if weights == "fp16" and k.shape[0] > 0:
        tol = tol + k.shape[0] * 2.0 ** -25 * v.abs().amax(0)
    tol_lse = torch.where(some, d + 2.0 ** -22 * lse.abs(), zero)
    return out, lse, tol + 1e-30, tol_lse


def window_keep(rows, keys, window, sinks):
    """Which of the key positions a row position attends to."""
    i, j = rows[:, None], keys[None, :]
    return (j <= i) & ((i - j < window) | (j < sinks))
