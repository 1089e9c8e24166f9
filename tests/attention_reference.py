"""Plain 64-bit forms of the attention operators and the error bounds their tests use.

Bounds (relative half steps: bf16 2^-8, fp16 2^-11, E4M3 2^-4 and 2^-10 absolute in its
subnormals; fp32 sums and products are counted with 2^-20 of the sum of magnitudes, which covers
a few hundred roundings of 2^-24 that partly cancel and the 2^-22 of the base-2 exponential):

  a score's error      d = 2^-20 (1 + scale sum_i |q_i k_i|)
  a weight's           2 d, plus its rounding for the product with v (half a step of its type; a
                       weight in fp16's subnormals is off by 2^-25 of the largest)
  an output's          the weights' error times sum_j p_j |v_j|, once more for the division by
                       their sum, plus its own rounding 2^-8 |out|
  lse's                d + 2^-22 |lse|
"""
import torch

HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "split": 2.0 ** -16}


def attend64(q, k, v, scale, weights):
    """One query row set against its keys: q [rows, d], k, v [keys, d] or [rows, keys allowed] masks by
    the caller.  Returns (out, lse, tol_out, tol_lse) in float64; no keys: zeros and -inf."""
    q, k, v = q.double(), k.double(), v.double()
    if k.shape[0] == 0:
        z = torch.zeros((q.shape[0], v.shape[1]), dtype=torch.float64, device=q.device)
        lse = torch.full((q.shape[0],), -float("inf"), dtype=torch.float64, device=q.device)
        return z, lse, z, torch.zeros_like(lse)
    s = (q @ k.T) * scale
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    out = p @ v
    d = 2.0 ** -20 * (1.0 + abs(scale) * (q.abs() @ k.abs().T).amax(1))
    spread = p @ v.abs()
    step = HALF_STEP[weights]
    tol = 2.0 ** -8 * out.abs() + 2.0 * (2.0 * d[:, None] + step) * spread
    if weights == "fp16":
        tol = tol + k.shape[0] * 2.0 ** -25 * v.abs().amax(0)
    return out, lse, tol + 1e-30, d + 2.0 ** -22 * lse.abs()


def causal64(q, k, v, scale, weights):
    """attend64 for row i over keys 0..i (q, k, v [rows, d])."""
    q, k, v = q.double(), k.double(), v.double()
    n = q.shape[0]
    keep = torch.ones((n, n), dtype=torch.bool, device=q.device).tril()
    s = torch.where(keep, (q @ k.T) * scale, torch.tensor(-float("inf"), dtype=torch.float64, device=q.device))
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    big = torch.where(keep, q.abs() @ k.abs().T, torch.zeros((), dtype=torch.float64, device=q.device)).amax(1)
    d = 2.0 ** -20 * (1.0 + abs(scale) * big)
    out = p @ v
    tol = 2.0 ** -8 * out.abs() + 2.0 * (2.0 * d[:, None] + HALF_STEP[weights]) * (p @ v.abs())
    return out, lse, tol + 1e-30, d + 2.0 ** -22 * lse.abs()


def rotate64(x, positions, inv_freq):
    """x [tokens, heads, d] rotated to its positions in 64 bits, and the bound of an fp32 rotation
    (before the rounding to the output's type)."""
    half = inv_freq.numel()
    x = x.double()
    theta = positions.double()[:, None] * inv_freq.double()
    c, s = theta.cos()[:, None], theta.sin()[:, None]
    a, b = x[..., :half], x[..., half:2 * half]
    out = torch.cat([a * c - b * s, b * c + a * s, x[..., 2 * half:]], -1)
    near = 2.0 ** -21 * (a.abs() + b.abs())
    return out, torch.cat([near, near, torch.zeros_like(x[..., 2 * half:])], -1)


def assert_within(got, want, tol, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    off = (got - want).abs() - tol
    worst = off.max().item() if off.numel() else -1.0
    assert worst <= 0, f"{what}: {int((off > 0).sum())} of {off.numel()} values off, by up to {worst:.3e} over the bound"
