"""Plain float64 implementations of the 8-bit latent cache and of attention over listed rows and
drafted trees, and the error bounds the GPU tests hold the kernels to.

Everything here is elementary torch arithmetic in float64 (integers for bit patterns); nothing
calls the library.
"""
from __future__ import annotations

import math

import torch

GROUP = 128
E4M3_MAX = 448.0


# ----------------------------------------------------------------------------- quantisation
def quantise_rows(x: torch.Tensor):
    """x float64 [..., k] -> (E4M3 values float64, exponents int64 of the scales).

    Smallest e in -100..100 with amax <= 448 * 2^e over the finite values (0 where amax is 0); values
    rounded to the nearest E4M3 number, ties to the even mantissa, magnitudes held to 448; NaN stays."""
    fin = torch.isfinite(x)
    amax = torch.where(fin, x.abs(), torch.zeros_like(x)).amax(dim=-1)
    e = torch.full(amax.shape, -100, dtype=torch.int64)
    for k in range(-100, 100):                     # the definition, literally
        e = torch.where(amax > E4M3_MAX * 2.0 ** k, torch.full_like(e, k + 1), e)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    y = x * torch.exp2(-e.double())[..., None]
    mag = y.abs().clamp(max=E4M3_MAX)
    # spacing of E4M3 numbers: 2^(exponent - 3), exponents from -6 up (subnormals share -6's)
    exp = torch.floor(torch.log2(mag.clamp(min=2.0 ** -6)))
    step = torch.exp2(exp - 3)
    q = torch.round(mag / step) * step             # torch.round: ties to even
    return torch.where(torch.isnan(x), x, torch.copysign(q.clamp(max=E4M3_MAX), x)), e


def grouped(x: torch.Tensor):
    """[..., d] -> [..., groups, 128], zeros behind the last dim."""
    d = x.shape[-1]
    g = -(-d // GROUP)
    return torch.nn.functional.pad(x, (0, g * GROUP - d)).view(*x.shape[:-1], g, GROUP)


def quantise_latent(x: torch.Tensor, d_latent: int):
    """bf16 rows [..., d] -> (E4M3 values [..., d_latent], scales [..., groups]) in float64."""
    g = grouped(x[..., :d_latent].double())
    q, e = quantise_rows(g)
    scale = torch.exp2(e.double())
    scale = torch.where(torch.isnan(g).any(dim=-1), torch.full_like(scale, math.nan), scale)
    return q.reshape(*x.shape[:-1], -1)[..., :d_latent], scale


def code_values(codes: torch.Tensor) -> torch.Tensor:
    """uint8 E4M3 codes -> float64, from the bit definition."""
    c = codes.to(torch.int64)
    sign = torch.where(c >= 128, -1.0, 1.0).double()
    exp, man = (c >> 3) & 15, c & 7
    mag = torch.where(exp == 0, man.double() * 2.0 ** -9, (8 + man).double() * torch.exp2(exp.double() - 10))
    return torch.where((c & 127) == 127, torch.full_like(mag, math.nan), sign * mag)


def dequantised(codes, scales, rope):
    """float64 rows [..., d_latent + d_rope] of an 8-bit cache."""
    d = codes.shape[-1]
    s = scales.double().repeat_interleave(GROUP, dim=-1)[..., :d]
    return torch.cat([code_values(codes) * s, rope.double()], dim=-1)


# ----------------------------------------------------------------------------- attention
def path_of(parents, i: int):
    """Nodes on node i's path (i first), or None for an absent node or one below it. ``parents``: a list."""
    path = []
    while True:
        path.append(i)
        v = parents[i]
        if v < -1 or v >= i:
            return None
        if v == -1:
            return path
        i = v


def attend(q, rows, d_latent: int, scale: float):
    """q float64 [H, d], rows float64 [k, d] -> (out [H, d_latent], lse [H], bound of out, bound of lse).

    The bounds, from the arithmetic the kernel does:
    * a logit: bf16 products are exact in fp32; the tensor core adds 16 products at a time into an fp32
      accumulator, at most 36 steps of one rounding or truncation (2^-23 of what has been summed, so at
      most of S = scale * sum |q_d row_d|), as much again inside the steps, and the two fp32 products with
      the scale: dz = 80 * 2^-23 * max S.
    * a weight: e^dz from its logit, 2^-21 from the exponential, half a bf16 step (2^-8 relative) from the
      rounding for the output product; the sum it is divided by carries the same errors, so a weight is
      off by at most twice that. out: that times sum p |v|, plus fp32 sums (2^-16 covers 2^7 roundings)
      and half a bf16 step of the result itself. A weight below 2^-126 of the largest is no normal fp32
      number and becomes zero, so each row's |v| enters with 2^-126 too: it shows only where the rows a
      weight meets differ by a factor of that size (2^-126 * 448 * 2^59 = 2^-58 beside weights of one).
    * lse: dz, the exponentials' error, and fp32 sums and products of numbers of its size."""
    h = q.shape[0]
    if rows.shape[0] == 0:
        z = torch.zeros((h, d_latent), dtype=torch.float64)
        return z, torch.full((h,), -math.inf, dtype=torch.float64), z, torch.zeros(h, dtype=torch.float64)
    z = (q @ rows.T) * scale
    m = z.amax(dim=1, keepdim=True)
    p = torch.exp(z - m)
    total = p.sum(dim=1, keepdim=True)
    p = p / total
    v = rows[:, :d_latent]
    out = p @ v
    lse = (torch.log(total) + m).squeeze(1)
    s = abs(scale) * (q.abs() @ rows.abs().T).amax(dim=1)
    dz = 80 * 2.0 ** -23 * s
    weight = 2 * (2.0 ** -8 + 2.0 ** -21 + torch.expm1(dz))
    bound = (weight + 2.0 ** -16)[:, None] * (p @ v.abs()) + 2.0 ** -8 * out.abs() + 2.0 ** -126 * v.abs().sum(dim=0)
    bound_lse = dz + 2.0 ** -20 + 2.0 ** -21 * lse.abs()
    return out, lse, bound, bound_lse


def check(out, lse, ref):
    """Asserts one query's out [H, d] and lse [H] against attend()'s result."""
    r_out, r_lse, b_out, b_lse = ref
    out, lse = out.double().cpu(), lse.double().cpu()
    assert torch.equal(torch.isfinite(lse), torch.isfinite(r_lse)), "lse finiteness"
    assert torch.isfinite(out).all(), "out holds a NaN or an infinity"
    over = (out - r_out).abs() - b_out
    assert (over <= 0).all(), f"out beyond its bound by {over.max().item():.3g}"
    f = torch.isfinite(r_lse)
    assert (lse[~f] == r_lse[~f]).all(), "lse of an empty row"
    over = (lse - r_lse).abs()[f] - b_lse[f]
    assert (over <= 0).all(), f"lse beyond its bound by {over.max().item():.3g}"
