"""Plain 64-bit forms of the pre-norm block's operators (layer norm, linear layer with its epilogue, 8-bit
checkpoint) and the error bounds their kernels are held to.

Bounds. U is half a unit in the last place of fp32 (2^-24), half(t) that of an output type. A sum of n fp32
products or terms, added in any order, is off by at most n·U·Σ|terms| to first order. The tensor cores add 16
products at a time to an fp32 accumulator and may cut rather than round it, which loses up to 2U of it per step:
(K/8 + 8)·U·Σ|a·b| covers the K/16 steps of a product and the few adds around it. Φ of the tensor-core epilogues
is off by at most 1.5e-7 (Abramowitz & Stegun 7.1.26) plus the approximations of 2^x and 1/x (2 units each) and
a handful of fp32 steps: ACT bounds the error of act(h)/|h| and of act′(h), with (1 + |h|)."""
import math

import torch

U = 2.0 ** -24
ACT = 1.5e-7 + 24 * U
SLOPE = 1.13  # |GeLU′| never exceeds it


def half(dtype):
    return torch.finfo(dtype).eps / 2


def act64(x, name):
    """(act, act′) in 64 bits."""
    if name == "none":
        return x, torch.ones_like(x)
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-x / math.sqrt(2.0))
        return x * cdf, cdf + x * torch.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    u = math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)
    du = math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * x * x)
    t = torch.tanh(u)
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * du


def product_error(a, b):
    """Bound on the error of a·b (64-bit copies of the operands the kernel read)."""
    K = a.shape[1]
    return (K / 8 + 8) * U * (a.abs() @ b.abs())


def close(got, want, bound, what):
    """|got − want| ≤ bound + half a unit of got's type, element by element."""
    err = (got.double() - want).abs() - bound - half(got.dtype) * want.abs()
    # an output below the type's normal range is rounded to its smallest steps
    err = err - torch.finfo(got.dtype).tiny
    assert torch.isfinite(got).all(), what
    worst = float(err.max()) if err.numel() else -1.0
    assert worst <= 0.0, f"{what}: {worst:.3g} beyond the bound (|want| up to {float(want.abs().max()):.3g})"


def eight_bits(H):
    """(C, S) of H by the format's definition, on 64-bit values: the smallest power of two, at least 2^-127, for
    which every rounded quotient is within ±127."""
    T, F = H.shape
    nb = -(-F // 32)
    x = torch.zeros(T, nb * 32, dtype=torch.float64, device=H.device)
    x[:, :F] = H.double()
    x = x.view(T, nb, 32)
    bad = ~(x.abs() < 127.5 * 2.0 ** 121).all(2)  # NaN, infinite, or rounding to 2^128
    x = torch.where(bad[..., None], torch.zeros_like(x), x)
    top = x.abs().amax(2)
    e = torch.full_like(top, -127.0)
    for k in range(-126, 123):  # raise e while the block does not fit
        e = torch.where(torch.round(torch.ldexp(top, -e.int())) > 127, torch.full_like(e, float(k)), e)
    C = torch.round(torch.ldexp(x, -e.int()[..., None])).to(torch.int8).view(T, nb * 32)
    S = torch.where(bad, torch.full_like(e, 255.0), e + 127).to(torch.uint8).t().contiguous()
    return C, S


def eight_bit_values(C, S, F):
    T = C.shape[0]
    v = torch.ldexp(C.double().view(T, -1, 32), (S.t().int() - 127)[..., None])
    v = torch.where((S.t() == 255)[..., None], torch.full_like(v, float("nan")), v)
    return v.reshape(T, -1)[:, :F]
