"""Layer norm's backward where rows have an offset. (Bounds: fused_util and test_gpu_norm.)"""
import pytest
import torch

from fused_util import U, close
from tensor_transformer_mlp_block_b200 import binding
from test_gpu_norm import DT, EPS, make, terms

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("offset", [100.0, 1000.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("h", [96, 512, 1000, 4096, 12288, 16384, 771, 4099, 40000])
def test_offset_costs_no_precision(h, dtype, offset):
    """Rows with a mean of 100 and 1000 standard deviations, the mean and rstd given (64-bit values rounded to fp32,
    as the backward gets them): (x − mean)·rstd is two fp32 steps, so x̂ is off by 2U relative whatever the offset
    (3U below, second orders included). Four rows, each in a group of its own: dgamma's sum is one rounded product
    a row and three additions."""
    T = 4
    X, gamma, _, dY, _ = make(T, h, dtype, seed=h)
    shift = offset * torch.tensor([1.0, -1.0009, 1.07, -1.3], device="cuda")[:, None]
    X = (X.float() + shift).to(DT[dtype])
    dY = (dY.float() + 1.0).to(DT[dtype])  # Σ g far from zero: an error that a whole row shares stays in dX
    x, y, g = X.double(), dY.double(), gamma.double()
    mu = x.mean(1, keepdim=True)
    rs = 1.0 / torch.sqrt((x - mu).square().mean(1, keepdim=True) + EPS)
    mean, rstd = mu[:, 0].float(), rs[:, 0].float()
    mu, rs = mean.double()[:, None], rstd.double()[:, None]
    dX, dg, db = binding.layernorm_backward(dY, X, gamma, mean, rstd)
    xh, gy = (x - mu) * rs, y * g
    dxh = 3 * U * xh.abs()
    c1, c2 = gy.mean(1, keepdim=True), (gy * xh).mean(1, keepdim=True)
    n = (terms(T, h) + 6) * U
    dc1 = n * gy.abs().mean(1, keepdim=True)
    dc2 = n * (gy * xh).abs().mean(1, keepdim=True) + (gy.abs() * dxh).mean(1, keepdim=True)
    bound = rs * (dc1 + xh.abs() * dc2 + dxh * c2.abs() + 6 * U * (gy.abs() + c1.abs() + (xh * c2).abs()))
    close(dg, (y * xh).sum(0), T * U * (y * xh).abs().sum(0) + (y.abs() * dxh).sum(0), "dgamma")
    close(db, y.sum(0), T * U * y.abs().sum(0), "dbeta")
    close(dX, rs * (gy - c1 - xh * c2), bound, "dX")
