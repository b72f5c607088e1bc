"""Layer norm's backward where a group of threads walks many rows (ring stages refilled, phases turning, sums over a
group's rows), and where rows have an offset. (Bounds: fused_util and test_gpu_norm.)"""
import pytest
import torch

from fused_util import U, close
from tensor_transformer_mlp_block_b200 import binding
from test_gpu_norm import DT, EPS, check_backward, make, terms

pytestmark = pytest.mark.gpu

# Rows per group of threads on 148 SMs (groups: a warp, or a block): at least six, where a ring holds up to four.
# A warp per row (2368 groups), blocks of 64 (1184), 160 and 256 (296), 512 and 768 threads (148); 32 elements a
# thread; one stage (fp32 from 12288 on). Then rows that are not whole vectors: 128 threads (888 groups), 288 (296),
# 512 (148), and rows too wide for registers (one group per 128 rows).
RING = [(14211, 96, "bf16"), (14211, 96, "fp32"), (14211, 512, "bf16"), (7107, 1000, "bf16"), (7107, 1000, "fp32"),
        (1779, 2056, "bf16"), (1779, 4096, "bf16"), (891, 4096, "fp32"), (891, 8192, "bf16"), (891, 12288, "bf16"),
        (891, 12288, "fp32"), (891, 16384, "bf16"), (891, 16384, "fp32")]
SINGLE = [(5331, 771, "bf16"), (1779, 4099, "fp32"), (891, 8191, "bf16"), (300, 16391, "fp32"), (300, 40000, "bf16")]


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("T,h,dtype", RING + SINGLE)
def test_many_rows_per_group(T, h, dtype, residual):
    """Against 64 bits; a row's dX has the bits that it has in a call of few rows, where no stage is used twice; and
    every run gives the same bits."""
    X, gamma, _, dY, dR = make(T, h, dtype, seed=T + h)
    dR = dR if residual else None
    _, mean, rstd = binding.layernorm_forward(X, gamma, None, eps=EPS)
    want = binding.layernorm_backward(dY, X, gamma, mean, rstd, residual_grad=dR)
    check_backward(X, gamma, dY, dR, mean, rstd, want)
    for i in range(0, T, 140):
        s = slice(i, min(T, i + 140))
        part = binding.layernorm_backward(dY[s], X[s], gamma, mean[s], rstd[s],
                                          residual_grad=None if dR is None else dR[s])
        assert torch.equal(part[0], want[0][s]), i
    for _ in range(10):
        again = binding.layernorm_backward(dY, X, gamma, mean, rstd, residual_grad=dR)
        assert all(torch.equal(a, b) for a, b in zip(again, want))
    assert binding.last_device_status() == binding.OK


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
