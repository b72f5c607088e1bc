"""Layer norm, forward and backward, against the formulas in 64 bits (bounds: fused_util)."""
import pytest
import torch

from fused_util import U, close
from tensor_transformer_mlp_block_b200 import binding

pytestmark = pytest.mark.gpu
EPS = 1e-5
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}

# one warp per row, several widths per thread, one row per block, rows that are no multiple of 16 bytes, rows too
# wide for registers; 0, 1 and odd numbers of rows
SHAPES = [(1, 1), (3, 7), (1, 256), (5, 264), (2, 512), (9, 1000), (4, 1024), (3, 1032), (0, 64), (1, 12288),
          (7, 771), (33, 2049), (2, 8192), (2, 8200), (3, 16384), (2, 16391), (2, 33000), (517, 1000), (1500, 96)]


def make(T, h, dtype, seed=0, offset=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dt = DT[dtype]
    X = (r(T, h) * torch.exp(0.5 * r(h)) + offset * r(h)).to(dt)
    return X, (1 + 0.1 * r(h)).to(dt), (0.1 * r(h)).to(dt), r(T, h).to(dt), r(T, h).to(dt)


def terms(T, h):
    """Longest chain of additions a sum over a row goes through: a thread's elements, its warp, the warps."""
    return max(32, -(-h // 1024)) + 20


def stats64(x):
    mu = x.mean(1, keepdim=True)
    return mu, 1.0 / torch.sqrt((x - mu).square().mean(1, keepdim=True) + EPS)


def check_forward(X, gamma, beta, Y, mean, rstd):
    x = X.double()
    T, h = x.shape
    g = torch.ones(h, device="cuda", dtype=torch.float64) if gamma is None else gamma.double()
    b = torch.zeros(h, device="cuda", dtype=torch.float64) if beta is None else beta.double()
    mu, rs = stats64(x)
    n = terms(T, h) * U
    dmu = n * x.abs().mean(1, keepdim=True)
    xh = (x - mu) * rs
    # rstd: the squares' sum is off by n relative, and by dmu² from the mean's own error
    drs = n * rs + rs ** 3 * dmu ** 2
    close(mean, mu[:, 0], dmu[:, 0], "mean")
    close(rstd, rs[:, 0], drs[:, 0], "rstd")
    bound = g.abs() * (rs * (dmu + 2 * U * (x.abs() + mu.abs())) + xh.abs() * (drs / rs + 4 * U)) + 2 * U * b.abs()
    close(Y, xh * g + b, bound + 2 * U * (xh * g).abs(), "Y")


def check_backward(X, gamma, dY, dR, mean, rstd, got):
    dX, dg, db = got
    x, y = X.double(), dY.double()
    T, h = x.shape
    g = torch.ones(h, device="cuda", dtype=torch.float64) if gamma is None else gamma.double()
    mu, rs = mean.double()[:, None], rstd.double()[:, None]
    xh = (x - mu) * rs
    gy = y * g
    c1, c2 = gy.mean(1, keepdim=True), (gy * xh).mean(1, keepdim=True)
    want = rs * (gy - c1 - xh * c2)
    n = (terms(T, h) + 6) * U
    dxh = 3 * U * (xh.abs() + rs * mu.abs())
    dc1 = n * gy.abs().mean(1, keepdim=True)
    dc2 = n * (gy * xh).abs().mean(1, keepdim=True) + (gy.abs() * dxh).mean(1, keepdim=True)
    bound = rs * (dc1 + xh.abs() * dc2 + dxh * c2.abs() + 6 * U * (gy.abs() + c1.abs() + (xh * c2).abs()))
    if dR is not None:
        want = want + dR.double()
        bound = bound + U * (want.abs() + dR.double().abs())
    close(dX, want, bound, "dX")
    # the rows of a block one after another, then the blocks in eight runs (at most 1024 blocks of each kind)
    rows = -(-T // 148) + 16 + 160
    close(dg, (y * xh).sum(0), rows * U * (y * xh).abs().sum(0) + (y.abs() * dxh).sum(0), "dgamma")
    close(db, y.sum(0), rows * U * y.abs().sum(0), "dbeta")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,h", SHAPES)
def test_forward_and_backward(T, h, dtype):
    X, gamma, beta, dY, dR = make(T, h, dtype, seed=T + h)
    Y, mean, rstd = binding.layernorm_forward(X, gamma, beta, eps=EPS)
    got = binding.layernorm_backward(dY, X, gamma, mean, rstd, residual_grad=dR)
    torch.cuda.synchronize()
    if T == 0:
        assert Y.shape == (0, h) and got[0].shape == (0, h)
        assert (got[1] == 0).all() and (got[2] == 0).all()
        return
    check_forward(X, gamma, beta, Y, mean, rstd)
    check_backward(X, gamma, dY, dR, mean, rstd, got)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("h", [96, 1000, 4096, 40000])
def test_optional_arguments(h, dtype):
    X, gamma, beta, dY, _ = make(19, h, dtype, seed=h)
    Y, mean, rstd = binding.layernorm_forward(X, None, None, eps=EPS)
    check_forward(X, None, None, Y, mean, rstd)
    check_backward(X, None, dY, None, mean, rstd, binding.layernorm_backward(dY, X, None, mean, rstd))
    Y2, m2, r2 = binding.layernorm_forward(X, gamma, None, eps=EPS, stats=False)
    assert m2 is None and r2 is None
    check_forward(X, gamma, None, Y2, mean, rstd)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_unaligned_rows_give_the_same(dtype):
    """A pointer that is not 16-byte aligned goes element by element; the sums then run in another order."""
    T, h = 21, 2048
    X, gamma, beta, dY, dR = make(T, h, dtype, seed=3)

    def shifted(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:] = t.reshape(-1)
        return buf[1:].view(t.shape)

    Y, mean, rstd = binding.layernorm_forward(shifted(X), shifted(gamma), shifted(beta), eps=EPS)
    check_forward(X, gamma, beta, Y, mean, rstd)
    got = binding.layernorm_backward(shifted(dY), shifted(X), shifted(gamma), mean, rstd, residual_grad=shifted(dR))
    check_backward(X, gamma, dY, dR, mean, rstd, got)


@pytest.mark.parametrize("h", [64, 1000, 4096, 33000])
def test_large_offset_keeps_the_variance(h):
    """Rows with a mean of 100 standard deviations: E[x²] − mean² would lose the variance, the centred sum does
    not."""
    X, gamma, beta, _, _ = make(16, h, "fp32", seed=h)
    X = X + 1000.0
    Y, mean, rstd = binding.layernorm_forward(X, gamma, beta, eps=EPS)
    check_forward(X, gamma, beta, Y, mean, rstd)


def test_constant_rows_and_special_values():
    h = 512
    X = torch.full((6, h), 3.0, device="cuda")
    X[1] = 0.0
    X[2, 7] = float("nan")
    X[3, 7] = float("inf")
    X[4] = torch.linspace(-1, 1, h, device="cuda")
    one = torch.ones(h, device="cuda")
    Y, mean, rstd = binding.layernorm_forward(X, one, None, eps=EPS)
    assert (Y[0] == 0).all() and (Y[1] == 0).all() and (Y[5] == 0).all()
    assert Y[2].isnan().all() and Y[3].isnan().any()
    # the rows beside them are untouched
    check_forward(X[4:5], one, None, Y[4:5], mean[4:5], rstd[4:5])
    # a zero variance without eps: 0·∞ is NaN in this row alone
    Y0, _, r0 = binding.layernorm_forward(X, one, None, eps=0.0)
    assert Y0[0].isnan().all() and torch.isinf(r0[0]) and torch.isfinite(Y0[4]).all()


def test_in_place_gradient_and_repeatable():
    T, h = 300, 1024
    X, gamma, beta, dY, dR = make(T, h, "bf16", seed=11)
    _, mean, rstd = binding.layernorm_forward(X, gamma, beta, eps=EPS)
    want = binding.layernorm_backward(dY, X, gamma, mean, rstd, residual_grad=dR)
    for alias in ("dY", "dR"):
        y, r = dY.clone(), dR.clone()
        out = (y if alias == "dY" else r, torch.empty_like(want[1]), torch.empty_like(want[2]))
        binding.layernorm_backward(y, X, gamma, mean, rstd, residual_grad=r, out=out)
        assert all(torch.equal(a, b) for a, b in zip(out, want)), alias
    X, gamma, beta, dY, dR = make(9, 40000, "bf16", seed=12)  # the looped kernels too
    _, mean, rstd = binding.layernorm_forward(X, gamma, beta, eps=EPS)
    want = binding.layernorm_backward(dY, X, gamma, mean, rstd, residual_grad=dR)
    y = dY.clone()
    got = binding.layernorm_backward(y, X, gamma, mean, rstd, residual_grad=dR,
                                     out=(y, torch.empty_like(want[1]), torch.empty_like(want[2])))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradients_match_differences():
    """L = Σ dY ⊙ Y in 64 bits, central differences: with step s the difference quotient is off by O(s²) of a third
    derivative of order one and 1e-16·L/s of rounding, both below 1e-7 here; the fp32 gradients are off by 1e-6."""
    T, h, s = 3, 40, 1e-4
    X, gamma, beta, dY, _ = make(T, h, "fp32", seed=5)
    x, g, b, y = X.double(), gamma.double(), beta.double(), dY.double()

    def loss(x, g, b):
        mu, rs = stats64(x)
        return float((((x - mu) * rs * g + b) * y).sum())

    _, mean, rstd = binding.layernorm_forward(X, gamma, beta, eps=EPS)
    dX, dg, db = binding.layernorm_backward(dY, X, gamma, mean, rstd)
    for i, j in [(0, 0), (1, 17), (2, 39)]:
        e = torch.zeros_like(x)
        e[i, j] = s
        assert abs((loss(x + e, g, b) - loss(x - e, g, b)) / (2 * s) - float(dX[i, j])) < 1e-5
        v = torch.zeros_like(g)
        v[j] = s
        assert abs((loss(x, g + v, b) - loss(x, g - v, b)) / (2 * s) - float(dg[j])) < 1e-5
        assert abs((loss(x, g, b + v) - loss(x, g, b - v)) / (2 * s) - float(db[j])) < 1e-5


def test_rows_past_32_bits():
    """Element offsets beyond 2^32: the last rows are computed, and nothing else is written behind them."""
    h = 4096
    T = 2 ** 32 // h + 5
    X = torch.zeros(T, h, dtype=torch.bfloat16, device="cuda")
    Y = torch.full((T, h), 7.0, dtype=torch.bfloat16, device="cuda")
    rows, gamma, beta, dY, dR = make(5, h, "bf16", seed=8)
    X[-5:] = rows
    out = (Y, torch.empty(T, device="cuda"), torch.empty(T, device="cuda"))
    _, mean, rstd = binding.layernorm_forward(X, gamma, beta, eps=EPS, out=out)
    check_forward(rows, gamma, beta, Y[-5:], mean[-5:], rstd[-5:])
    Y.zero_()
    Y[-5:] = dY
    dX, dg, db = binding.layernorm_backward(Y, X, gamma, mean, rstd, out=(X.new_empty(0).new_full((T, h), 3.0), torch.empty(h, device="cuda"), torch.empty(h, device="cuda")))
    want = binding.layernorm_backward(dY, rows, gamma, mean[-5:].clone(), rstd[-5:].clone())
    assert torch.equal(dX[-5:], want[0]) and (dX[:-5] == 0).all()


def test_refusals_on_the_gpu():
    X, gamma, beta, dY, _ = make(8, 64, "bf16")
    _, mean, rstd = binding.layernorm_forward(X, gamma, beta)
    with pytest.raises(ValueError, match="gamma"):
        binding.layernorm_forward(X, gamma.float(), beta)
    with pytest.raises(ValueError, match="beta"):
        binding.layernorm_forward(X, gamma, beta[:32])
    with pytest.raises(ValueError, match="contiguous"):
        binding.layernorm_forward(X.t().contiguous().t(), gamma, beta)
    with pytest.raises(TypeError):
        binding.layernorm_forward(X.half(), gamma, beta)
    with pytest.raises(ValueError, match="mean"):
        binding.layernorm_backward(dY, X, gamma, None, None)
    with pytest.raises(ValueError, match="workspace"):
        binding.layernorm_backward(dY, X, gamma, mean, rstd, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(binding.TPMLPError):
        binding.layernorm_forward(X, gamma, beta, eps=-1.0)
