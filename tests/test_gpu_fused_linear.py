"""The linear layer with bias, activation and residual in its epilogue, forward and backward, against the formulas
in 64 bits (bounds: fused_util). A product that reads a stored, rounded tensor is compared with the exact product
of that stored tensor."""
import pytest
import torch

from fused_util import ACT, SLOPE, U, act64, close, half, product_error
from tensor_transformer_mlp_block_b200 import binding

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(autouse=True)
def _auto_policy():
    binding.set_split_policy(0)
    yield
    binding.set_split_policy(0)


def make(T, K, N, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[dtype]
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(X=r(T, K).to(dt), W=(r(K, N) / K ** 0.5).to(dt), bias=(0.3 * r(N)).to(dt), R=r(T, N).to(dt),
                dY=r(T, N).to(dt), H=(2 * r(T, N)).to(dt))


def check_forward(v, act, Y, H=None, bias=True, residual=True):
    x, w = v["X"].double(), v["W"].double()
    h = x @ w + (v["bias"].double() if bias else 0.0)
    dh = product_error(x, w) + 2 * U * h.abs()
    if H is not None:
        close(H, h, dh, "H")
    y = act64(h, act)[0]
    bound = dh if act == "none" else SLOPE * dh + ACT * h.abs()
    if residual:
        y = y + v["R"].double()
        bound = bound + U * (y.abs() + v["R"].double().abs())
    close(Y, y, bound + U * y.abs(), "Y")


def check_backward(v, act, got, dH, grad):
    dX, dW, db = got
    y, x, w = v["dY"].double(), v["X"].double(), v["W"].double()
    T = x.shape[0]
    g = y
    if act != "none":
        h = v["H"].double()
        g = y * act64(h, act)[1]
        dg = y.abs() * ACT * (1 + h.abs())
        close(dH, g, dg + U * g.abs(), "dH")
    else:
        dg = torch.zeros_like(g)
    # summed before dH is rounded: rows in chunks of 128 (16 a phase), then the chunks
    n = 16 + 8 + -(-T // 1024) + 8
    close(db, g.sum(0), n * U * g.abs().sum(0) + dg.sum(0), "dbias")
    s = (v["dY"] if act == "none" else dH).double()
    close(dW, x.t() @ s, product_error(x.t(), s), "dW")
    close(dX, s @ w.t(), product_error(s, w.t()), "dX")
    assert dW.dtype == grad and db.dtype == grad


# the tensor cores' path: one row, few rows, a tile and a row more, several tiles; ragged K and N
TC = [(1, 64, 64), (1, 8, 8), (2, 4096, 136), (7, 200, 520), (16, 1024, 264), (17, 3000, 48), (33, 768, 2304),
      (64, 512, 1000), (65, 256, 512), (128, 128, 128), (129, 64, 264), (300, 200, 520), (513, 1024, 768)]
# the plain path: fp32, and bf16 whose rows are no multiple of 16 bytes
PLAIN = [(1, 12, 48), (37, 13, 45), (1, 77, 1), (130, 65, 131), (3, 1001, 333), (257, 1, 70), (700, 259, 515)]


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,K,N", TC + PLAIN)
def test_forward_bf16(T, K, N, act):
    v = make(T, K, N, "bf16", seed=T + K + N)
    Y = binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation=act, residual=v["R"])
    check_forward(v, act, Y)
    Y0 = binding.fused_linear_forward(v["X"], v["W"], None, activation=act)
    check_forward(v, act, Y0, bias=False, residual=False)
    if act != "none":
        Y1, H = binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation=act, residual=v["R"],
                                             keep_hidden=True)
        check_forward(v, act, Y1, H)
        Y2, H2 = binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation=act, keep_hidden=True)
        check_forward(v, act, Y2, H2, residual=False)
        assert torch.equal(H, H2)
    assert binding.last_device_status() == binding.OK


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,K,N", PLAIN + [(64, 64, 64), (512, 384, 640)])
def test_forward_fp32(T, K, N, act):
    v = make(T, K, N, "fp32", seed=T + K + N)
    Y = binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation=act, residual=v["R"])
    # one fp32 accumulator per output, K additions in order
    x, w = v["X"].double(), v["W"].double()
    h = x @ w + v["bias"].double()
    dh = (K + 2) * U * (x.abs() @ w.abs() + v["bias"].double().abs())
    y = act64(h, act)[0] + v["R"].double()
    close(Y, y, SLOPE * dh + ACT * h.abs() + 2 * U * (y.abs() + v["R"].double().abs()), "Y")


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,K,N", TC + PLAIN)
def test_backward_bf16(T, K, N, act, grad):
    v = make(T, K, N, "bf16", seed=T + 2 * K + N)
    dH = torch.empty_like(v["dY"]) if act != "none" else None
    got = binding.fused_linear_backward(v["dY"], v["X"], v["W"], v["H"] if act != "none" else None, activation=act,
                                        grad_dtype=grad, out=(None, None, None, dH))
    check_backward(v, act, got, dH, grad)
    assert binding.last_device_status() == binding.OK


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,K,N", PLAIN + [(512, 384, 640)])
def test_backward_fp32(T, K, N, act):
    v = make(T, K, N, "fp32", seed=T + 2 * K + N)
    dH = torch.empty_like(v["dY"]) if act != "none" else None
    dX, dW, db = binding.fused_linear_backward(v["dY"], v["X"], v["W"], v["H"] if act != "none" else None,
                                               activation=act, out=(None, None, None, dH))
    y, x, w, h = (v[k].double() for k in ("dY", "X", "W", "H"))
    g = y * act64(h, act)[1]
    if act != "none":
        close(dH, g, y.abs() * ACT * (1 + h.abs()), "dH")
    s = y if act == "none" else dH.double()
    close(dW, x.t() @ s, T * U * (x.abs().t() @ s.abs()), "dW")
    close(dX, s @ w.t(), N * U * (s.abs() @ w.abs().t()), "dX")
    close(db, g.sum(0), (40 + T / 1024) * U * g.abs().sum(0) + (y.abs() * ACT * (1 + h.abs())).sum(0), "dbias")


@pytest.mark.parametrize("policy", [0, 1, 2, 3])
@pytest.mark.parametrize("split", ["columns", "rows"])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_splits_and_schedules(policy, split, act):
    """Every work schedule, both splits: split tiles are finished by the residual epilogue too."""
    binding.set_split_policy(policy)
    for T, K, N, p in [(256, 512, 1024, 4), (640, 4096, 512, 2), (24, 2048, 512, 8)]:
        v = make(T, K, N, "bf16", seed=policy + T)
        Y = binding.fused_linear_forward(v["X"], v["W"], v["bias"], p, split, activation=act, residual=v["R"])
        check_forward(v, act, Y)
        dH = torch.empty_like(v["dY"]) if act != "none" else None
        got = binding.fused_linear_backward(v["dY"], v["X"], v["W"], v["H"] if act != "none" else None, p, split,
                                            activation=act, out=(None, None, None, dH))
        check_backward(v, act, got, dH, torch.float32)
    assert binding.last_device_status() == binding.OK


@pytest.mark.parametrize("T", [1, 40, 100, 200, 2100])
@pytest.mark.parametrize("K", [64, 4096])
def test_long_and_relayed_products(T, K):
    """K on both sides of the relaying epilogue's threshold, enough tiles for the long-product variant."""
    v = make(T, K, 4096 + 8, "bf16", seed=T)
    for act in ("none", "gelu", "gelu_tanh"):
        check_forward(v, act, binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation=act,
                                                           residual=v["R"]))
        if act != "none":
            Y, H = binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation=act, residual=v["R"],
                                                keep_hidden=True)
            check_forward(v, act, Y, H)
    assert binding.last_device_status() == binding.OK


def test_long_product_variant():
    """Four waves of tiles and 64 k-blocks: the kernels with two staging slots per warp."""
    v = make(8200, 4096, 2568, "bf16", seed=1)
    for act in ("none", "gelu", "gelu_tanh"):
        check_forward(v, act, binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation=act,
                                                           residual=v["R"]))
        if act != "none":
            Y, H = binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation=act, residual=v["R"],
                                                keep_hidden=True)
            check_forward(v, act, Y, H)
    R = v["R"].clone()
    binding.fused_linear_forward(v["X"], v["W"], v["bias"], residual=R, out=R)
    check_forward(v, "none", R)


@pytest.mark.parametrize("T,K,N", [(8200, 4096, 2568), (6144, 1024, 2048), (1777, 4096, 1032)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_residual_is_the_same_every_time(T, K, N, act):
    """The residual's buffer is read and loaded again many times over; every run gives the first one's bits, and
    those are right."""
    v = make(T, K, N, "bf16", seed=3)
    want = binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation=act, residual=v["R"])
    check_forward(v, act, want)
    got, bad = torch.empty_like(want), torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(150):
        got.fill_(9.0)
        binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation=act, residual=v["R"], out=got)
        bad += (got != want).sum()
    assert int(bad) == 0
    assert binding.last_device_status() == binding.OK


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_offsets_past_32_bits(dtype):
    """More than 2^31 outputs: the last rows come out right."""
    T, K, N = 70016, 16, 33000
    v = make(300, K, N, dtype, seed=2)
    X = torch.zeros(T, K, dtype=DT[dtype], device="cuda")
    X[-300:] = v["X"]
    Y = binding.fused_linear_forward(X, v["W"], v["bias"], activation="gelu")
    want = binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation="gelu")
    zero = binding.fused_linear_forward(X[:300].contiguous(), v["W"], v["bias"], activation="gelu")
    # (another number of rows may mean another kernel and order of sums: 16 products)
    assert float((Y[-300:].double() - want.double()).abs().max()) <= 2 ** -7 * float(want.double().abs().max())
    assert torch.equal(Y[:300], zero) and torch.equal(Y[35000], zero[0])
    del want, zero
    if dtype == "bf16":
        dX, dW, db = binding.fused_linear_backward(Y, X, v["W"])
        ref = Y[-300:].double() @ v["W"].double().t()
        close(dX[-300:], ref, product_error(Y[-300:].double(), v["W"].double().t()), "dX")


@pytest.mark.parametrize("T", [1, 16, 64, 200])
def test_residual_in_place(T):
    v = make(T, 512, 768, "bf16", seed=T)
    want = binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation="gelu", residual=v["R"])
    R = v["R"].clone()
    got = binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation="gelu", residual=R, out=R)
    assert got is R and torch.equal(R, want)


@pytest.mark.parametrize("T", [1, 5, 64, 130])
def test_nothing_else_is_written(T):
    """Outputs inside larger buffers: the elements before and behind them keep their values."""
    v = make(T, 264, 72, "bf16", seed=T)
    buf = torch.full((T + 4, 72), 9.0, dtype=torch.bfloat16, device="cuda")
    hid = torch.full((T + 4, 72), 9.0, dtype=torch.bfloat16, device="cuda")
    Y, H = binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation="gelu", residual=v["R"],
                                        out=buf[2:T + 2], hidden=hid[2:T + 2])
    check_forward(v, "gelu", Y, H)
    for b in (buf, hid):
        assert (b[:2] == 9).all() and (b[T + 2:] == 9).all()


def test_rows_are_independent():
    """A NaN or an infinity in one row of X (or of the residual) stays in that row."""
    for T in (3, 40, 300):
        v = make(T, 256, 512, "bf16", seed=T)
        want = binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation="gelu", residual=v["R"])
        X, R = v["X"].clone(), v["R"].clone()
        X[1, 5] = float("nan")
        R[2, 7] = float("inf")
        got = binding.fused_linear_forward(X, v["W"], v["bias"], activation="gelu", residual=R)
        assert got[1].isnan().all() and torch.isinf(got[2, 7])
        got[1], got[2, 7] = want[1], want[2, 7]
        assert torch.equal(got, want)


def test_empty():
    v = make(4, 64, 32, "bf16")
    X, dY = v["X"][:0], v["dY"][:0]
    assert binding.fused_linear_forward(X, v["W"], v["bias"], activation="gelu").shape == (0, 32)
    for grad in (torch.float32, torch.bfloat16):
        dX, dW, db = binding.fused_linear_backward(dY, X, v["W"], v["H"][:0], activation="gelu", grad_dtype=grad)
        assert dX.shape == (0, 64) and (dW == 0).all() and (db == 0).all()


def test_gradients_match_differences():
    """L = Σ dY ⊙ act(X·W + bias) in 64 bits, central differences (steps and errors as in the layer norm's test)."""
    T, K, N, s = 4, 9, 6, 1e-4
    for act in ("gelu", "gelu_tanh"):
        v = make(T, K, N, "fp32", seed=2)
        Y, H = binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation=act, keep_hidden=True)
        dX, dW, db = binding.fused_linear_backward(v["dY"], v["X"], v["W"], H, activation=act)
        x, w, b, y = (v[k].double() for k in ("X", "W", "bias", "dY"))
        loss = lambda x, w, b: float((act64(x @ w + b, act)[0] * y).sum())  # noqa: E731
        for i, j, k in [(0, 0, 0), (3, 8, 5), (2, 4, 1)]:
            ex, ew, eb = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(b)
            ex[i, j], ew[j, k], eb[k] = s, s, s
            assert abs((loss(x + ex, w, b) - loss(x - ex, w, b)) / (2 * s) - float(dX[i, j])) < 1e-5
            assert abs((loss(x, w + ew, b) - loss(x, w - ew, b)) / (2 * s) - float(dW[j, k])) < 1e-5
            assert abs((loss(x, w, b + eb) - loss(x, w, b - eb)) / (2 * s) - float(db[k])) < 1e-5


def test_refusals_on_the_gpu():
    v = make(8, 64, 96, "bf16")
    f, b = binding.fused_linear_forward, binding.fused_linear_backward
    with pytest.raises(ValueError, match="activation"):
        f(v["X"], v["W"], v["bias"], activation="relu")
    with pytest.raises(ValueError, match="pre-activation"):
        f(v["X"], v["W"], v["bias"], keep_hidden=True)
    with pytest.raises(ValueError, match="residual"):
        f(v["X"], v["W"], v["bias"], residual=v["R"][:4])
    with pytest.raises(ValueError, match="W has"):
        f(v["X"], v["W"].float(), v["bias"])
    with pytest.raises(binding.TPMLPError) as e:
        f(v["X"], v["W"], v["bias"], 5)
    assert e.value.status == binding.ERR_INVALID
    with pytest.raises(ValueError, match="H is the pre-activation"):
        b(v["dY"], v["X"], v["W"], activation="gelu")
    with pytest.raises(ValueError, match="H is the pre-activation"):
        b(v["dY"], v["X"], v["W"], v["H"])
    with pytest.raises(TypeError):
        b(v["dY"], v["X"], v["W"], grad_dtype=torch.float16)
    with pytest.raises(ValueError, match="workspace"):
        b(v["dY"], v["X"], v["W"], workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    w = make(8, 64, 96, "fp32")
    with pytest.raises(TypeError):
        b(w["dY"], w["X"], w["W"], grad_dtype=torch.bfloat16)
    buf = torch.empty(8 * 96 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(8, 96)
    with pytest.raises(binding.TPMLPError) as e:
        f(v["X"], v["W"], v["bias"], out=buf)
    assert e.value.status == binding.ERR_ALIGN
    assert half(torch.bfloat16) == 2.0 ** -8
