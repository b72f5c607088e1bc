"""The 8-bit checkpoint: its format against the definition, and the block that uses it against the formulas in 64
bits (bounds: fused_util)."""
import pytest
import torch

from fused_util import ACT, SLOPE, U, act64, close, eight_bit_values, eight_bits, product_error
from tensor_transformer_mlp_block_b200 import binding

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,F", [(1, 1), (1, 32), (3, 31), (5, 33), (32, 256), (33, 264), (31, 1000), (100, 77),
                                 (65, 4096), (257, 520)])
def test_encode_is_the_definition(T, F, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + F)
    H = torch.randn(T, F, generator=g, device="cuda") * torch.exp(3 * torch.randn(T, 1, generator=g, device="cuda"))
    H = H.to(DT[dtype])
    C, S = binding.ckpt8_encode(H)
    c, s = eight_bits(H)
    assert torch.equal(S, s) and torch.equal(C, c)
    for out in (torch.bfloat16, torch.float32):
        assert torch.equal(binding.ckpt8_decode(C, S, F, dtype=out).double(), eight_bit_values(C, S, F))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("F", [4, 36, 100, 252, 260, 516, 1004])
def test_decode_by_width_and_alignment(F, dtype):
    """Widths of whole 4, 8 or single elements, into aligned and unaligned rows; nothing beside them is written."""
    T, dt = 67, DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(F)
    H = torch.randn(T, F, generator=g, device="cuda").to(dt)
    C, S = binding.ckpt8_encode(H)
    want = eight_bit_values(C, S, F)
    for off in (0, 1, 2, 4, 8):
        buf = torch.full((T * F + 16,), 9.0, dtype=dt, device="cuda")
        out = buf[off:off + T * F].view(T, F)
        binding.ckpt8_decode(C, S, F, dtype=dt, out=out)
        assert torch.equal(out.double(), want)
        assert (buf[:off] == 9).all() and (buf[off + T * F:] == 9).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_encode_special_values(dtype):
    dt = DT[dtype]
    H = torch.zeros(14, 40, device="cuda", dtype=torch.float32)
    H[1, 3] = float("nan")
    H[2, 39] = float("inf")
    H[3, 0] = -float("inf")
    H[4] = 127.5
    H[5, :4] = torch.tensor([127.0, 0.5, 1.5, -2.5])
    H[6] = 2.0 ** -126
    H[7] = 1e-40
    H[8] = torch.finfo(dt).max
    H[9] = -torch.finfo(dt).max
    H[10] = -0.0
    H[11, :8] = torch.tensor([127.49, 63.75, 63.8, 31.9, 255.0, 254.9, -255.0, 1e-30])
    H[12] = torch.finfo(dt).tiny
    H[13] = 2.0 ** -121 * 1.9921875
    H = H.to(dt)
    C, S = binding.ckpt8_encode(H)
    c, s = eight_bits(H)
    assert torch.equal(S, s) and torch.equal(C, c)
    got, want = binding.ckpt8_decode(C, S, 40, dtype=torch.float32), eight_bit_values(C, S, 40)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(torch.nan_to_num(got.double()), torch.nan_to_num(want))
    # the block beside a bad one is kept
    assert torch.isfinite(got[1, 32:]).all() and torch.isfinite(got[2, :32]).all()


def test_encode_unaligned_and_bounds():
    F, T = 96, 10
    buf = torch.randn(T * F + 1, device="cuda").to(torch.bfloat16)
    H = buf[1:].view(T, F)
    C, S = binding.ckpt8_encode(H)
    c, s = eight_bits(H)
    assert torch.equal(S, s) and torch.equal(C, c)
    # an element is off by at most 1/127 of its block's largest magnitude
    v = binding.ckpt8_decode(C, S, F, dtype=torch.float32)
    top = H.float().view(T, 3, 32).abs().amax(2, keepdim=True)
    assert ((v - H.float()).view(T, 3, 32).abs() <= top / 127).all()


def make(T, h, F, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[dtype]
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(X=r(T, h).to(dt), A=(r(h, F) / h ** 0.5).to(dt), a=(0.3 * r(F)).to(dt),
                B=(r(F, h) / F ** 0.5).to(dt), b=(0.3 * r(h)).to(dt), R=r(T, h).to(dt), dZ=r(T, h).to(dt))


def acc(a, b, dtype):
    """fp32 outputs of the plain path: one accumulator, K additions."""
    return product_error(a, b) if dtype == "bf16" else a.shape[1] * U * (a.abs() @ b.abs())


def check_forward(v, act, C, S, Y, Z, dtype, bias=True, residual=True):
    x, A, B = v["X"].double(), v["A"].double(), v["B"].double()
    T, F = x.shape[0], A.shape[1]
    h = x @ A + (v["a"].double() if bias else 0.0)
    dh = acc(x, A, dtype) + 2 * U * h.abs()
    # the scale of the largest magnitude, or of its neighbour where the rounding of H decides
    lo, hi = eight_bits((h.abs() - dh).clamp(min=0))[1], eight_bits(h.abs() + dh)[1]
    assert (S >= lo).all() and (S <= hi).all()
    step = torch.ldexp(torch.ones_like(h), (S.t().int() - 127).repeat_interleave(32, 1)[:, :F])
    err = (eight_bit_values(C, S, F) - h).abs()
    assert (err <= step / 2 + dh).all(), float((err - step / 2 - dh).max())
    if F % 32:
        assert (C[:, F:] == 0).all()
    close(Y, act64(h, act)[0], SLOPE * dh + ACT * h.abs(), "Y")
    y = Y.double()
    z = y @ B + (v["b"].double() if bias else 0.0)
    dz = acc(y, B, dtype) + 2 * U * z.abs()
    if residual:
        z = z + v["R"].double()
        dz = dz + U * (z.abs() + v["R"].double().abs())
    close(Z, z, dz, "Z")


def check_backward(v, act, C, S, g, dtype):
    x, A, B, z = (v[k].double() for k in ("X", "A", "B", "dZ"))
    T, F = x.shape[0], A.shape[1]
    h = eight_bit_values(C, S, F)
    y, d = act64(h, act)
    p = z @ B.t()
    dp = acc(z, B.t(), dtype)
    close(g["Y"], y, ACT * h.abs(), "Y")
    close(g["dH"], p * d, SLOPE * dp + p.abs() * ACT * (1 + h.abs()) + U * (p * d).abs(), "dH")
    Y, dH = g["Y"].double(), g["dH"].double()
    close(g["dB"], Y.t() @ z, acc(Y.t(), z, dtype), "dB")
    close(g["dA"], x.t() @ dH, acc(x.t(), dH, dtype), "dA")
    close(g["dX"], dH @ A.t(), acc(dH, A.t(), dtype), "dX")
    n = 16 + 8 + -(-T // 512) + 8 + 64
    close(g["da"], dH.sum(0), n * U * dH.abs().sum(0), "da")
    close(g["db"], z.sum(0), n * U * z.abs().sum(0), "db")


# tensor-core path (one row to several tiles, F with a short last block), then the plain path
SHAPES = [(1, 64, 64, 2), (5, 200, 520, 2), (64, 128, 512, 4), (129, 64, 264, 3), (300, 200, 520, 2),
          (513, 256, 1032, 1), (256, 4096, 520, 2), (700, 4096, 264, 1)]
PLAIN = [(1, 12, 48, 2), (37, 12, 44, 2), (65, 33, 70, 1), (200, 130, 259, 1)]


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,h,F,p,dtype", [(*s, "bf16") for s in SHAPES + PLAIN] + [(*s, "fp32") for s in PLAIN] +
                         [(512, 12, 48, 2, "fp32"), (130, 256, 512, 2, "fp32")])
def test_block(T, h, F, p, dtype, act):
    v = make(T, h, F, dtype, seed=T + h + F)
    Y = torch.empty(T, F, dtype=DT[dtype], device="cuda")
    C, S, Z = binding.forward_ckpt8(v["X"], v["A"], v["a"], v["B"], v["b"], p, residual=v["R"], activation=act,
                                    scratch=Y)
    check_forward(v, act, C, S, Y, Z, dtype)
    for grad in {torch.float32, DT[dtype]}:
        g = binding.backward_ckpt8(v["dZ"], v["X"], v["A"], v["B"], C, S, p, activation=act, grad_dtype=grad)
        assert all(g[k].dtype == grad for k in ("dA", "da", "dB", "db"))
        check_backward(v, act, C, S, g, dtype)
    C, S, Z = binding.forward_ckpt8(v["X"], v["A"], None, v["B"], None, p, activation=act, scratch=Y)
    check_forward(v, act, C, S, Y, Z, dtype, bias=False, residual=False)
    assert binding.last_device_status() == binding.OK


@pytest.mark.parametrize("policy", [1, 2, 3])
def test_schedules(policy):
    binding.set_split_policy(policy)
    try:
        for T, h, F, p in [(384, 512, 1024, 4), (2048, 1024, 4096, 4)]:
            v = make(T, h, F, "bf16", seed=policy)
            Y = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
            C, S, Z = binding.forward_ckpt8(v["X"], v["A"], v["a"], v["B"], v["b"], p, residual=v["R"], scratch=Y)
            check_forward(v, "gelu", C, S, Y, Z, "bf16")
            for grad in (torch.float32, torch.bfloat16):
                check_backward(v, "gelu", C, S, binding.backward_ckpt8(v["dZ"], v["X"], v["A"], v["B"], C, S, p,
                                                                      grad_dtype=grad), "bf16")
    finally:
        binding.set_split_policy(0)
    assert binding.last_device_status() == binding.OK


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh"])
def test_long_products(act):
    """Enough k-blocks and tiles for the relaying, double-staged kernels."""
    T, h, F, p = 2304, 4096, 9216 + 8, 1
    v = make(T, h, F, "bf16", seed=1)
    Y = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
    C, S, Z = binding.forward_ckpt8(v["X"], v["A"], v["a"], v["B"], v["b"], p, residual=v["R"], activation=act,
                                    scratch=Y)
    check_forward(v, act, C, S, Y, Z, "bf16")
    for grad in (torch.float32, torch.bfloat16):
        check_backward(v, act, C, S, binding.backward_ckpt8(v["dZ"], v["X"], v["A"], v["B"], C, S, p, activation=act,
                                                            grad_dtype=grad), "bf16")
    assert binding.last_device_status() == binding.OK


@pytest.mark.parametrize("T,h,F", [(8192, 12288, 9472), (8192, 4096, 32768)])
def test_dynamic_schedule_gives_the_same(T, h, F):
    """Products long enough for the dynamic schedule (the first and third, then the second and last): bit for bit
    what the static one gives; rows of the results against the formulas."""
    v = make(T, h, F, "bf16", seed=2)
    assert any(binding.plan_dynamic(T, h, F, 1).values())
    got = []
    for on in (True, False):
        binding.set_dynamic_schedule(on)
        try:
            C, S, Z = binding.forward_ckpt8(v["X"], v["A"], v["a"], v["B"], v["b"], 1, residual=v["R"])
            g = binding.backward_ckpt8(v["dZ"], v["X"], v["A"], v["B"], C, S, 1, grad_dtype=torch.bfloat16)
            got.append(dict(C=C, S=S, Z=Z, **{k: g[k] for k in ("dX", "dH", "Y", "dA", "da", "dB", "db")}))
        finally:
            binding.set_dynamic_schedule(True)
    for k in got[0]:
        assert torch.equal(got[0][k], got[1][k]), k
    assert binding.last_device_status() == binding.OK
    rows = torch.tensor([0, 77, T - 1], device="cuda")
    part = {k: (t[rows] if k in ("X", "R", "dZ") else t) for k, t in v.items()}
    x, A, B, z = (part[k].double() for k in ("X", "A", "B", "dZ"))
    hh = x @ A + part["a"].double()
    C, S = got[0]["C"][rows], got[0]["S"][:, rows].contiguous()
    step = torch.ldexp(torch.ones_like(hh), (S.t().int() - 127).repeat_interleave(32, 1)[:, :F])
    bound = step / 2 + product_error(x, A) + 2 * U * hh.abs()
    assert ((eight_bit_values(C, S, F) - hh).abs() <= bound).all()
    y, d = act64(eight_bit_values(C, S, F), "gelu")
    p = z @ B.t()
    close(got[0]["dH"][rows], p * d, SLOPE * product_error(z, B.t()) + p.abs() * ACT * 6 + U * (p * d).abs(), "dH")
    dH = got[0]["dH"][rows].double()
    close(got[0]["dX"][rows], dH @ A.t(), product_error(dH, A.t()), "dX")


def test_agrees_with_the_block_that_keeps_h():
    """The forward's product and residual are forward()'s; the gradients differ by the checkpoint's rounding: at
    most 1/127 of a block's largest magnitude, a relative error of the gradients of a few parts in a thousand."""
    v = make(512, 256, 1024, "bf16", seed=4)
    H, Y, Z = binding.forward(v["X"], v["A"], v["a"], v["B"], v["b"], 2)
    C, S, Z8 = binding.forward_ckpt8(v["X"], v["A"], v["a"], v["B"], v["b"], 2)
    assert torch.equal(Z, Z8)
    g = binding.backward(v["dZ"], v["X"], v["A"], v["B"], H, Y, 2)
    g8 = binding.backward_ckpt8(v["dZ"], v["X"], v["A"], v["B"], C, S, 2)
    # |GeLU″| ≤ 0.8 and |GeLU′| ≤ 1.13: an error δ ≤ top/127 (rms ~ top/440, top ~ 2.5σ) of H moves dH and Y by
    # under 1 % of their rms
    for k in ("dX", "dA", "da", "dB"):
        rel = float((g8[k].double() - g[k].double()).norm() / g[k].double().norm())
        assert rel < 0.02, (k, rel)
    assert torch.equal(g["db"], g8["db"])


def test_nan_stays_in_its_row():
    T, h, F = 200, 128, 256
    v = make(T, h, F, "bf16", seed=6)
    C0, S0, Z0 = binding.forward_ckpt8(v["X"], v["A"], v["a"], v["B"], v["b"], 1)
    v["X"][77, 3] = float("nan")
    C, S, Z = binding.forward_ckpt8(v["X"], v["A"], v["a"], v["B"], v["b"], 1)
    assert (S[:, 77] == 255).all() and Z[77].isnan().all()
    S[:, 77], C[77], Z[77] = S0[:, 77], C0[77], Z0[77]
    assert torch.equal(S, S0) and torch.equal(C, C0) and torch.equal(Z, Z0)


def test_empty_and_in_place():
    v = make(16, 64, 128, "bf16", seed=3)
    want = binding.forward_ckpt8(v["X"], v["A"], v["a"], v["B"], v["b"], 2, residual=v["R"])
    R = v["R"].clone()
    binding.forward_ckpt8(v["X"], v["A"], v["a"], v["B"], v["b"], 2, residual=R, out=(None, None, R))
    assert torch.equal(R, want[2])
    C, S, Z = binding.forward_ckpt8(v["X"][:0], v["A"], v["a"], v["B"], v["b"], 2)
    assert C.shape == (0, 128) and S.shape == (4, 0) and Z.shape == (0, 64)
    for grad in (torch.float32, torch.bfloat16):
        g = binding.backward_ckpt8(v["dZ"][:0], v["X"][:0], v["A"], v["B"], C, S, 2, grad_dtype=grad)
        assert all((g[k] == 0).all() for k in ("dA", "da", "dB", "db"))


def test_refusals_on_the_gpu():
    v = make(8, 64, 96, "bf16")
    with pytest.raises(ValueError, match="activation"):
        binding.forward_ckpt8(v["X"], v["A"], None, v["B"], None, 1, activation="none")
    C, S, _ = binding.forward_ckpt8(v["X"], v["A"], None, v["B"], None, 1)
    with pytest.raises(ValueError, match="S has shape"):
        binding.backward_ckpt8(v["dZ"], v["X"], v["A"], v["B"], C, S.t().contiguous(), 1)
    with pytest.raises(ValueError, match="C has dtype"):
        binding.backward_ckpt8(v["dZ"], v["X"], v["A"], v["B"], C.view(torch.uint8), S, 1)
    with pytest.raises(TypeError):
        binding.backward_ckpt8(v["dZ"], v["X"], v["A"], v["B"], C, S, 1, grad_dtype=torch.float16)
    with pytest.raises(binding.TPMLPError):
        binding.forward_ckpt8(v["X"], v["A"], None, v["B"], None, 5)
    with pytest.raises(ValueError, match="C has shape"):
        binding.ckpt8_decode(C, S, 64)
    with pytest.raises(ValueError, match="workspace"):
        binding.forward_ckpt8(v["X"], v["A"], None, v["B"], None, 1,
                              workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        binding.ckpt8_encode(v["X"].half())
