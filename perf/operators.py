"""Cases of the block's fused operators: layer norm, the linear layer with bias, activation and
residual in its epilogue, and the MLP with its pre-activation kept in 8 bits between the forward
and the backward. Each case names one pass through one operator; `run` computes it in plain torch
operations, or, where `own` is true, through the library's entry points.

The operators, for X of T rows:

layer norm        x̂ = (x − mean)·rstd, rstd = 1/√(var + eps), Y = x̂·γ + β; mean and rstd are outputs.
                  Backward: g = dY·γ, dX = rstd·(g − mean(g) − x̂·mean(g·x̂)) + dR, with dR the
                  gradient that arrives along the residual path (or none); dγ = Σ dY·x̂, dβ = Σ dY.
linear            H = X·W + bias, Y = act(H) + R. Backward: dH = dY·act′(H), dX = dH·Wᵀ, dW = Xᵀ·dH,
                  dbias = Σ dH (R's gradient is dY itself). H is kept for it where there is an activation.
checkpointed MLP  H = X·A + a, Y = GeLU(H), Z = Y·B + b + R; of H the backward gets only an 8-bit copy:
                  blocks of 32 columns of a row, one power of two 2^e for the block, the smallest for
                  which every rint(h/2^e) is within ±127, and those integers. The backward computes with
                  H̃ = 2^e·integer: dH = (dZ·Bᵀ)·GeLU′(H̃), dB = GeLU(H̃)ᵀ·dZ, dA = Xᵀ·dH, dX = dH·Aᵀ and
                  the column sums da, db. The gradients of matrices and biases have the weights' type.
"""
import math

import torch

own = False

EPS = 1e-5
ROOT_HALF = math.sqrt(0.5)
TANH_C = math.sqrt(2.0 / math.pi)
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # serving: the norm before the block for one new token of the widest configuration; all latency
        dict(name="norm forward, one token", op="norm", back=False, T=1, h=12288, dtype="bf16", residual=False),
        # training, the 350m configuration's micro-batch
        dict(name="norm forward, 350m", op="norm", back=False, T=6144, h=1024, dtype="bf16", residual=False),
        # an odd width and an odd batch in full precision: rows start at any 4-byte boundary
        dict(name="norm forward, odd fp32", op="norm", back=False, T=1023, h=771, dtype="fp32", residual=False),
        # training, the 7b configuration, joined by the gradient that passes around the block
        dict(name="norm backward, 7b", op="norm", back=True, T=8192, h=4096, dtype="bf16", residual=True),
        # a short full-precision batch, where the weights' gradient is reduced over few rows
        dict(name="norm backward, short fp32", op="norm", back=True, T=517, h=1000, dtype="fp32", residual=False),
        # serving: one token through the 7b configuration's first product, bound by reading the weight
        dict(name="linear forward, one token", op="linear", back=False, T=1, K=4096, N=16384, dtype="bf16", act="gelu", residual=False),
        # serving: a small batch of tokens through the second product, joined with the residual stream
        dict(name="linear forward, few tokens", op="linear", back=False, T=24, K=16384, N=4096, dtype="bf16", act="none", residual=True),
        # a prompt of ragged length through an output projection at the 7b width
        dict(name="linear forward, ragged", op="linear", back=False, T=1777, K=4096, N=4096, dtype="bf16", act="gelu_tanh", residual=True),
        # training: the backward pass of a layer with an activation, 350m
        dict(name="linear backward, 350m", op="linear", back=True, T=6144, K=1024, N=4096, dtype="bf16", act="gelu", residual=False),
        # the smallest configuration, full precision: the backward pass from a kept checkpoint, all latency
        dict(name="checkpointed backward, tiny", op="mlp8", part="backward", T=512, h=12, F=48, p=2, dtype="fp32", act="gelu", residual=False),
        # a training step of the 350m configuration's block
        dict(name="checkpointed step, 350m", op="mlp8", part="step", T=6144, h=1024, F=4096, p=4, dtype="bf16", act="gelu", residual=True),
        # a training step of the 7b configuration's block, the largest
        dict(name="checkpointed step, 7b", op="mlp8", part="step", T=8192, h=4096, F=16384, p=2, dtype="bf16", act="gelu", residual=True),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "linear", "linear", "linear", "mlp8", "mlp8"])
    dtype = "fp32" if rng.random() < 0.25 else "bf16"
    residual = rng.random() < 0.5
    if op == "norm":
        h = _spread(rng, 64, 16384)
        if rng.random() < 0.75:
            h = max(64, h // 8 * 8)
        T = _spread(rng, 1, min(16384, 8192 * 4096 // h))
        return dict(op=op, back=rng.random() < 0.5, T=T, h=h, dtype=dtype, residual=residual)
    # widths: multiples of 8 (what the tensor cores' loads can describe), now and then any number
    odd = rng.random() < 0.12
    top = 1024 if dtype == "fp32" or odd else 16384
    K, N = (_spread(rng, 32, top) for _ in range(2))
    if not odd:
        K, N = max(32, K // 8 * 8), max(32, N // 8 * 8)
    act = rng.choice(["none", "gelu", "gelu_tanh"])
    if op == "linear":
        back = rng.random() < 0.4
        T = _spread(rng, 1, 2048 if dtype == "fp32" or odd else 4096 if back else 8192)
        return dict(op=op, back=back, T=T, K=K, N=N, dtype=dtype, act=act, residual=residual)
    T = _spread(rng, 16, 2048 if dtype == "fp32" or odd else 8192)
    h = min(K, 4096)
    p = rng.choice([1, 2, 4])
    F = max(p, N // p * p) if odd else max(32, N // 32 * 32)
    # In full precision the two passes are cases of their own: where H falls next to a border between two
    # of the copy's integers, the last bits of its sum decide, and a step's fp32 gradients would show it.
    part = rng.choice(["forward", "backward"] if dtype == "fp32" else ["step", "step", "forward", "backward"])
    return dict(op=op, part=part, T=T, h=h, F=F, p=p, dtype=dtype, act="gelu" if act == "none" else act,
                residual=residual and part != "backward")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, to=dt):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(to)

    s = dict(case)
    T = case["T"]
    if case["op"] == "norm":
        h = case["h"]
        # a residual stream: every channel has its own scale and offset, a few of them large
        scale = torch.exp(0.5 * torch.randn(h, generator=gen, device="cuda"))
        offset = 0.5 * torch.randn(h, generator=gen, device="cuda")
        s["X"] = (torch.randn(T, h, generator=gen, device="cuda") * scale + offset).to(dt)
        s["gamma"], s["beta"] = normal(h, std=0.1, mean=1.0), normal(h, std=0.1)
        if case["back"]:
            s["dY"] = normal(T, h)
            s["dR"] = normal(T, h) if case["residual"] else None
            # what the forward pass left
            x = s["X"].double()
            s["mean"] = x.mean(1).float()
            s["rstd"] = (1.0 / torch.sqrt(x.var(1, unbiased=False) + EPS)).float()
    elif case["op"] == "linear":
        K, N = case["K"], case["N"]
        s["X"], s["W"] = normal(T, K), normal(K, N, std=1.0 / math.sqrt(K))
        s["bias"] = normal(N, std=0.1)
        if case["back"]:
            s["dY"] = normal(T, N)
            s["H"] = normal(T, N) if case["act"] != "none" else None  # what the forward pass left
        else:
            s["R"] = normal(T, N) if case["residual"] else None
    else:
        h, F = case["h"], case["F"]
        s["X"], s["A"], s["a"] = normal(T, h), normal(h, F, std=1.0 / math.sqrt(h)), normal(F, std=0.1)
        s["B"], s["b"] = normal(F, h, std=1.0 / math.sqrt(F)), normal(h, std=0.1)
        s["R"] = normal(T, h) if case["residual"] else None
        if case["part"] != "forward":
            s["dZ"] = normal(T, h)
        if case["part"] == "backward":  # what the forward pass left
            s["C"], s["S"] = eight_bits(normal(T, F, to=torch.float32))
    return s


def run(s):
    if s["op"] == "norm":
        return norm_backward(s) if s["back"] else norm_forward(s)
    if s["op"] == "linear":
        return linear_backward(s) if s["back"] else linear_forward(s)
    if s["part"] == "backward":
        return mlp8_backward(s, s["C"], s["S"])
    Z, C, S = mlp8_forward(s)
    if s["part"] == "forward":
        return Z, checkpoint_values(s, C, S)
    return (Z, *mlp8_backward(s, C, S))


def act_value(x, act):
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * ROOT_HALF))
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(TANH_C * (x + 0.044715 * x * x * x)))
    return x


def act_slope(x, act):
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(x * ROOT_HALF)) + x * torch.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    t = torch.tanh(TANH_C * (x + 0.044715 * x * x * x))
    return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * TANH_C * (1.0 + 0.134145 * x * x)


def norm_forward(s):
    X, gamma, beta = s["X"], s["gamma"], s["beta"]
    if own:
        from tensor_transformer_mlp_block_b200 import binding
        return binding.layernorm_forward(X, gamma, beta, eps=EPS)
    x = X.float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).mean(1) + EPS)
    return (c * rstd[:, None] * gamma.float() + beta.float()).to(X.dtype), mean, rstd


def norm_backward(s):
    dY, X, gamma, mean, rstd, dR = s["dY"], s["X"], s["gamma"], s["mean"], s["rstd"], s["dR"]
    if own:
        from tensor_transformer_mlp_block_b200 import binding
        return binding.layernorm_backward(dY, X, gamma, mean, rstd, residual_grad=dR)
    dy = dY.float()
    xhat = (X.float() - mean[:, None]) * rstd[:, None]
    g = dy * gamma.float()
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    if dR is not None:
        dx = dx + dR.float()
    return dx.to(X.dtype), (dy * xhat).sum(0), dy.sum(0)


def linear_forward(s):
    X, W, bias, R, act = s["X"], s["W"], s["bias"], s["R"], s["act"]
    if own:
        from tensor_transformer_mlp_block_b200 import binding
        return binding.fused_linear_forward(X, W, bias, activation=act, residual=R)
    y = act_value(X.float() @ W.float() + bias.float(), act)
    return (y if R is None else y + R.float()).to(X.dtype)


def linear_backward(s):
    dY, X, W, H, act = s["dY"], s["X"], s["W"], s["H"], s["act"]
    if own:
        from tensor_transformer_mlp_block_b200 import binding
        return binding.fused_linear_backward(dY, X, W, H, activation=act, grad_dtype=W.dtype)
    dh = dY.float()
    if act != "none":
        dh = dh * act_slope(H.float(), act)
    return (dh @ W.float().T).to(X.dtype), (X.float().T @ dh).to(W.dtype), dh.sum(0).to(W.dtype)


def eight_bits(H):
    """The 8-bit copy of H (T × F): C, T rows of whole blocks of 32 integers (zeros behind column F), and S,
    the exponents e + 127 of the blocks, one row of T for each block of columns."""
    T, F = H.shape
    blocks = torch.nn.functional.pad(H, (0, -F % 32)).reshape(T, -1, 32)
    top = blocks.abs().amax(2, keepdim=True)
    e = torch.frexp(top)[1] - 7  # top/2^e is in [64, 128)
    e = e + (torch.round(torch.ldexp(top, -e)) > 127).to(e.dtype)
    e = torch.clamp(e, min=-127)
    C = torch.round(torch.ldexp(blocks, -e)).to(torch.int8).reshape(T, -1)
    return C, (e[:, :, 0].T + 127).to(torch.uint8).contiguous()


def eight_bit_values(C, S, F):
    """H̃ in fp32."""
    T = C.shape[0]
    return torch.ldexp(C.reshape(T, -1, 32).float(), (S.T.int() - 127)[:, :, None]).reshape(T, -1)[:, :F]


def checkpoint_values(s, C, S):
    if own:
        from tensor_transformer_mlp_block_b200 import binding
        return binding.ckpt8_decode(C, S, s["F"], dtype=torch.bfloat16)
    return eight_bit_values(C, S, s["F"]).to(torch.bfloat16)  # exact: 7 bits and a sign


def mlp8_forward(s):
    X, A, a, B, b, R, act = (s[k] for k in ("X", "A", "a", "B", "b", "R", "act"))
    if own:
        from tensor_transformer_mlp_block_b200 import binding
        C, S, Z = binding.forward_ckpt8(X, A, a, B, b, s["p"], residual=R, activation=act)
        return Z, C, S
    H = X.float() @ A.float() + a.float()
    Z = act_value(H, act) @ B.float() + b.float()
    return ((Z if R is None else Z + R.float()).to(X.dtype), *eight_bits(H))


def mlp8_backward(s, C, S):
    dZ, X, A, B, act = (s[k] for k in ("dZ", "X", "A", "B", "act"))
    if own:
        from tensor_transformer_mlp_block_b200 import binding
        g = binding.backward_ckpt8(dZ, X, A, B, C, S, s["p"], activation=act, grad_dtype=A.dtype)
        return g["dX"], g["dA"], g["da"], g["dB"], g["db"]
    H = eight_bit_values(C, S, s["F"])
    dz = dZ.float()
    dH = (dz @ B.float().T) * act_slope(H, act)
    out = (dH @ A.float().T, X.float().T @ dH, dH.sum(0), act_value(H, act).T @ dz, dz.sum(0))
    return tuple(t.to(X.dtype) for t in out)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    T = case["T"]
    if case["op"] == "norm":
        h = case["h"]
        if not case["back"]:
            return dict(bytes=e * (2 * T * h + 2 * h) + 8 * T, flops=8 * T * h)
        return dict(bytes=e * ((3 + case["residual"]) * T * h + h) + 8 * T + 8 * h, flops=14 * T * h)
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        if not case["back"]:
            return dict(bytes=e * (T * K + K * N + N + (1 + case["residual"]) * T * N), flops=2 * T * K * N)
        kept = 0 if case["act"] == "none" else 1
        return dict(bytes=e * ((1 + kept) * T * N + 2 * T * K + 2 * K * N + N), flops=4 * T * K * N)
    h, F = case["h"], case["F"]
    copy = T * (F + -(-F // 32))
    # X, R in, Z out, the weights, the 8-bit copy written (and its values returned, in 16 bits)
    forward = e * ((2 + case["residual"]) * T * h + 2 * h * F + F + h) + copy
    # X, dZ in, dX out, the weights, their gradients, the 8-bit copy read
    backward = e * (3 * T * h + 4 * h * F + F + h) + copy
    if case["part"] == "forward":
        return dict(bytes=forward + copy + 2 * T * F, flops=4 * T * h * F)
    if case["part"] == "backward":
        return dict(bytes=backward, flops=8 * T * h * F)
    # a step reads X and the weights once
    return dict(bytes=forward + backward - e * (T * h + 2 * h * F), flops=12 * T * h * F)


def exact(case, seed):
    """The definition in 64 bits. Products of this size take well under a second in double
    precision on the GPU."""
    s = prepare(case, seed)
    v = {k: (t.double() if isinstance(t, torch.Tensor) else t) for k, t in s.items()}
    if case["op"] == "norm":
        X, gamma = v["X"], v["gamma"]
        n = X.shape[1]
        if not case["back"]:
            mu = X.sum(1) / n
            var = (X - mu[:, None]).pow(2).sum(1) / n
            r = torch.rsqrt(var + EPS)
            return (X - mu[:, None]) * (r[:, None] * gamma) + v["beta"], mu, r
        dY, r = v["dY"], v["rstd"][:, None]
        xh = (X - v["mean"][:, None]) * r
        g = dY * gamma
        dx = g * r - r * (g.sum(1, keepdim=True) + xh * (g * xh).sum(1, keepdim=True)) / n
        return (dx if v["dR"] is None else dx + v["dR"]), torch.einsum("ij,ij->j", dY, xh), torch.einsum("ij->j", dY)
    if case["op"] == "linear":
        if not case["back"]:
            y = _exact_act(torch.addmm(v["bias"], v["X"], v["W"]), case["act"])[0]
            return y if v["R"] is None else y + v["R"]
        dH = v["dY"] if case["act"] == "none" else v["dY"] * _exact_act(v["H"], case["act"])[1]
        return torch.mm(dH, v["W"].t()), torch.mm(v["X"].t(), dH), torch.einsum("ij->j", dH)
    T, F = case["T"], case["F"]
    nb = -(-F // 32)
    first = []
    if case["part"] == "backward":
        Ht = (v["C"].view(T, nb, 32) * torch.exp2(v["S"].t() - 127.0)[..., None]).view(T, nb * 32)[:, :F]
    else:
        H = torch.addmm(v["a"], v["X"], v["A"])
        Z = torch.addmm(v["b"], _exact_act(H, case["act"])[0], v["B"])
        first = [Z if v["R"] is None else Z + v["R"]]
        Hp = torch.zeros(T, nb * 32, dtype=torch.float64, device=H.device)
        Hp[:, :F] = H
        Hp = Hp.view(T, nb, 32)
        top = Hp.abs().max(dim=2).values.clamp(min=1e-30)
        # the smallest power of two with top/2^e < 127.5: a value at 127.5 would round to 128
        step = torch.exp2(torch.floor(torch.log2(top / 127.5)) + 1.0)
        Ht = (torch.round(Hp / step[..., None]) * step[..., None]).view(T, nb * 32)[:, :F]
        if case["part"] == "forward":
            return first[0], Ht
    y, slope = _exact_act(Ht, case["act"])
    dH = torch.mm(v["dZ"], v["B"].t()) * slope
    return (*first, torch.mm(dH, v["A"].t()), torch.mm(v["X"].t(), dH), torch.einsum("ij->j", dH),
            torch.mm(y.t(), v["dZ"]), torch.einsum("ij->j", v["dZ"]))


def _exact_act(x, act):
    """(act(x), act′(x)) in 64 bits, through the complementary error function or the logistic function."""
    if act == "none":
        return x, torch.ones_like(x)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-x / math.sqrt(2.0))
        return x * cdf, cdf + x * torch.exp(-x * x / 2.0) / math.sqrt(2.0 * math.pi)
    c = 2.0 * math.sqrt(2.0 / math.pi)
    p = torch.sigmoid(c * (x + 0.044715 * x ** 3))
    return x * p, p + x * p * (1.0 - p) * c * (1.0 + 3.0 * 0.044715 * x * x)
