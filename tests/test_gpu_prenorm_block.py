"""The pre-norm block's operators together, as a training or serving step runs them: layer norm, the MLP with its
8-bit checkpoint and the residual, a projection with its epilogue; captured, replayed, on several streams and
threads. (Bounds: fused_util.)"""
import threading

import pytest
import torch

from fused_util import act64, eight_bit_values
from tensor_transformer_mlp_block_b200 import binding

pytestmark = pytest.mark.gpu
EPS = 1e-5


def make(T, h, F, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(S=(r(T, h) * torch.exp(0.3 * r(h))).to(dtype), gamma=(1 + 0.1 * r(h)).to(dtype),
                beta=(0.1 * r(h)).to(dtype), A=(r(h, F) / h ** 0.5).to(dtype), a=(0.1 * r(F)).to(dtype),
                B=(r(F, h) / F ** 0.5).to(dtype), b=(0.1 * r(h)).to(dtype), W=(r(h, h) / h ** 0.5).to(dtype),
                bias=(0.1 * r(h)).to(dtype), dO=r(T, h).to(dtype))


def step(v, p, grad=torch.float32):
    """O = P + MLP(LN(P)), P = S + GeLU(LN(S)·W + bias), and every gradient."""
    N0, m0, r0 = binding.layernorm_forward(v["S"], v["gamma"], v["beta"], eps=EPS)
    P, H0 = binding.fused_linear_forward(N0, v["W"], v["bias"], activation="gelu", residual=v["S"], keep_hidden=True)
    N1, m1, r1 = binding.layernorm_forward(P, v["gamma"], v["beta"], eps=EPS)
    C, S8, O = binding.forward_ckpt8(N1, v["A"], v["a"], v["B"], v["b"], p, residual=P)
    g = binding.backward_ckpt8(v["dO"], N1, v["A"], v["B"], C, S8, p, grad_dtype=grad)
    dP, dg1, db1 = binding.layernorm_backward(g["dX"], P, v["gamma"], m1, r1, residual_grad=v["dO"])
    dN0, dW, dbias = binding.fused_linear_backward(dP, N0, v["W"], H0, activation="gelu", grad_dtype=grad)
    dS, dg0, db0 = binding.layernorm_backward(dN0, v["S"], v["gamma"], m0, r0, residual_grad=dP)
    return dict(O=O, P=P, N1=N1, C=C, S8=S8, dA=g["dA"], da=g["da"], dB=g["dB"], db=g["db"], dP=dP, dW=dW,
                dbias=dbias, dS=dS, dgamma0=dg0, dbeta0=db0, dgamma1=dg1, dbeta1=db1)


def reference(v, got, H8):
    """The same block in 64 bits by autograd, H replaced by the 8-bit values in the backward (H8)."""
    x = {k: t.double().requires_grad_(k != "dO") for k, t in v.items()}

    def norm(t):
        c = t - t.mean(1, keepdim=True)
        return c / torch.sqrt(c.square().mean(1, keepdim=True) + EPS)

    g0, g1 = x["gamma"].detach().clone().requires_grad_(), x["gamma"].detach().clone().requires_grad_()
    b0, b1 = x["beta"].detach().clone().requires_grad_(), x["beta"].detach().clone().requires_grad_()
    N0 = norm(x["S"]) * g0 + b0
    H0 = N0 @ x["W"] + x["bias"]
    P = x["S"] + act64(H0, "gelu")[0]
    P.retain_grad()
    N1 = norm(P) * g1 + b1
    H = N1 @ x["A"] + x["a"]
    H = H + (H8 - H.detach())  # the backward's H
    O = act64(H, "gelu")[0] @ x["B"] + x["b"] + P
    O.backward(x["dO"])
    return dict(P=P, dA=x["A"].grad, da=x["a"].grad, dB=x["B"].grad, db=x["b"].grad, dP=P.grad, dW=x["W"].grad,
                dbias=x["bias"].grad, dS=x["S"].grad, dgamma0=g0.grad, dbeta0=b0.grad, dgamma1=g1.grad,
                dbeta1=b1.grad)


@pytest.mark.parametrize("T,h,F,p,dtype", [(300, 256, 1032, 2, torch.bfloat16), (37, 36, 92, 2, torch.bfloat16),
                                           (64, 48, 160, 1, torch.float32), (1, 128, 256, 1, torch.bfloat16)])
def test_block_gradients(T, h, F, p, dtype):
    """Every gradient of the two-layer block against 64-bit autograd. Each stored tensor is rounded once (half a
    unit u relative, √3 below that in the mean), at most nine of them on a path; in the norm, errors spread over a
    tensor add as their squares do: 9·u/√3 ≈ 5.2 u, doubled for the slopes (1.13 and the norms' gains)."""
    v = make(T, h, F, dtype, seed=T)
    got = step(v, p)
    ref = reference(v, got, eight_bit_values(got["C"], got["S8"], F))
    u = torch.finfo(dtype).eps / 2
    tol = max(10.4 * u, 2e-5)  # fp32: sums of up to F terms, no better than 2e-5
    for k, r in ref.items():
        r = r.detach()
        rel = float((got[k].double() - r).norm() / r.norm())
        assert rel <= tol, (k, rel, tol)
    assert binding.last_device_status() == binding.OK


def _clone(d):
    return {k: t.clone() for k, t in d.items()}


def test_repeatable_and_overlap():
    """The same bits on every run, with programmatic launches and without."""
    v = make(700, 512, 2048, seed=1)
    want = _clone(step(v, 2))
    for _ in range(3):
        got = step(v, 2)
        assert all(torch.equal(got[k], want[k]) for k in want)
    binding.set_launch_overlap(False)
    try:
        got = step(v, 2)
        assert all(torch.equal(got[k], want[k]) for k in want)
    finally:
        binding.set_launch_overlap(True)


@pytest.mark.parametrize("T", [1, 48, 600])
def test_captured_and_replayed(T):
    """A step captured once and replayed on new inputs; two graphs replayed in turn."""
    h, F, p = 256, 1024, 2
    ins = [make(T, h, F, seed=s) for s in (1, 2, 3)]
    want = [_clone(step(v, p)) for v in ins]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        v = _clone(ins[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(v, p)
        graphs.append((g, v, out))
    for k in (1, 2, 0, 1):
        for which, (g, v, out) in enumerate(graphs):
            i = (k + which) % 3
            for name in v:
                v[name].copy_(ins[i][name])
            g.replay()
        torch.cuda.synchronize()
        for which, (g, v, out) in enumerate(graphs):
            i = (k + which) % 3
            assert all(torch.equal(out[n], want[i][n]) for n in out), (k, which)
    assert binding.last_device_status() == binding.OK


def test_shared_workspace_in_order():
    """Calls of different operators may share one workspace on one stream."""
    v = make(300, 256, 1024, seed=4)
    want = _clone(step(v, 2))
    n = max(binding.layernorm_workspace_size(300, 256), binding.linear_ex_workspace_size(300, 256, 256),
            binding.ckpt8_workspace_size(300, 256, 1024, 2))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN patterns: nothing is read before it is written
    N0, m0, r0 = binding.layernorm_forward(v["S"], v["gamma"], v["beta"], eps=EPS)
    P, H0 = binding.fused_linear_forward(N0, v["W"], v["bias"], activation="gelu", residual=v["S"], keep_hidden=True,
                                         workspace=ws)
    N1, m1, r1 = binding.layernorm_forward(P, v["gamma"], v["beta"], eps=EPS)
    C, S8, O = binding.forward_ckpt8(N1, v["A"], v["a"], v["B"], v["b"], 2, residual=P, workspace=ws)
    g = binding.backward_ckpt8(v["dO"], N1, v["A"], v["B"], C, S8, 2, workspace=ws)
    dP, dg1, db1 = binding.layernorm_backward(g["dX"], P, v["gamma"], m1, r1, residual_grad=v["dO"], workspace=ws)
    dN0, dW, dbias = binding.fused_linear_backward(dP, N0, v["W"], H0, activation="gelu", workspace=ws)
    for k, t in dict(O=O, dP=dP, dW=dW, dbias=dbias, dA=g["dA"], db=g["db"], dgamma1=dg1, dbeta1=db1).items():
        assert torch.equal(t, want[k]), k


def test_other_streams():
    """On a stream that is not current (its outputs belong to it), and on two at once."""
    vs = [make(400, 256, 1024, seed=s) for s in (5, 6)]
    want = [_clone(step(v, 2)) for v in vs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    v = vs[0]
    for _ in range(20):
        s.wait_stream(torch.cuda.current_stream())
        Y, m, r = binding.layernorm_forward(v["S"], v["gamma"], v["beta"], eps=EPS, stream=s)
        P, H = binding.fused_linear_forward(Y, v["W"], v["bias"], activation="gelu", residual=v["S"],
                                            keep_hidden=True, stream=s)
        Y1, m1, r1 = binding.layernorm_forward(P, v["gamma"], v["beta"], eps=EPS, stream=s)
        C, S8, O = binding.forward_ckpt8(Y1, v["A"], v["a"], v["B"], v["b"], 2, residual=P, stream=s)
        g = binding.backward_ckpt8(v["dO"], Y1, v["A"], v["B"], C, S8, 2, stream=s)
        dP, _, _ = binding.layernorm_backward(g["dX"], P, v["gamma"], m1, r1, residual_grad=v["dO"], stream=s)
        torch.empty(1 << 20, device="cuda").fill_(7.0)  # the current stream's allocations do not get in the way
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(O, want[0]["O"]) and torch.equal(dP, want[0]["dP"])
    streams = [torch.cuda.Stream() for _ in vs]
    outs = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(step(vs[i], 2))
    torch.cuda.synchronize()
    for i in range(2):
        for got in outs[i]:
            assert all(torch.equal(got[k], want[i][k]) for k in want[i])


def test_two_threads():
    vs = [make(300, 256, 1024, seed=s) for s in (7, 8)]
    want = [_clone(step(v, 2)) for v in vs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(15):
                    got = step(vs[i], 2)
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(got[k], want[i][k]) for k in want[i]):
                        bad.append(i)
        except Exception as e:  # noqa: BLE001
            bad.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in ts]
    [t.join(120) for t in ts]
    assert not bad and not any(t.is_alive() for t in ts)


def test_serving_single_tokens_equal_the_batch():
    """A token alone gives what it gives in a batch of the few-row kernel's same tile (its sums run in the same
    order), and what the many-row kernel gives up to rounding."""
    v = make(400, 512, 1024, seed=9)
    Y = binding.fused_linear_forward(v["S"], v["W"], v["bias"], activation="gelu_tanh", residual=v["S"])
    few = binding.fused_linear_forward(v["S"][:16], v["W"], v["bias"], activation="gelu_tanh", residual=v["S"][:16])
    for i in (0, 7, 15):
        row = v["S"][i:i + 1].contiguous()
        one = binding.fused_linear_forward(row, v["W"], v["bias"], activation="gelu_tanh", residual=row)
        assert torch.equal(one[0], few[i])
    # two roundings to bf16 (each half a unit) of values whose sums differ in their last fp32 bits
    diff = (few.double() - Y[:16].double()).abs()
    assert (diff <= 2 * 2.0 ** -8 * Y[:16].double().abs() + 1e-4).all()


def test_wrong_device_stream_is_refused():
    v = make(4, 64, 64)

    class Other:
        device = torch.device("cuda", 99)

    with pytest.raises(ValueError, match="stream"):
        binding.layernorm_forward(v["S"], v["gamma"], v["beta"], stream=Other())


def test_overlapping_outputs_are_refused():
    """An output that is an input, or shares memory with one, would be written while other rows are still read."""
    T, h = 64, 128
    g = torch.Generator(device="cuda").manual_seed(5)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()

    X, W, b, R = rand(T, h), rand(h, h), rand(h), rand(T, h)
    before = binding.launch_count()

    def refused(f, *args, **kw):
        with pytest.raises(binding.TPMLPError) as e:
            f(*args, **kw)
        assert e.value.status == binding.ERR_INVALID

    both = rand(2 * T, h)
    refused(binding.fused_linear_forward, X, W, b, residual=X, out=X)
    refused(binding.fused_linear_forward, X, W, b, residual=both[:T], out=both[8:T + 8])
    refused(binding.fused_linear_forward, X, W, b, activation="gelu", out=both[:T], hidden=both[1:T + 1])
    refused(binding.fused_linear_backward, R, X, W, out=(R, None, None, None))
    refused(binding.fused_linear_backward, R, X, W, rand(T, h), activation="gelu", out=(None, None, None, X))
    refused(binding.layernorm_forward, X, b, b, out=(X, None, None))
    mean, rstd = torch.zeros(T, device="cuda"), torch.ones(T, device="cuda")
    refused(binding.layernorm_backward, R, X, b, mean, rstd, out=(X, None, None))
    refused(binding.layernorm_backward, both[1:T + 1], X, b, mean, rstd, out=(both[:T], None, None))
    refused(binding.forward_ckpt8, X, W, b, W, b, 2, residual=X, scratch=R, out=(None, None, R))
    refused(binding.forward_ckpt8, X, W, b, W, b, 2, out=(None, None, X))
    assert binding.launch_count() == before
    C, S, Z = binding.forward_ckpt8(X, W, b, W, b, 2)
    before = binding.launch_count()
    for k in ("dX", "dH", "Y"):
        refused(binding.backward_ckpt8, R, X, W, W, C, S, 2, out={k: R})
    assert binding.launch_count() == before
    # the allowed ones: the residual in place, a gradient in place
    want = binding.fused_linear_forward(X, W, b, residual=R)
    R2 = R.clone()
    assert torch.equal(binding.fused_linear_forward(X, W, b, residual=R2, out=R2), want)
    # neighbours in one buffer
    buf = rand(2 * T, h)
    buf[:T] = X
    assert torch.equal(binding.fused_linear_forward(buf[:T], W, b, residual=R, out=buf[T:]), want)
