"""Calls of the pre-norm block's operators that their documentation allows: outputs in place on every path, one tensor
as several arguments, split products of few rows, extreme widths, two calls at once, NaN in one place. (Bounds:
fused_util.)"""
import pytest
import torch

import test_gpu_ckpt8 as ck
import test_gpu_fused_linear as fl
import test_gpu_norm as nm
from fused_util import U, close, product_error
from tensor_transformer_mlp_block_b200 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _auto_policy():
    binding.set_split_policy(0)
    yield
    binding.set_split_policy(0)
    assert binding.last_device_status() == binding.OK


# plain path (64-wide tiles, K split over a cluster and not; 128-wide tiles), then the tensor cores' with H kept: one
# CTA's few rows, a pair's tiles, relayed and double-staged
@pytest.mark.parametrize("T,K,N,dtype", [(1, 33, 70, "fp32"), (37, 1024, 132, "fp32"), (130, 65, 131, "bf16"),
                                         (3100, 40, 3200, "fp32"), (96, 512, 768, "bf16"), (300, 200, 520, "bf16"),
                                         (2100, 4096, 4104, "bf16"), (8200, 4096, 2568, "bf16")])
@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh"])
def test_residual_in_place_on_every_path(T, K, N, dtype, act):
    v = fl.make(T, K, N, dtype, seed=T)
    keep = act != "none"
    want = binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation=act, residual=v["R"], keep_hidden=keep)
    R = v["R"].clone()
    got = binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation=act, residual=R, out=R, keep_hidden=keep)
    for a, b in zip(got if keep else (got,), want if keep else (want,)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,h,dtype", [(14211, 96, "bf16"), (1779, 4096, "bf16"), (891, 4096, "fp32"),
                                       (891, 16384, "fp32"), (5331, 771, "bf16"), (300, 16391, "fp32")])
def test_norm_gradients_in_place(T, h, dtype):
    """dX over dY, over dR, and over one tensor that is both, with many rows to a group of threads."""
    X, gamma, beta, dY, dR = nm.make(T, h, dtype, seed=h)
    _, mean, rstd = binding.layernorm_forward(X, gamma, beta)
    for y, r in ((dY, dR), (dY, dY)):
        want = binding.layernorm_backward(y, X, gamma, mean, rstd, residual_grad=r)
        nm.check_backward(X, gamma, y, r, mean, rstd, want)
        for alias in ("y", "r"):
            y2 = y.clone()
            r2 = y2 if r is y else r.clone()
            out = (y2 if alias == "y" else r2, torch.empty_like(want[1]), torch.empty_like(want[2]))
            binding.layernorm_backward(y2, X, gamma, mean, rstd, residual_grad=r2, out=out)
            assert all(torch.equal(a, b) for a, b in zip(out, want)), alias


def test_one_tensor_as_several_inputs():
    v = fl.make(200, 256, 256, "bf16", seed=1)
    same = dict(v, R=v["X"])
    fl.check_forward(same, "gelu", binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation="gelu",
                                                                residual=v["X"]))
    assert torch.equal(binding.layernorm_forward(v["X"], v["bias"], v["bias"])[0],
                       binding.layernorm_forward(v["X"], v["bias"], v["bias"].clone())[0])
    C, S, Z = binding.forward_ckpt8(v["X"], v["W"], v["bias"], v["W"], v["bias"], 2, residual=v["X"])
    C2, S2, Z2 = binding.forward_ckpt8(v["X"].clone(), v["W"], v["bias"], v["W"].clone(), v["bias"].clone(), 2,
                                       residual=v["X"])
    assert torch.equal(C, C2) and torch.equal(S, S2) and torch.equal(Z, Z2)
    g = binding.backward_ckpt8(v["X"], v["X"], v["W"], v["W"], C, S, 2)
    ck.check_backward(dict(X=v["X"], A=v["W"], B=v["W"], dZ=v["X"]), "gelu", C, S, g, "bf16")


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh"])
@pytest.mark.parametrize("T", [1, 64, 128])
def test_checkpointed_few_rows_split(T, act):
    """Policy 3 splits the first product of few rows (64 tiles of 16 k-blocks on 148 CTAs): the 8-bit epilogues
    finish split tiles, and the call needs its workspace."""
    h, F = 1024, 16384
    binding.set_split_policy(3)
    assert binding.plan_schedules(T, h, F, 1)["F1"] == binding.SCHED_STREAMK
    v = ck.make(T, h, F, "bf16", seed=T)
    Y = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
    C, S, Z = binding.forward_ckpt8(v["X"], v["A"], v["a"], v["B"], v["b"], 1, residual=v["R"], activation=act,
                                    scratch=Y)
    ck.check_forward(v, act, C, S, Y, Z, "bf16")
    for grad in (torch.float32, torch.bfloat16):
        ck.check_backward(v, act, C, S, binding.backward_ckpt8(v["dZ"], v["X"], v["A"], v["B"], C, S, 1,
                                                               activation=act, grad_dtype=grad), "bf16")


@pytest.mark.parametrize("T,K,N", [(1, 65536, 8), (5, 8, 200000), (128, 40000, 24), (1, 8, 8), (100, 72, 100008)])
def test_extreme_widths_of_few_rows(T, K, N):
    v = fl.make(T, K, N, "bf16", seed=T)
    for act in ("none", "gelu"):
        fl.check_forward(v, act, binding.fused_linear_forward(v["X"], v["W"], v["bias"], activation=act,
                                                              residual=v["R"]))


def test_clusters_and_rings_at_once():
    """Few-row products whose clusters fill the GPU, and norms, on three streams: the bits of each by itself."""
    few = [fl.make(24, 16384, 4096, "bf16", seed=s) for s in (1, 2)]
    X, gamma, beta, dY, dR = nm.make(3000, 4096, "bf16", seed=3)
    run = [lambda v=v: (binding.fused_linear_forward(v["X"], v["W"], v["bias"], residual=v["R"]),) for v in few]
    _, mean, rstd = binding.layernorm_forward(X, gamma, beta)
    run.append(lambda: binding.layernorm_backward(dY, X, gamma, mean, rstd, residual_grad=dR))
    want = [f() for f in run]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in run]
    got = [[] for _ in run]
    for _ in range(20):
        for f, s, g in zip(run, streams, got):
            with torch.cuda.stream(s):
                g.append(f())
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for one in g:
            assert all(torch.equal(a, b) for a, b in zip(one, w))


@pytest.mark.parametrize("T,h,dtype", [(1779, 4096, "bf16"), (14211, 96, "fp32"), (1779, 4099, "fp32")])
def test_nan_in_a_gradient(T, h, dtype):
    """A NaN in dY reaches its row of dX and its column of dgamma and dbeta, and nothing else."""
    X, gamma, beta, dY, _ = nm.make(T, h, dtype, seed=h)
    _, mean, rstd = binding.layernorm_forward(X, gamma, beta)
    want = binding.layernorm_backward(dY, X, gamma, mean, rstd)
    dY = dY.clone()
    dY[T // 2, 17] = float("nan")
    dX, dg, db = binding.layernorm_backward(dY, X, gamma, mean, rstd)
    assert dX[T // 2].isnan().all() and dg[17].isnan() and db[17].isnan()
    dX[T // 2], dg[17], db[17] = want[0][T // 2], want[1][17], want[2][17]
    assert torch.equal(dX, want[0]) and torch.equal(dg, want[1]) and torch.equal(db, want[2])


@pytest.mark.parametrize("T", [40, 300])
def test_captured_backwards_with_a_given_workspace(T):
    """A linear layer's and a norm's backward captured with the caller's outputs and workspace, replayed on new
    gradients, between eager calls that use the same workspace."""
    h, N = 512, 1024
    v = fl.make(T, h, N, "bf16", seed=T)
    X, gamma, beta, _, _ = nm.make(T, h, "bf16", seed=T)
    _, mean, rstd = binding.layernorm_forward(X, gamma, beta)
    ws = torch.empty(max(binding.linear_ex_workspace_size(T, h, N), binding.layernorm_workspace_size(T, h)),
                     dtype=torch.uint8, device="cuda")
    e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    out = (e(T, h), e(h, N), e(N), e(T, N))
    nout = (e(T, h), e(h, dt=torch.float32), e(h, dt=torch.float32))
    dY = v["dY"].clone()

    def both():
        binding.fused_linear_backward(dY, X, v["W"], v["H"], activation="gelu", grad_dtype=torch.bfloat16, out=out,
                                      workspace=ws)
        binding.layernorm_backward(out[0], X, gamma, mean, rstd, out=nout, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    both()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        both()
    for s in range(4):
        dY.copy_(fl.make(T, h, N, "bf16", seed=50 + s)["dY"])
        both()
        want = [t.clone() for t in (*out, *nout)]
        ws.fill_(255)
        for t in (*out, *nout):
            t.fill_(5.0)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip((*out, *nout), want)), s


def test_workspace_must_be_aligned():
    v = fl.make(8, 64, 96, "bf16")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    with pytest.raises(binding.TPMLPError) as e:
        binding.fused_linear_backward(v["dY"], v["X"], v["W"], workspace=ws[8:])
    assert e.value.status == binding.ERR_ALIGN
    X, gamma, beta, dY, _ = nm.make(8, 64, "bf16")
    _, mean, rstd = binding.layernorm_forward(X, gamma, beta)
    with pytest.raises(binding.TPMLPError) as e:
        binding.layernorm_backward(dY, X, gamma, mean, rstd, workspace=ws[4:])
    assert e.value.status == binding.ERR_ALIGN


def test_long_sums_of_the_linear_backward():
    """Many more rows than columns: the weights' gradient sums over 40 000 rows."""
    T, K, N = 40000, 264, 136
    v = fl.make(T, K, N, "bf16", seed=4)
    dX, dW, db = binding.fused_linear_backward(v["dY"], v["X"], v["W"])
    x, y, w = v["X"].double(), v["dY"].double(), v["W"].double()
    close(dW, x.t() @ y, product_error(x.t(), y), "dW")
    close(dX, y @ w.t(), product_error(y, w.t()), "dX")
    close(db, y.sum(0), (16 + 8 + T / 1024 + 8) * U * y.abs().sum(0), "dbias")
