"""What the pre-norm block's entry points refuse, before any launch (no GPU needed): sizes, null pointers, types,
activations; and the host-side workspace sizes."""
import ctypes

import pytest
import torch

from tensor_transformer_mlp_block_b200 import binding

VP = ctypes.c_void_p(256)  # never dereferenced: validation fails first
NO = None


@pytest.fixture(scope="module")
def lib():
    from tensor_transformer_mlp_block_b200 import build
    build.build()
    before = binding.launch_count()
    yield binding.lib()
    assert binding.launch_count() == before


def norm_fwd(lib, X=VP, Y=VP, mean=VP, rstd=VP, T=4, h=8, eps=1e-5, dt=0):
    return lib.tp_layernorm_fwd(X, NO, NO, Y, mean, rstd, T, h, eps, dt, NO)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(h=0), dict(h=-8), dict(dt=2), dict(X=NO), dict(Y=NO), dict(mean=NO), dict(rstd=NO),
    dict(eps=-1e-5), dict(eps=float("nan")), dict(eps=float("inf")),
])
def test_layernorm_forward_refuses(lib, bad):
    assert norm_fwd(lib, **bad) == binding.ERR_INVALID


@pytest.mark.parametrize("bad", [dict(T=2 ** 31), dict(h=2 ** 31)])
def test_layernorm_forward_refuses_sizes(lib, bad):
    assert norm_fwd(lib, **bad) == binding.ERR_UNSUPPORTED


def test_layernorm_forward_refuses_overlap(lib):
    """4 × 8 bf16: X at 4096..4160. An output that shares a byte with it, or with another output, is refused."""
    at = ctypes.c_void_p
    for y in (4096, 4096 - 63, 4096 + 63):
        assert norm_fwd(lib, X=at(4096), Y=at(y), mean=at(8192), rstd=at(8208)) == binding.ERR_INVALID
    assert norm_fwd(lib, X=at(4096), Y=at(256), mean=at(4156), rstd=at(8208)) == binding.ERR_INVALID
    assert norm_fwd(lib, X=at(4096), Y=at(256), mean=at(8192), rstd=at(8204)) == binding.ERR_INVALID
    if not torch.cuda.is_available():  # side by side is no overlap: the next refusal is the missing GPU
        for y in (4096 - 64, 4096 + 64):
            assert norm_fwd(lib, X=at(4096), Y=at(y), mean=at(8192), rstd=at(8208)) == binding.ERR_CUDA


@pytest.mark.parametrize("i", range(9))
def test_layernorm_backward_refuses_null(lib, i):
    args = [VP] * 9
    args[i] = NO
    st = lib.tp_layernorm_bwd(*args, 4, 8, 0, VP, 0, NO)
    if i in (2, 5):  # gamma and dR may be null: the next refusal is the workspace or the missing GPU
        assert st in (binding.ERR_WORKSPACE, binding.ERR_CUDA, binding.ERR_UNSUPPORTED)
    else:
        assert st == binding.ERR_INVALID
    assert lib.tp_layernorm_bwd(*[VP] * 9, -1, 8, 0, VP, 0, NO) == binding.ERR_INVALID
    assert lib.tp_layernorm_bwd(*[VP] * 9, 4, 0, 0, VP, 0, NO) == binding.ERR_INVALID
    assert lib.tp_layernorm_bwd(*[VP] * 9, 4, 8, 5, VP, 0, NO) == binding.ERR_INVALID


def test_layernorm_workspace(lib):
    assert binding.layernorm_workspace_size(-1, 8) == 0
    assert binding.layernorm_workspace_size(4, 0) == 0
    for T, h in [(0, 8), (1, 1), (517, 1000), (8192, 4096), (3, 100001)]:
        for dt in (torch.bfloat16, torch.float32):
            n = binding.layernorm_workspace_size(T, h, dt)
            assert n >= 2 * 4 * h and n % 256 == 0
    # bounded by the GPU's blocks, not by the rows
    assert binding.layernorm_workspace_size(10 ** 6, 4096) == binding.layernorm_workspace_size(10 ** 7, 4096)


def linear_fwd(lib, X=VP, W=VP, H=NO, Y=VP, T=4, K=16, N=8, p=1, split=0, dt=0, act=2):
    n = lib.tpmlp_linear_ex_workspace_size(4, 16, 8, 1, 0, 0)
    return lib.tp_linear_fwd_ex(X, W, NO, NO, H, Y, T, K, N, p, split, dt, act, VP, n + (1 << 20), NO)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(K=0), dict(N=0), dict(p=0), dict(p=3), dict(split=2), dict(dt=3), dict(split=1, p=3)])
def test_linear_forward_refuses(lib, bad):
    assert linear_fwd(lib, **bad) == binding.ERR_INVALID


def test_linear_workspace(lib):
    assert binding.linear_ex_workspace_size(4, 16, 8, 3) == 0
    assert binding.linear_ex_workspace_size(4, 0, 8) == 0
    assert binding.linear_ex_workspace_size(4096, 1024, 4096) >= 32 * 4096 * 4


def test_ckpt8_refuses(lib):
    assert lib.tpmlp_ckpt8_encode(VP, VP, VP, -1, 8, 0, NO) == binding.ERR_INVALID
    assert lib.tpmlp_ckpt8_encode(VP, VP, VP, 4, 0, 0, NO) == binding.ERR_INVALID
    assert lib.tpmlp_ckpt8_encode(VP, VP, VP, 4, 8, 2, NO) == binding.ERR_INVALID
    assert lib.tpmlp_ckpt8_encode(NO, VP, VP, 4, 8, 0, NO) == binding.ERR_INVALID
    assert lib.tpmlp_ckpt8_decode(VP, NO, VP, 4, 8, 0, NO) == binding.ERR_INVALID
    assert lib.tpmlp_ckpt8_decode(VP, VP, VP, 2 ** 31, 8, 0, NO) == binding.ERR_UNSUPPORTED
    assert lib.tpmlp_ckpt8_decode(VP, VP, VP, 4, 2 ** 31 - 1, 0, NO) == binding.ERR_UNSUPPORTED
    for bad in (dict(T=-1), dict(h=0), dict(F=0), dict(p=3), dict(dt=2), dict(act=2)):
        a = dict(T=4, h=8, F=16, p=1, dt=0, act=0) | bad
        assert lib.tp_mlp_fwd_ckpt8(*[VP] * 10, a["T"], a["h"], a["F"], a["p"], a["dt"], a["act"], VP, 1 << 30,
                                    NO) == binding.ERR_INVALID, bad
        assert lib.tp_mlp_bwd_ckpt8(*[VP] * 13, a["T"], a["h"], a["F"], a["p"], a["dt"], 1, a["act"], VP, 1 << 30,
                                    NO) == binding.ERR_INVALID, bad


def test_ckpt8_workspace(lib):
    """The block's own: the 8-bit copy needs no more."""
    for args in [(37, 12, 44, 2), (256, 64, 128, 2), (8192, 4096, 16384, 2)]:
        assert binding.ckpt8_workspace_size(*args) == binding.workspace_size(*args) > 0
    assert binding.ckpt8_workspace_size(256, 64, 128, 3) == 0


def test_binding_refuses_cpu_tensors_and_shapes():
    X = torch.zeros(4, 8, dtype=torch.bfloat16)
    v = torch.zeros(8, dtype=torch.bfloat16)
    st = torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        binding.layernorm_forward(X, v, v)
    with pytest.raises(ValueError, match="CUDA"):
        binding.layernorm_backward(X, X, v, st, st)
    with pytest.raises(ValueError, match="CUDA"):
        binding.fused_linear_forward(X, X.t().contiguous(), None)
    with pytest.raises(ValueError, match="CUDA"):
        binding.fused_linear_backward(X, X, X)
    with pytest.raises(ValueError, match="CUDA"):
        binding.forward_ckpt8(X, X, None, X, None, 1)
    with pytest.raises(ValueError, match="CUDA"):
        binding.ckpt8_encode(X)
    with pytest.raises(ValueError, match="two dimensions"):
        binding.ckpt8_encode(v)


def test_format_of_the_reference():
    """The tests' own 8-bit form: the scale is the smallest that fits, ties to even, special values."""
    from fused_util import eight_bit_values, eight_bits
    x = torch.zeros(7, 33, dtype=torch.float64)
    x[0, 0] = 127.0        # e = 0
    x[1, 0] = 127.5        # rounds to 128: e = 1
    x[2, 0] = 127.49
    x[2, 1] = 0.5          # tie to 0
    x[2, 2] = 1.5          # tie to 2
    x[3, 0] = float("nan")
    x[3, 32] = 1.0         # the next block is untouched
    x[4, 5] = -float("inf")
    x[5, 0] = 2.0 ** -140  # below the smallest scale: reads as zero
    x[6, 0] = 3.4e38       # finite, but 64·2^122 is not
    C, S = eight_bits(x)
    assert S[0].tolist() == [127, 128, 127, 255, 255, 0, 255]
    assert C[0, 0] == 127 and C[1, 0] == 64 and C[2, :3].tolist() == [127, 0, 2]
    v = eight_bit_values(C, S, 33)
    assert v[3, :32].isnan().all() and v[3, 32] == 1.0 and v[4, :32].isnan().all() and v[5, 0] == 0
    assert v[6, :32].isnan().all()
    y, s = eight_bits(torch.full((1, 1), 127.4 * 2.0 ** 121, dtype=torch.float64))
    assert y[0, 0] == 127 and s[0, 0] == 127 + 121
