"""The residual's epilogue where a launch both relays (long K, more than two tiles per CTA pair) and ends in split
tiles: there the relay warps, whose staging slots were hand-off buffers during the whole tiles, load residual chunks
themselves. (Bounds: fused_util.)"""
import pytest
import torch

from fused_util import U, close, product_error
from tensor_transformer_mlp_block_b200 import binding

PAIRS = 74  # CTA pairs of a B200
# rows, K, columns: 153 tiles (5 behind two full waves), and 304 (8 behind four: the double-staged kernel)
SHAPES = [(2100, 16384, 4104), (4800, 16384, 4096)]


def split_units(T, K, N):
    units = binding.schedule_units(binding.SCHED_STREAMK, -(-T // 256), -(-N // 256), -(-K // 64), PAIRS)
    return [u for u in units if u["pieces"] > 1]


@pytest.mark.parametrize("T,K,N", SHAPES)
def test_shapes_reach_the_path(T, K, N):
    """Host: the default policy plans a stream-K tail behind whole tiles that relay (K >= 2048, over 2 tiles a pair)."""
    from tensor_transformer_mlp_block_b200 import build
    build.build()
    tiles = -(-T // 256) * -(-N // 256)
    assert tiles > 2 * PAIRS and K >= 2048 and tiles % PAIRS
    assert binding.plan_schedules(T, N, K, 1)["F2"] == binding.SCHED_STREAMK  # the same product: T x N, K deep
    units = split_units(T, K, N)
    assert len({(u["mb"], u["nb"]) for u in units}) == tiles % PAIRS
    assert (SHAPES.index((T, K, N)) == 1) == (tiles >= 4 * PAIRS)


@pytest.mark.gpu
@pytest.mark.parametrize("policy", [0, 3])
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_relayed_and_split(T, K, N, policy):
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    X, W, bias, R = r(T, K).bfloat16(), (r(K, N) / K ** 0.5).bfloat16(), r(N).bfloat16(), r(T, N).bfloat16()
    binding.set_split_policy(policy)
    try:
        Y = binding.fused_linear_forward(X, W, bias, residual=R)
        x, w = X.double(), W.double()
        h = x @ w + bias.double()
        y = h + R.double()
        bound = product_error(x, w) + 2 * U * h.abs() + U * (y.abs() + R.double().abs())
        close(Y, y, bound + U * y.abs(), "Y")
        del x, w, h, y, bound
        # the same bits every time, in place too
        got, bad = torch.empty_like(Y), torch.zeros((), dtype=torch.int64, device="cuda")
        for i in range(40):
            if i % 2:
                got.copy_(R)
                binding.fused_linear_forward(X, W, bias, residual=got, out=got)
            else:
                got.fill_(9.0)
                binding.fused_linear_forward(X, W, bias, residual=R, out=got)
            bad += (got != Y).sum()
        assert int(bad) == 0
        assert binding.last_device_status() == binding.OK
    finally:
        binding.set_split_policy(0)


@pytest.mark.gpu
def test_checkpointed_block():
    """The block's second product with the residual stream, T x F times F x h, takes the same path."""
    T, F, h = SHAPES[0]
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    X, A, B = r(T, h).bfloat16(), (r(h, F) / h ** 0.5).bfloat16(), (r(F, h) / F ** 0.5).bfloat16()
    R, act = r(T, h).bfloat16(), torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
    C, S, Z = binding.forward_ckpt8(X, A, None, B, None, 1, residual=R, scratch=act)
    y, b = act.double(), B.double()
    z = y @ b + R.double()
    close(Z, z, product_error(y, b) + 2 * U * (z.abs() + R.double().abs()), "Z")
    for _ in range(20):
        again = binding.forward_ckpt8(X, A, None, B, None, 1, residual=R)
        assert all(torch.equal(a, w) for a, w in zip(again, (C, S, Z)))
    assert binding.last_device_status() == binding.OK
