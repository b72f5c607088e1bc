"""Which forward calls need a workspace: only those in which some product splits its tiles."""
import pytest
import torch

from tensor_transformer_mlp_block_b200 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _auto_policy():
    yield
    binding.set_split_policy(0)


def call(v, out, p, ws):
    """tp_mlp_fwd_ckpt8 itself, bf16 and erf GeLU."""
    T, h = v["X"].shape
    F = v["A"].shape[1]
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    return binding.lib().tp_mlp_fwd_ckpt8(
        *(ptr(v[k]) for k in ("X", "A", "a", "B", "b", "R")), *(ptr(t) for t in out), T, h, F, p, 0, 0, ptr(ws),
        0 if ws is None else ws.nbytes, torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("policy,p", [(0, 1), (2, 2), (3, 1)])
@pytest.mark.parametrize("T", [1, 64, 128, 129])
def test_few_rows_need_none(T, policy, p):
    """h = 4096 forbids splitting the first product; the second (K = 16384, 16 tiles, planned as a stream-K tail or
    by shards) is the few-row kernel's up to 128 rows. From 129 on it splits and the call says so."""
    h, F = 4096, 16384
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    v = dict(X=r(T, h), A=r(h, F) / 64, a=r(F), B=r(F, h) / 128, b=r(h), R=r(T, h))
    binding.set_split_policy(policy)
    assert binding.plan_schedules(T, h, F, p)["F2"] != binding.SCHED_TILES
    (c, s) = binding.ckpt8_shapes(T, F)
    new = lambda: [torch.zeros(c, dtype=torch.int8, device="cuda"),  # noqa: E731
                   torch.zeros(s, dtype=torch.uint8, device="cuda"),
                   torch.zeros(T, F, dtype=torch.bfloat16, device="cuda"),
                   torch.zeros(T, h, dtype=torch.bfloat16, device="cuda")]
    full = torch.empty(binding.ckpt8_workspace_size(T, h, F, p), dtype=torch.uint8, device="cuda")
    want, got = new(), new()
    assert call(v, want, p, full) == binding.OK
    launches = binding.launch_count()
    if T <= 128:
        assert call(v, got, p, None) == binding.OK
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    else:
        assert call(v, got, p, None) == binding.ERR_WORKSPACE
        assert binding.launch_count() == launches
    assert binding.last_device_status() == binding.OK
