"""Linear attention calls whose tensors pass 2^31 elements, and calls without a token: what lies behind the
border equals a small call's."""
import pytest
import torch

from gated_delta_rule_90_b200 import binding
from linear_bounds import DECAYS, STATE, out_bound
from test_gpu_linear import BF, rel

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("path", ["simt", "tc"])
def test_tokens_behind_2_to_the_31_elements(cuda_device, path):
    """One packed batch of which v, out, dout and dv have 2.3e9 elements; its last two sequences alone."""
    gen = torch.Generator(device=cuda_device).manual_seed(51)
    T, H, dk, dv = 140000, 128, 16, 128
    cu = [0, 60000, 139000, 139301, T]
    a, b = cu[2], cu[4]

    def tokens(h, d):  # random only where it is looked at, the rest one number
        t = torch.full((1, T, h, d), 0.01, dtype=BF, device=cuda_device)
        t[:, a:] = torch.randn(1, b - a, h, d, generator=gen, device=cuda_device).mul_(d ** -0.5).to(BF)
        return t

    q, k, v, dout = tokens(1, dk), tokens(1, dk), tokens(H, dv), tokens(H, dv)
    g = torch.rand(1, T, H, generator=gen, device=cuda_device).mul_(-0.2)
    S0, dS = (0.3 * torch.randn(4, H, dv, dk, generator=gen, device=cuda_device) for _ in range(2))
    assert v.numel() > 2 ** 31
    c = torch.tensor(cu, dtype=torch.int32, device=cuda_device)
    out, S = binding.gdr_fwd_linear(q, k, v, g, S0, cu_seqlens=c, path=path)
    got = binding.gdr_bwd_linear(q, k, v, g, dout, S0, dS, cu_seqlens=c, path=path)
    part = [t[:, a:].contiguous() for t in (q, k, v, g, dout)]
    c2 = torch.tensor([0, cu[3] - a, b - a], dtype=torch.int32, device=cuda_device)
    out2, S2 = binding.gdr_fwd_linear(*part[:4], S0[2:], cu_seqlens=c2, path=path)
    want = binding.gdr_bwd_linear(*part, S0[2:], dS[2:], cu_seqlens=c2, path=path)
    assert binding.device_status() == binding.GDR_OK
    # both sides are off by their own roundings
    assert rel(out[:, a:], out2) <= 2 * out_bound(False, path) and rel(S[2:], S2) <= 2 * STATE
    for x, y in zip(got[:3], want[:3]):
        assert rel(x[:, a:], y) <= 2 * out_bound(False, path)
    assert rel(got[3][:, a:], want[3]) <= 2 * DECAYS and rel(got[4][2:], want[4]) <= 2 * STATE


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_decode_states_behind_2_to_the_31_elements(cuda_device, dtype):
    gen = torch.Generator(device=cuda_device).manual_seed(52)
    N, H, d, last = 4200, 32, 128, 5
    S = torch.zeros(N, H, d, d, device=cuda_device)
    assert S.numel() > 2 ** 31
    q, k, v = (torch.randn(N, H, d, generator=gen, device=cuda_device).mul_(0.1).to(dtype) for _ in range(3))
    g = torch.rand(N, H, generator=gen, device=cuda_device).mul_(-0.2)
    S[-last:] = torch.randn(last, H, d, d, generator=gen, device=cuda_device)
    small = S[-last:].clone()
    out = binding.gdr_decode_step_linear(q, k, v, g, S)
    want = binding.gdr_decode_step_linear(*(t[-last:].contiguous() for t in (q, k, v, g)), small)
    assert torch.equal(out[-last:], want) and torch.equal(S[-last:], small)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("gate", ["token", "head"])
@pytest.mark.parametrize("T", [0, 40])
def test_a_packed_batch_of_empty_sequences(cuda_device, dtype, gate, T):
    """No sequence has a token (of none, or of 40 that belong to nobody): the states pass through, dg of a
    head's decay is zero, and the rows are left as they were."""
    def t(*s):
        return torch.randn(*s, device=cuda_device).to(dtype)

    q, k, v, dout = t(1, T, 2, 32), t(1, T, 2, 32), t(1, T, 4, 16), t(1, T, 4, 16)
    g = torch.full((4,) if gate == "head" else (1, T, 4), -0.1, device=cuda_device)
    S0, dS = torch.randn(3, 4, 16, 32, device=cuda_device), torch.randn(3, 4, 16, 32, device=cuda_device)
    cu = torch.zeros(4, dtype=torch.int32, device=cuda_device)
    rows = [torch.full_like(x, 7.0) for x in (v, q, k, v, g)]
    _, S = binding.gdr_fwd_linear(q, k, v, g, S0, cu_seqlens=cu, out=rows[0])
    got = binding.gdr_bwd_linear(q, k, v, g, dout, S0, dS, cu_seqlens=cu, dq=rows[1], dk=rows[2], dv=rows[3],
                                 dg=rows[4])
    assert binding.device_status() == binding.GDR_OK
    assert torch.equal(S, S0) and torch.equal(got[4], dS)
    assert all((x == 7).all() for x in rows[:4])
    assert (got[3] == (0 if gate == "head" else 7)).all()
