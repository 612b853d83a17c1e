"""Packed batches of very many sequences: more than the planning kernel takes
in one round (1,024), and long ones among them whose blocks have several runs of
512 tokens, against the 64-bit token recurrence."""
import pytest
import torch

import linear_reference as ref
from linear_bounds import DECAYS, STATE, out_bound
from test_gpu_linear import F32, PATHS, bwd, d64, fwd, inputs, rel

pytestmark = pytest.mark.gpu


def offsets(long):
    """1,300 sequences of 0, 1 or 2 tokens, the long ones put between them."""
    lens = [i % 3 for i in range(1300)]
    for at, n in long:
        lens.insert(at, n)
    return [0] + torch.tensor(lens).cumsum(0).tolist()


# long sequences (before which short one, tokens), H, Hk, dk, dv, gate.  With 12 heads and two column groups
# the tensor-core gradients cut at 1,152 and 1,024 tokens, three runs and two
CASES = [([(3, 1500), (1030, 600), (1290, 900)], 12, 3, 128, 16, "token"),
         ([(0, 2200), (1300, 700)], 12, 6, 16, 128, "head")]


@pytest.mark.parametrize("path,dtype", PATHS)
@pytest.mark.parametrize("long,H,Hk,dk,dv,gate", CASES)
def test_many_sequences(cuda_device, path, dtype, long, H, Hk, dk, dv, gate):
    cu = offsets(long)
    x = inputs(cuda_device, 41, 1, cu[-1], H, Hk, dk, dv, dtype, gate, cu)
    out, S = fwd(x, path=path)
    r, Sr = ref.forward(*d64(x["q"], x["k"], x["v"], x["g"], x["S0"]), cu=cu)
    assert rel(out, r) <= out_bound(dtype == F32, path)
    err = (S.double() - Sr).flatten(1).norm(dim=1) / Sr.flatten(1).norm(dim=1)
    assert float(err.max()) <= STATE
    got = bwd(x, path=path)
    want = ref.gradients(*d64(x["q"], x["k"], x["v"], x["g"], x["dout"], x["S0"], x["dS"]), cu=cu)
    for name, a, b in zip(("dq", "dk", "dv"), got, want):
        assert rel(a, b) <= out_bound(dtype == F32, path), (name, rel(a, b))
    err = (got[4].double() - want[4]).flatten(1).norm(dim=1) / want[4].flatten(1).norm(dim=1)
    assert float(err.max()) <= STATE
    if gate == "token":
        assert rel(got[3], want[3]) <= DECAYS
    else:  # a sum over all tokens, with signs: its terms' size counts
        g = x["g"].double().expand(1, cu[-1], H).contiguous()
        each = ref.gradients(*d64(x["q"], x["k"], x["v"]), g, *d64(x["dout"], x["S0"], x["dS"]), cu=cu)[3]
        assert float((got[3].double() - want[3]).norm()) <= DECAYS * float(each.norm()) * cu[-1] ** 0.5


@pytest.mark.parametrize("path,dtype", PATHS)
def test_a_batch_gives_what_its_sequences_give(cuda_device, path, dtype):
    """dg of a head's decay from 200 sequences at once against the sum of the calls for each sequence."""
    lens = [(i * 37) % 11 for i in range(200)]
    lens[60] = 1400
    cu = [0] + torch.tensor(lens).cumsum(0).tolist()
    x = inputs(cuda_device, 42, 1, cu[-1], 8, 4, 64, 32, dtype, "head", cu)
    whole = bwd(x, path=path)
    total, size = torch.zeros(8, dtype=torch.float64, device=cuda_device), 0.0
    for s, (a, b) in enumerate(zip(cu, cu[1:])):
        y = {n: x[n][:, a:b].contiguous() for n in ("q", "k", "v", "dout")}
        y.update(g=x["g"], S0=x["S0"][s:s + 1], dS=x["dS"][s:s + 1], cu=None)
        if b == a:
            assert torch.equal(whole[4][s], x["dS"][s])
            continue
        one = bwd(y, path=path)
        total += one[3].double()
        size += float(one[3].double().norm()) ** 2
        assert rel(whole[4][s:s + 1], one[4]) <= 2 * STATE
        for i in range(3):
            assert rel(whole[i][:, a:b], one[i]) <= 2 * out_bound(dtype == F32, path)
    assert float((whole[3].double() - total).norm()) <= 2 * DECAYS * 200 ** 0.5 * size ** 0.5
