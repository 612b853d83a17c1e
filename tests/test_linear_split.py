"""The bounds of linear_bounds.py against planted mistakes, on the CPU: the state's
update with its operand w c split into bf16 terms by truncation, as the
tensor-core path does it, and with a term left out; an output with one rounding
to bf16 more than the path makes; the gradient of the decays summed in 32 bits
from the sequence's end instead of from the end of each 512 tokens."""
import torch

from linear_bounds import BF16_ROUND, DECAYS, STATE, out_bound

F32, F64, BF = torch.float32, torch.float64, torch.bfloat16


def truncated(x):
    """The bf16 number that keeps the upper half of x's bits, as fp32."""
    return (x.contiguous().view(torch.int32) & -65536).view(F32)


def split(x, terms):
    out = []
    for _ in range(terms):
        out.append(truncated(x))
        x = x - out[-1]
    return out, x


def rel(x, r):
    return float((x.double() - r).norm() / r.norm())


def update(seed=3, tokens=128, dk=64, dv=64):
    gen = torch.Generator().manual_seed(seed)
    k = torch.nn.functional.normalize(torch.randn(tokens, dk, generator=gen), dim=-1).to(BF).float()
    v = torch.randn(tokens, dv, generator=gen).to(BF).float()
    g = -0.1 * torch.nn.functional.softplus(torch.randn(tokens, generator=gen))
    G = g.double().cumsum(0)
    w = (G[-1] - G).float().exp()
    return k, w[:, None] * v, (G[-1] - G).exp()[:, None] * v.double()


def test_three_terms_hold_all_bits():
    _, wc, _ = update()
    terms, left = split(wc, 3)
    assert not left.any()
    assert torch.equal(terms[0] + (terms[1] + terms[2]), wc)
    assert all(torch.equal(t, t.to(BF).float()) for t in terms)


def test_a_state_with_two_terms_is_over_the_bound():
    k, wc, exact = update()
    want = exact.t() @ k.double()
    for terms, good in ((3, True), (2, False)):
        S = sum((t.double().t() @ k.double()) for t in split(wc, terms)[0]).float()
        assert (rel(S, want) <= STATE) == good
    assert 2.0 ** -18 < rel(sum(t.double().t() @ k.double() for t in split(wc, 2)[0]), want) < 2.0 ** -16


def test_one_rounding_more_is_over_the_bound():
    """Of the values just above a power of two, whose roundings are the largest: one rounding at the bound of
    one, two at the bound of two, three over it."""
    gen = torch.Generator().manual_seed(4)
    x = 1 + torch.rand(1 << 16, generator=gen) / 32
    far = torch.rand(3, 1 << 16, generator=gen) * 2 - 1  # roundings in units of their largest size
    err = [float((far[:n].sum(0) * 2.0 ** -8).double().norm() / x.double().norm()) for n in (1, 2, 3)]
    assert err[0] <= out_bound(False, "simt") and err[1] <= out_bound(False, "tc") < err[2]
    assert 0.9 * BF16_ROUND < err[0]


def test_decay_sums_that_do_not_start_again_are_over_the_bound():
    """Differences R - C that are off by 2^-22 of their terms, summed over 512 tokens and over 65,536: the
    part of dg that the decays leave has the size of 12 tokens' terms."""
    gen = torch.Generator().manual_seed(5)
    far = 2.0 ** -22 * torch.randn(65536, generator=gen, dtype=F64)
    size = 12 ** 0.5
    late = far.flip(0).cumsum(0) / size
    again = far.view(-1, 512).flip(1).cumsum(1) / size
    assert float(again.pow(2).mean()) ** 0.5 <= DECAYS < float(late.pow(2).mean()) ** 0.5
