"""GPU test of the gate's gradients against differences of its own forward pass in float32.

Steps are multiples of a power of two that keep every operand a bfloat16 number, and go along the gradient's
signs, so that the slope is the sum of all its entries' sizes.  With f(t) the sum of dh h at t steps,
f'(0) = (8 (f(1) - f(-1)) - (f(2) - f(-2))) / 12 but for f'''''(t) / 30.  Bounds:
- each of the values is off by at most sum |dh| e, e the bound of h (_product_cases): 18 / 12 of the largest;
- h = act(zg + t a) (zu + t b) has the fifth derivative act^(5) a^5 (zu + t b) + 5 act^(4) a^4 b, and |act^(4)|, |act^(5)| <= 4 for
  all three (the largest is 2.4);
- an entry of the gradient is off by its rounding, 2^-8 of it, and by dz's, 2^-8 of its terms, and by the errors of both products and
  of the sums, which float32 leaves below 2^-14 of its terms here.
"""
import pytest
import torch

import post_weight_quantization_gq_amd as gq
from _product_cases import BF, F32, act64, gate64, generator, normal

pytestmark = pytest.mark.gpu


def multiples(device, *shape, most, unit, seed):
    return (torch.randint(-most, most + 1, shape, generator=generator(device, seed), device=device) * unit).to(BF)


@pytest.mark.parametrize("leaf", ["x", "G", "U"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gradient_against_differences_of_the_forward_pass(device, act, leaf):
    n, d_in, d_ff = 32, 128, 72
    at = dict(x=multiples(device, n, d_in, most=30, unit=2.0 ** -4, seed=1),
              G=multiples(device, d_ff, d_in, most=63, unit=2.0 ** -8, seed=2),
              U=multiples(device, d_ff, d_in, most=63, unit=2.0 ** -8, seed=3))
    dh = normal(device, n, d_ff, seed=9, dtype=F32)
    leaves = {k: t.clone().requires_grad_() for k, t in at.items()}
    gq.ffn_gate(*leaves.values(), act=act, out_dtype=F32).backward(dh)
    grad = leaves[leaf].grad.double()
    s = (2.0 ** (-6 if leaf == "x" else -10) * torch.sign(grad)).to(BF)

    def value(t):
        moved = {**at, leaf: at[leaf] + t * s}
        assert torch.equal(moved[leaf].double(), at[leaf].double() + t * s.double())
        h = gq.ffn_gate(*moved.values(), act=act, out_dtype=F32)
        limit = gate64(*(moved[k].double() for k in "xGU"), act, d_in)[1] + 2.0 ** -24 * h.double().abs()
        return (dh.double() * h.double()).sum(), (dh.double().abs() * limit).sum()

    (f1, e1), (g1, _), (f2, e2), (g2, _) = (value(t) for t in (1, -1, 2, -2))
    slope = (8 * (f1 - g1) - (f2 - g2)) / 12
    off = 18 / 12 * 2 * torch.maximum(e1, e2)              # (the other two's bounds within twice these)
    x, G, U = (at[k].double() for k in "xGU")
    zg, zu, step = x @ G.T, x @ U.T, s.double()
    zero = torch.zeros_like(zg)
    a = step @ G.T if leaf == "x" else (x @ step.T if leaf == "G" else zero)
    b = step @ U.T if leaf == "x" else (x @ step.T if leaf == "U" else zero)
    off += (dh.double().abs() * 4 * (a.abs() ** 5 * (zu.abs() + 2 * b.abs()) + 5 * a ** 4 * b.abs())).sum() / 30 * 16
    v, d = act64(zg, act)
    dzg, dzu = (dh.double() * zu * d).abs(), (dh.double() * v).abs()
    terms = dzg @ G.abs() + dzu @ U.abs() if leaf == "x" else (dzg if leaf == "G" else dzu).T @ x.abs()
    off += (step.abs() * (2.0 ** -8 * grad.abs() + (2.0 ** -8 + 2.0 ** -14) * terms)).sum()
    got = (grad * step).sum()
    print(f"{act} {leaf}: slope {float(slope):.6g}, gradient's {float(got):.6g}, off {float(abs(got - slope)):.3g} of {float(off):.3g}", flush=True)
    assert abs(got - slope) <= off and off <= 0.1 * slope
