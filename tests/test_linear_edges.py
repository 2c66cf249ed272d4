"""Linear attention at the ends of what it takes, and how exact the states are that leave it (definitions: test_linear.py)."""
import pytest
import torch

from exact_attention_blackwell_tma_gb300 import binding
from test_linear import U, Problem, bounds, within

gpu = pytest.mark.gpu


# ------------------------------------------------------------------ scales of any size in the backward

def check_scaled(p, grads, what):
    """dq, dk, dv, dS for p.scale, of any finite size: the bounds of test_linear.py with the gradient of the state, G, as it
    is; 2^-122 for the states that are below bf16's range: half a step of 2^-133 in each of d <= 192 products with |a| < 8."""
    dq, dk, dv, dS = (x.flatten(0, -3) if i < 3 else x for i, x in enumerate(grads))
    for b, at, n, (q, k, v, do), S, (rq, rk, rv, rS) in p.references():
        for h in range(p.Hkv):
            G = torch.zeros_like(S[h]) if p.dstate is None else p.dstate[b, h].double()
            back = lambda x: x.flip(0)   # noqa: E731
            x = p.scale
            _, eS = bounds([back(k[:, h])], [back(x * q[:, h])], [back(do[:, h])], p.logs()[h], G, 1)
            ek, _ = bounds([back(v[:, h])], [back(x * do[:, h])], [back(q[:, h])], p.logs()[h], G.T, 1)
            ev, _ = bounds([back(k[:, h])], [back(x * q[:, h])], [back(do[:, h])], p.logs()[h], G, 1)
            eq, _ = bounds([do[:, h]], [v[:, h]], [k[:, h]], p.logs()[h], S[h].T, 0)
            least = 2.0 ** -122
            for name, got, ref, e in (("dq", dq[at:at + n, h], rq[:, h], x * eq[0]), ("dk", dk[at:at + n, h], rk[:, h], back(ek[0])),
                                      ("dv", dv[at:at + n, h], rv[:, h], back(ev[0]))):
                within(got, ref, e * (1 + U) + U * ref.abs(), f"{what} {name} {b} {h}", floor=least)
            within(dS[b, h], rS[h], eS, f"{what} dS {b} {h}", floor=least)


@gpu
@pytest.mark.parametrize("scale,size", [(2.0 ** -140, 0.0), (2.0 ** -140, 1.0), (2.0 ** -129, 1.0), (2.0 ** -100, 2.0 ** 60),
                                        (1e-20, 1e20), (0.3, 1.0), (2.0 ** 60, 1.0)])
@pytest.mark.parametrize("d,dv,lens", [(64, 64, [300, 0, 40]), (192, 128, [1700])])
def test_backward_of_any_scale(scale, size, d, dv, lens):
    """dfinal and the products q dO^T meet at their own sizes: scales whose reciprocal is no fp32 number among them."""
    p = Problem(lens, 2, 2, d, dv, seed=51)
    p.scale = scale
    p.dstate = None if size == 0 else p.dstate * size
    grads = p.backward(scale=scale)
    binding.check_status()
    check_scaled(p, grads, f"scale {scale}")


@gpu
def test_gradient_of_a_sequence_without_tokens():
    """It is that of its final state, to the bit."""
    p = Problem([0, 200, 0], 4, 2, 128, 128, seed=52)
    *_, dS = p.backward()
    assert torch.equal(dS[0], p.dstate[0]) and torch.equal(dS[2], p.dstate[2]) and not torch.equal(dS[1], p.dstate[1])
    binding.check_status()
