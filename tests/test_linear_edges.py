"""Linear attention at the ends of what it takes, and how exact the states are that leave it (definitions: test_linear.py)."""
import subprocess
import sys

import pytest
import torch

from exact_attention_blackwell_tma_gb300 import binding
from test_linear import DIMS, U, Problem, bounds, within

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


# ------------------------------------------------------------------ sizes of the workspace

@pytest.fixture(scope="module")
def built():
    from exact_attention_blackwell_tma_gb300 import build
    return build.build()


def test_size_of_refused_head_dims(built):
    """Head dims that the calls refuse have no size; the query returns (asked in a process of its own)."""
    dims = [(96, 96), (9792, 9792), (64, 9792), (1 << 20, 1 << 20), (128, 64), (128, 192), (320, 320), (0, 64), (-64, -64),
            (2 ** 31 - 1, 2 ** 31 - 1)]
    code = ("from exact_attention_blackwell_tma_gb300 import binding as b\n"
            f"for d, e in {dims}:\n"
            "    print([b.attn_linear_workspace_size(1, 1, 1, 128, p, d, e, f) for p in (0, 1) for f in (0, 1)], flush=True)")
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, f"ended with {run.returncode} after {run.stdout!r}"
    assert run.stdout.split("\n")[:-1] == ["[0, 0, 0, 0]"] * len(dims)


def test_size_of_supported_head_dims(built):
    for d, d_v in DIMS:
        assert binding.attn_linear_workspace_size(1, 1, 1, 128, False, d, d_v, True) == d * d_v * 4


@gpu
@pytest.mark.parametrize("d", [96, 9792])
def test_tensors_of_refused_head_dims(d):
    x, l = torch.zeros((1, 2, 1, d), dtype=torch.bfloat16, device="cuda"), torch.zeros(1, device="cuda")
    for call in (lambda: binding.linear_forward(x, x, x, l), lambda: binding.linear_backward(x, x, x, l, x)):
        with pytest.raises(binding.AttnError) as err:
            call()
        assert err.value.code == binding.ATTN_ERR_ARG
