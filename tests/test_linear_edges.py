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


# ------------------------------------------------------------------ the states that leave a call, in fp32

def state_of(k, v, l, S0):
    """S_n of one head from its definition in float64, and the sum of the absolute values of its terms."""
    n = k.shape[0]
    place = torch.arange(n, device=k.device, dtype=torch.float64)
    w = torch.exp(l * (n - 1 - place))[:, None]
    over = torch.exp(l * n)
    return (w * k).T @ v + over * S0, (w * k.abs()).T @ v.abs() + over * S0.abs()


@gpu
@pytest.mark.parametrize("d,dv", DIMS)
@pytest.mark.parametrize("n", [2, 7, 16])
def test_states_of_few_tokens(d, dv, n):
    """Element by element. A product k_s v_s takes its decay as exp2 (2 units of 2^-23) of an exponent of at most 11.6, which is
    rounded twice (2 11.6 ln 2 2^-24), and in fp32 (2^-24); its three bf16 terms hold all of it, and 16 tokens are one sum of
    the tensor cores for each, cut off at most 2^-22 below: 2^-22 + 16.1 2^-24 + 2^-24 + 3 2^-22, below 2^-18.9 of the terms.
    Two terms leave up to 2^-17 of a product."""
    p = Problem([n], 2, 2, d, dv, logs=[-0.3, -0.5], states=False, seed=61 + n)
    _, final = p.forward(final_state=True)
    p.state, scale = torch.zeros_like(final), 1.0
    dq, dk, dv_, dS = p.backward(scale=scale)
    binding.check_status()
    zero = torch.zeros_like(final[0, 0], dtype=torch.float64)
    for h in range(2):
        l = p.logs()[h]
        for name, got, (ref, size) in (
                ("S", final[0, h], state_of(p.k[:, h].double(), p.v[:, h].double(), l, zero)),
                # dS_0 = D (q_1 dO_1^T + D q_2 dO_2^T ..): a walk from the last token on, with one more factor of D
                ("dS", dS[0, h], [torch.exp(l) * x for x in state_of(p.q[:, h].flip(0).double(), p.do[:, h].flip(0).double(), l, zero)])):
            within(got, ref, 2.0 ** -18.9 * size, f"{name} {h}", floor=1e-30)


@gpu
@pytest.mark.parametrize("d,dv,H,Hkv,lens,packed", [
    (64, 64, 2, 2, [5000], True), (128, 128, 8, 2, [3000, 700, 2100], True), (128, 128, 4, 4, [6000, 6000], False),
    (192, 128, 4, 1, [4000, 90], True), (256, 256, 2, 1, [2500], True), (64, 64, 12, 1, [130, 1, 900], True)])
def test_states_of_many_tokens(d, dv, H, Hkv, lens, packed):
    """Relative error of a state as a whole, |got - ref|_2 / |ref|_2. A chunk's share is 24 sums of the tensor cores, each cut
    off by half a unit on average, at most 2^-24 of it: 24 2^-24 = 1.43e-6. The decay over a chunk is off by 2^-22 = 0.24e-6, and
    the slowest head here remembers two chunks. Two bf16 terms instead of three are off by 2.4e-6 (the same in a simulation of
    a million products)."""
    p = Problem(lens, H, Hkv, d, dv, packed=packed, seed=71)
    scale = 1.0
    _, final = p.forward(final_state=True)
    *_, dS = p.backward(scale=scale)
    binding.check_status()
    per, flat = H // Hkv, [x.flatten(0, -3).double() for x in (p.q, p.k, p.v, p.do)]
    at = 0
    for b, n in enumerate(lens):
        q, k, v, do = (x[at:at + n] for x in flat)
        at += n
        for h in range(Hkv):
            l = p.logs()[h]
            ref, _ = state_of(k[:, h], v[:, h], l, p.state[b, h].double())
            back = torch.exp(l * n) * p.dstate[b, h].double()
            for x in range(h * per, (h + 1) * per):
                back = back + torch.exp(l) * state_of(q[:, x].flip(0), do[:, x].flip(0), l, torch.zeros_like(ref))[0]
            for name, got, want in (("S", final[b, h], ref), ("dS", dS[b, h], back)):
                err = ((got.double() - want).norm() / want.norm()).item()
                assert err <= 1.7e-6, f"{name} of sequence {b}, head {h}: {err:.3e}"
