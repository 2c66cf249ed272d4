"""Linear attention with a decay per head against its definition in float64: forward, backward, single tokens.

Bounds. Within chunks of 128 positions the kernels round P_ij = decay^(i-j) <a_i, b_j> and the state X that is
carried in to bf16 (U = 2^-8 of each, half a step) before their products; the output is rounded once. Sums are
fp32, and what a chunk adds to X on the way to the next ones takes its weighted operand in 16 bits (24 in the states that
leave a call): F = 2^-15 of the sums of absolute values covers both (256 products of 2^-24 each in a score, 2^-17 of the
operand, 2^-22 for each of the 24 sums of a chunk's share that the tensor cores cut off, 2^-24 per chunk added to a state,
over fewer than 100).
"""
import math

import pytest
import torch

from exact_attention_blackwell_tma_gb300 import binding

gpu = pytest.mark.gpu

U, F, CHUNK = 2.0 ** -8, 2.0 ** -15, 128


def definition(q, k, v, l, S0, scale):
    """One sequence: q [n, H, d], k [n, Hkv, d], v [n, Hkv, dv], S0 [Hkv, d, dv] (float64) -> o, S_n."""
    n, H, Hkv = q.shape[0], q.shape[1], k.shape[1]
    place = torch.arange(n, device=q.device, dtype=torch.float64)
    gap = place[:, None] - place[None, :]
    # 0 * inf: a token's own weight is 1 for every decay
    logs = torch.where(gap > 0, l[:, None, None] * gap.clamp(min=1), 0.0)
    D = torch.where(gap >= 0, torch.exp(logs), 0.0).repeat_interleave(H // Hkv, 0)
    kx, vx = k.repeat_interleave(H // Hkv, 1), v.repeat_interleave(H // Hkv, 1)
    into = torch.exp(l[:, None] * (place + 1)).repeat_interleave(H // Hkv, 0)
    P = torch.einsum("ihd,jhd->hij", q, kx) * D
    o = torch.einsum("hij,jhd->ihd", P, vx)
    o = o + torch.einsum("ihd,hde->ihe", into.t()[..., None] * q, S0.repeat_interleave(H // Hkv, 0))
    rest = n - 1 - place
    w = torch.exp(torch.where(rest > 0, l[:, None] * rest.clamp(min=1), 0.0))
    S = torch.einsum("jhd,jhe->hde", w.t()[..., None] * k, v)
    S = S + (S0 if n == 0 else torch.exp(l * n)[:, None, None] * S0)
    return o * scale, S


def bounds(a, b, c, l, X0, e):
    """Error bounds of sum_(j<=i) D^(i-j) <a_i, b_j> c_j + D^(i+1-e) a_i X of one state head, [m][n, width] lists over
    its members (a: one per output, or one; b and c: one pair, or one per query head), and of the final state."""
    n, X = a[0].shape[0], X0
    absX = X0.abs()
    outs = [torch.zeros((n, c[0].shape[1]), dtype=torch.float64, device=a[0].device) for _ in a]

    def power(m):
        return torch.where(m > 0, torch.exp(l * m.clamp(min=1)), 1.0)

    # chunks are counted from the sequence's first token: a walk from its last (e = 1) meets the short one first
    starts = [0, *range((n - 1) % CHUNK + 1 if e else CHUNK, n, CHUNK)] if n else []
    for s, t in zip(starts, [*starts[1:], n]):
        i = torch.arange(t - s, device=a[0].device, dtype=torch.float64)
        gap = i[:, None] - i[None, :]
        D = torch.where(gap >= 0, power(gap), 0.0)
        into = power(i + 1 - e)[:, None]
        for m, x in enumerate(a):
            x = x[s:t]
            bound = into * (U * (x.abs() @ X.abs()) + F * (x.abs() @ absX))
            for y, z in zip(b, c):
                y, z = y[s:t], z[s:t]
                bound = bound + U * ((x @ y.T * D).abs() @ z.abs()) + F * ((x.abs() @ y.abs().T * D) @ z.abs())
            outs[m][s:t] = bound
        w = power(t - s - 1 - i + e)[:, None]
        over = power(torch.tensor(float(t - s), dtype=torch.float64, device=a[0].device))
        X = over * X + sum((w * y[s:t]).T @ z[s:t] for y, z in zip(b, c))
        absX = over * absX + sum((w * y[s:t]).abs().T @ z[s:t].abs() for y, z in zip(b, c))
    return outs, F * absX


def within(got, ref, bound, what, floor=1e-7):
    got = got.double()
    assert got.shape == ref.shape, f"{what}: {got.shape}, {ref.shape}"
    assert torch.isfinite(got).all(), f"{what}: not finite"
    if got.numel():
        over = ((got - ref).abs() - bound - floor).max().item()
        assert over <= 0, f"{what}: {over:.3e} past its bound"


class Problem:
    """A batch of sequences, dense or packed, with the tensors of a call."""

    def __init__(self, lens, H, Hkv, d, dv, packed=True, states=True, logs=None, seed=0, behind=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.Hkv, self.d, self.dv, self.packed = lens, H, Hkv, d, dv, packed
        T = sum(lens) + behind

        def rows(h, w):
            x = torch.randn((T, h, w), generator=g).to(torch.bfloat16).cuda()
            return x if packed else x.unflatten(0, (len(lens), -1))

        self.q, self.k, self.v, self.do = rows(H, d), rows(Hkv, d), rows(Hkv, dv), rows(H, dv)
        self.cu = None
        if packed:
            self.cu = torch.tensor([sum(lens[:b]) for b in range(len(lens) + 1)], dtype=torch.int32).cuda()
        logs = [-2.0 ** (-8 * (h + 1) / Hkv) for h in range(Hkv)] if logs is None else logs
        self.log_decay = torch.tensor(logs, dtype=torch.float32).cuda()
        shape = (len(lens), Hkv, d, dv)
        self.state = (3 * torch.randn(shape, generator=g)).cuda() if states else None
        self.dstate = torch.randn(shape, generator=g).cuda() if states else None
        self.scale = 1 / math.sqrt(d)

    def sequences(self):
        """(b, first row, rows) of every sequence, and its tensors in float64 (requiring gradients)."""
        at = 0
        for b, n in enumerate(self.lens):
            flat = [x.flatten(0, -3)[at:at + n].double().requires_grad_() for x in (self.q, self.k, self.v)]
            S = (torch.zeros(self.Hkv, self.d, self.dv, dtype=torch.float64).cuda() if self.state is None
                 else self.state[b].double()).requires_grad_()
            yield b, at, n, flat, S
            at += n

    def logs(self):
        return self.log_decay.double().clamp(max=0.0)

    def check_forward(self, o, final, what=""):
        o, per, l = o.flatten(0, -3), self.H // self.Hkv, self.logs()
        for b, at, n, (q, k, v), S in self.sequences():
            with torch.no_grad():
                ref, last = definition(q, k, v, l, S, self.scale)
                for h in range(self.Hkv):
                    heads = list(range(h * per, (h + 1) * per))
                    e, eS = bounds([q[:, x] for x in heads], [k[:, h]], [v[:, h]], l[h], S[h], 0)
                    for x, bound in zip(heads, e):
                        within(o[at:at + n, x], ref[:, x], self.scale * bound * (1 + U) + U * ref[:, x].abs(),
                               f"{what} o of sequence {b}, head {x}")
                    if final is not None:
                        within(final[b, h], last[h], eS, f"{what} state of sequence {b}, head {h}")

    def references(self):
        """Per sequence: dq, dk, dv, dS0 by autograd through the definition."""
        for b, at, n, (q, k, v), S in self.sequences():
            o, last = definition(q, k, v, self.logs(), S, self.scale)
            do = self.do.flatten(0, -3)[at:at + n].double()
            loss = (o * do).sum()
            if self.dstate is not None:
                loss = loss + (last * self.dstate[b].double()).sum()
            yield b, at, n, (q.detach(), k.detach(), v.detach(), do), S.detach(), torch.autograd.grad(loss, (q, k, v, S))

    def check_backward(self, dq, dk, dv, dS, what=""):
        dq, dk, dv, per, l = dq.flatten(0, -3), dk.flatten(0, -3), dv.flatten(0, -3), self.H // self.Hkv, self.logs()
        for b, at, n, (q, k, v, do), S, (rq, rk, rv, rS) in self.references():
            for h in range(self.Hkv):
                heads = list(range(h * per, (h + 1) * per))
                G = (torch.zeros_like(S[h]) if self.dstate is None else self.dstate[b, h].double()) / self.scale
                back = lambda x: x.flip(0)   # noqa: E731
                eq, _ = bounds([do[:, x] for x in heads], [v[:, h]], [k[:, h]], l[h], S[h].T, 0)
                ek, _ = bounds([back(v[:, h])], [back(do[:, x]) for x in heads], [back(q[:, x]) for x in heads], l[h], G.T, 1)
                ev, eS = bounds([back(k[:, h])], [back(q[:, x]) for x in heads], [back(do[:, x]) for x in heads], l[h], G, 1)
                for x, bound in zip(heads, eq):
                    within(dq[at:at + n, x], rq[:, x], self.scale * bound * (1 + U) + U * rq[:, x].abs(), f"{what} dq {b} {x}")
                within(dk[at:at + n, h], rk[:, h], self.scale * back(ek[0]) * (1 + U) + U * rk[:, h].abs(), f"{what} dk {b} {h}")
                within(dv[at:at + n, h], rv[:, h], self.scale * back(ev[0]) * (1 + U) + U * rv[:, h].abs(), f"{what} dv {b} {h}")
                if dS is not None:
                    within(dS[b, h], rS[h], self.scale * eS, f"{what} dS {b} {h}")

    def forward(self, **kw):
        return binding.linear_forward(self.q, self.k, self.v, self.log_decay, cu_seqlens=self.cu, state=self.state, **kw)

    def backward(self, **kw):
        return binding.linear_backward(self.q, self.k, self.v, self.log_decay, self.do, cu_seqlens=self.cu,
                                       state=self.state, dstate=self.dstate, **kw)

    def check(self, what=""):
        o, final = self.forward(final_state=True)
        grads = self.backward()
        binding.check_status()
        self.check_forward(o, final, what)
        self.check_backward(*grads, what)


DIMS = [(64, 64), (128, 128), (192, 192), (192, 128), (256, 256)]


@gpu
@pytest.mark.parametrize("d,dv", DIMS)
@pytest.mark.parametrize("H,Hkv", [(2, 2), (3, 1)])
def test_packed(d, dv, H, Hkv):
    Problem([1, 0, 63, 64, 65, 200, 2], H, Hkv, d, dv, seed=d + dv + H).check()


@gpu
@pytest.mark.parametrize("d,dv", DIMS)
@pytest.mark.parametrize("states", [True, False])
def test_dense(d, dv, states):
    Problem([101, 101], 4, 2, d, dv, packed=False, states=states, seed=d).check()


@gpu
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 64, 128])
def test_dense_lengths(n):
    Problem([n] * 3, 2, 2, 64, 64, packed=False, seed=n).check()


@gpu
@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("d,dv,H,Hkv", [(64, 64, 2, 2), (128, 128, 4, 1), (192, 128, 2, 1), (256, 256, 1, 1)])
def test_many_segments(packed, d, dv, H, Hkv):
    """Sequences that several thread blocks walk, a segment each."""
    lens = [1500, 3, 2049] if packed else [1601, 1601]
    assert binding.attn_linear_workspace_size(len(lens), H, Hkv, sum(lens) if packed else lens[0], packed, d, dv, False) > 0
    Problem(lens, H, Hkv, d, dv, packed=packed, seed=d + packed).check()


@gpu
@pytest.mark.parametrize("n", [127, 128, 129, 191, 192, 257])
def test_lengths_around_a_chunk(n):
    Problem([n], 3, 1, 128, 128, seed=n).check()
    Problem([n, n], 2, 2, 128, 128, packed=False, states=False, seed=n).check()


@gpu
@pytest.mark.parametrize("d,dv,H,Hkv", [(64, 64, 6, 3), (128, 128, 2, 2), (192, 128, 3, 3)])
def test_more_runs_than_thread_blocks(d, dv, H, Hkv):
    """Ranges of units that span many short sequences and heads, empty sequences among them."""
    g = torch.Generator().manual_seed(d)
    lens = torch.randint(0, 41, (70,), generator=g).tolist() + [700] + [0, 0] + torch.randint(0, 300, (9,), generator=g).tolist()
    Problem(lens, H, Hkv, d, dv, seed=d).check()


@gpu
@pytest.mark.parametrize("packed", [True, False])
def test_runs_that_several_ranges_cut(packed):
    lens = [3000, 5, 0, 5200] if packed else [4100, 4100]
    Problem(lens, 2, 2, 128, 128, packed=packed, seed=3, states=packed).check()


@gpu
def test_offsets_that_change_between_replays():
    """A captured call reads the offsets when it runs; its segments follow them."""
    p = Problem([700, 41, 300, 1], 4, 2, 64, 64, seed=18)
    for _ in range(2):
        p.forward(final_state=True), p.backward()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, final = p.forward(final_state=True)
        grads = p.backward()
    for lens in ([700, 41, 300, 1], [0, 1, 2, 1039], [260, 261, 260, 261], [1042, 0, 0, 0]):
        p.lens = lens
        p.cu.copy_(torch.tensor([sum(lens[:b]) for b in range(5)], dtype=torch.int32))
        graph.replay()
        binding.check_status()
        p.check_forward(o, final, f"{lens}")
        p.check_backward(*grads, f"{lens}")


@gpu
@pytest.mark.parametrize("n", [90, 900])
def test_states_in_place(n):
    """The final state in state's buffer, and its gradient in dfinal's or in state's."""
    p = Problem([n, 33], 4, 2, 128, 128, seed=19)
    o, final = p.forward(final_state=True)
    *_, want = p.backward()
    state = p.state.clone()
    o2, same = binding.linear_forward(p.q, p.k, p.v, p.log_decay, cu_seqlens=p.cu, state=state, final_state=state)
    assert torch.equal(o, o2) and torch.equal(final, same)
    ws = torch.empty(binding.attn_linear_workspace_size(2, 4, 2, n + 33, True, 128, 128, True), dtype=torch.uint8, device="cuda")
    for where in ("dfinal", "state"):
        state, dfinal = p.state.clone(), p.dstate.clone()
        into = dfinal if where == "dfinal" else state
        dq, dk, dv = torch.empty_like(p.q), torch.empty_like(p.k), torch.empty_like(p.v)
        rc = binding.attn_linear_bwd(p.q, p.k, p.v, p.do, 512, 256, 256, 512, p.log_decay, state, dfinal, dq, dk, dv, into, 2, 4, 2,
                                     n + 33, 128, 128, p.scale, p.cu, ws, ws.numel())
        assert rc == binding.ATTN_OK
        binding.check_status()
        p.check_backward(dq, dk, dv, into, where)
        assert torch.equal(into, want)


@gpu
def test_outputs_at_any_16_byte_boundary():
    """Outputs that start 16 bytes into an allocation, next to bytes that stay as they are."""
    p = Problem([200], 2, 2, 128, 128, seed=20)
    flat = torch.full((200 * 2 * 128 + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = flat[8:-8].view(200, 2, 128)
    o, _ = p.forward(out=out)
    assert o.data_ptr() == out.data_ptr() and torch.equal(o, p.forward()[0])
    assert (flat[:8] == 7).all() and (flat[-8:] == 7).all()


@gpu
def test_two_calls_at_once():
    """Calls on two streams at the same time, each with a workspace of its own."""
    a, b = Problem([3000, 700], 4, 2, 128, 128, seed=21), Problem([2500], 4, 4, 64, 64, seed=22)
    want = [[*x.forward(final_state=True), *x.backward()] for x in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [[*x.forward(final_state=True, stream=s), *x.backward(stream=s)] for x, s in zip((a, b), streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for g, w in zip(got, want) for x, y in zip(g, w))
    binding.check_status()


@gpu
@pytest.mark.parametrize("packed", [True, False])
def test_decays(packed):
    """None at all, slow, fast, far below the smallest float, only the current token; above 1 counts as none."""
    Problem([700, 700], 6, 6, 64, 64, packed=packed, logs=[0.0, -1e-4, -0.7, -60.0, -math.inf, 0.25], seed=5).check()


@gpu
def test_groups():
    Problem([130, 70], 12, 2, 64, 64, seed=6).check()
    Problem([400], 9, 1, 128, 128, seed=7).check()


@gpu
def test_gradients_against_differences():
    """Of sum(o do) + sum(S_n dS) along random directions, in float64 (the loss is a polynomial of degree one in each
    tensor, so differences along one tensor are exact up to their own rounding)."""
    p = Problem([90], 2, 1, 64, 64, seed=8)
    dq, dk, dv, dS = p.backward()
    g = torch.Generator().manual_seed(9)
    for b, at, n, (q, k, v, do), S, _ in p.references():
        args = [q, k, v, S]

        def loss(*x):
            o, last = definition(*x[:3], p.logs(), x[3], p.scale)
            return ((o * do).sum() + (last * p.dstate[b].double()).sum()).item()

        for i, grad in enumerate((dq, dk, dv, dS[b])):
            for _ in range(3):
                u = torch.randn(args[i].shape, generator=g).double().cuda()
                ends = [loss(*args[:i], args[i] + s * u, *args[i + 1:]) for s in (0.5, -0.5)]
                got, size = (grad.double().reshape(u.shape) * u).sum().item(), (grad.double().reshape(u.shape) * u).norm().item()
                # independent roundings of about 2^-8 of each term: eight standard deviations of their sum
                assert abs(got - (ends[0] - ends[1])) <= 8 * 2 * U * size, (i, got, ends[0] - ends[1])


@gpu
def test_strided_rows_and_rows_behind_the_last():
    p = Problem([70, 9, 130], 4, 2, 64, 64, seed=10, behind=5)
    T = p.q.shape[0]
    fused = torch.full((T, 4 * 64 + 2 * 64 + 2 * 64 + 8), math.nan, dtype=torch.bfloat16, device="cuda")
    q, k, v = fused[:, :256].unflatten(1, (4, 64)), fused[:, 256:384].unflatten(1, (2, 64)), fused[:, 384:512].unflatten(1, (2, 64))
    n = T - 5
    for dst, src in ((q, p.q), (k, p.k), (v, p.v)):
        dst[:n] = src[:n]
    p.q, p.k, p.v = q, k, v     # the rows behind the last sequence hold NaN
    wide = torch.full((T, 4 * 64 + 16), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:n, :256] = p.do[:n].flatten(1)
    p.do = wide[:, :256].unflatten(1, (4, 64))
    outs = [torch.full((T, h, 64), 7.0, dtype=torch.bfloat16, device="cuda") for h in (4, 4, 2, 2)]
    o, final = p.forward(final_state=True, out=outs[0])
    grads = p.backward(dq=outs[1], dk=outs[2], dv=outs[3])
    binding.check_status()
    p.check_forward(o, final)
    p.check_backward(*grads)
    for x in outs:
        assert (x[n:] == 7.0).all()


def part_of(p, a, b, state, dstate):
    """Tokens [a, b) of a single sequence as a problem of its own, from `state` on."""
    x = Problem([b - a], p.H, p.Hkv, p.d, p.dv)
    x.q, x.k, x.v, x.do = (t[a:b] for t in (p.q, p.k, p.v, p.do))
    x.log_decay, x.state, x.dstate = p.log_decay, state, dstate
    return x


@gpu
def test_a_prompt_in_parts():
    """The state carries a prompt over calls of any lengths, single tokens among them, as if it were one."""
    p = Problem([333], 4, 2, 128, 128, seed=11)
    state, at = p.state.clone(), 0
    for n in (100, 1, 64, 1, 1, 166):
        x = part_of(p, at, at + n, state.clone(), None)
        if n == 1:
            o = binding.linear_step(x.q, x.k, x.v, p.log_decay, state)
        else:
            o, same = binding.linear_forward(x.q, x.k, x.v, p.log_decay, cu_seqlens=x.cu, state=state, final_state=state)
            assert same is state
        binding.check_status()
        x.check_forward(o, state, f"tokens {at} ..")
        at += n
    for _, _, _, (q, k, v), S in p.sequences():
        with torch.no_grad():
            _, last = definition(q, k, v, p.logs(), S, p.scale)
            for h in range(p.Hkv):
                within(state[0, h], last[h], bounds([q[:, h]], [k[:, h]], [v[:, h]], p.logs()[h], S[h], 0)[1], f"state {h}")


@gpu
def test_gradients_through_parts():
    """dstate passes from call to call as one backward of the whole would have it."""
    p = Problem([300], 2, 2, 64, 64, seed=12)
    _, middle = binding.linear_forward(p.q[None, :140], p.k[None, :140], p.v[None, :140], p.log_decay, state=p.state,
                                       final_state=True)
    G = p.dstate
    for a, b, state in ((140, 300, middle), (0, 140, p.state)):
        x = part_of(p, a, b, state, G)
        *grads, G = x.backward()
        binding.check_status()
        x.check_backward(*grads, G, f"tokens {a} ..")
    for b, _, n, (q, k, v, do), S, grads in p.references():
        for h in range(p.Hkv):
            _, e = bounds([k[:, h].flip(0)], [q[:, h].flip(0)], [do[:, h].flip(0)], p.logs()[h],
                          p.dstate[0, h].double() / p.scale, 1)
            within(G[0, h], grads[3][h], p.scale * e, f"gradient of the first state, head {h}")


@gpu
@pytest.mark.parametrize("d,dv", DIMS)
@pytest.mark.parametrize("B,H,Hkv", [(1, 1, 1), (5, 6, 2), (3, 11, 1)])
def test_step(d, dv, B, H, Hkv):
    p = Problem([1] * B, H, Hkv, d, dv, seed=13 + B)
    state = p.state.clone()
    o = binding.linear_step(p.q, p.k, p.v, p.log_decay, state)
    for b, at, _, (q, k, v), S in p.sequences():
        with torch.no_grad():
            ref, last = definition(q, k, v, p.logs(), S, p.scale)
            size, _ = definition(q.abs(), k.abs(), v.abs(), p.logs(), S.abs(), p.scale)
        # all fp32 until o: d products and the decay, 2^-24 each
        within(o[b], ref[0], U * ref[0].abs() + F * size[0], f"o {b}")
        within(state[b], last, 2.0 ** -21 * (last.abs() + S.detach().abs() + 16), f"state {b}")


@gpu
def test_step_decays_and_strides():
    p = Problem([1] * 3, 5, 5, 64, 64, logs=[0.0, -1e-3, -80.0, -math.inf, 0.5], seed=14)
    x = torch.full((3, 3 * 5 * 64 + 8), math.nan, dtype=torch.bfloat16, device="cuda")
    q, k, v = (x[:, 320 * i:320 * (i + 1)].unflatten(1, (5, 64)) for i in range(3))
    for dst, src in ((q, p.q), (k, p.k), (v, p.v)):
        dst.copy_(src)
    state = p.state.clone()
    o = binding.linear_step(q, k, v, p.log_decay, state)
    again, same = p.state.clone(), binding.linear_step(p.q, p.k, p.v, p.log_decay, p.state)
    assert torch.equal(o, same) and torch.equal(state, p.state)
    p.state = again
    p.check_forward(o, state)


@gpu
def test_empty_batches():
    for B, L in ((0, 5), (2, 0)):
        q = torch.zeros((B, L, 2, 64), dtype=torch.bfloat16, device="cuda")
        S = torch.randn((B, 2, 64, 64), device="cuda")
        l = torch.zeros(2, device="cuda")
        o, final = binding.linear_forward(q, q, q, l, state=S, final_state=True)
        *grads, G = binding.linear_backward(q, q, q, l, q, state=S, dstate=S)
        assert o.shape == q.shape and torch.equal(final, S) and torch.allclose(G, S, rtol=1e-6)
    e = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert binding.linear_step(e, e, e, l, torch.zeros((0, 2, 64, 64), device="cuda")).shape == (0, 2, 64)
    binding.check_status()


@gpu
def test_repeats_graphs_and_streams():
    """Bit-identical when repeated, on another stream, and captured twice with workspaces of their own."""
    p = Problem([900, 40, 1300], 4, 2, 64, 64, seed=15)
    first = [*p.forward(final_state=True), *p.backward()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = [*p.forward(final_state=True, stream=side), *p.backward(stream=side)]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = [*p.forward(final_state=True), *p.backward()]
        graphs.append((graph, outs))
    for graph, outs in graphs:
        for x in outs:
            x.zero_()
    for graph, _ in graphs:
        graph.replay()
        graph.replay()
    torch.cuda.synchronize()
    for _, outs in graphs:
        assert all(torch.equal(a, b) for a, b in zip(first, outs))


@gpu
def test_unwanted_outputs_change_nothing():
    p = Problem([500, 77], 2, 2, 64, 64, seed=16)
    o, final = p.forward(final_state=True)
    o2, none = p.forward()
    assert none is None
    p.check_forward(o, final)   # (each within its bounds: a wanted state is summed in more bits, which o may show in its last)
    p.check_forward(o2, None)
    ws = torch.empty(binding.attn_linear_workspace_size(2, 2, 2, 577, True, 64, 64, True), dtype=torch.uint8, device="cuda")
    o3, _ = p.forward(workspace=ws.fill_(255))   # whatever the workspace holds
    assert torch.equal(o2, o3)
    o4, final4 = p.forward(final_state=True, workspace=ws.fill_(255))
    assert torch.equal(o, o4) and torch.equal(final, final4)


@gpu
def test_bad_offsets_are_reported():
    p = Problem([100, 60], 2, 2, 64, 64, seed=17)
    good = p.forward(final_state=True)
    for cu in ([0, 100, 500], [0, -5, 160], [-7, 100, 160], [0, 170, 160]):
        p.cu = torch.tensor(cu, dtype=torch.int32).cuda()
        p.forward(final_state=True)
        p.backward()
        with pytest.raises(binding.AttnError) as err:
            binding.check_status()
        assert err.value.code == binding.ATTN_ERR_ARG
    p.cu = torch.tensor([0, 100, 160], dtype=torch.int32).cuda()
    assert all(torch.equal(a, b) for a, b in zip(good, p.forward(final_state=True)))
    binding.check_status()


# ---------------------------------------------------------------- refusals (no GPU needed)

def _codes(**kw):
    """Return codes of the three calls with pointers that are never read."""
    a = dict(q=4096, k=4096, v=4096, qs=128, ks=128, vs=128, l=4096, S=None, o=4096, F=None, B=1, H=2, Hkv=2, L=64, d=64, dv=64,
             scale=0.1, cu=None, ws=None, n=0)
    a.update(kw)
    b = binding
    return (b.attn_linear_fwd(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["l"], a["S"], a["o"], a["F"], a["B"],
                              a["H"], a["Hkv"], a["L"], a["d"], a["dv"], a["scale"], a["cu"], a["ws"], a["n"], stream=0),
            b.attn_linear_bwd(a["q"], a["k"], a["v"], a["o"], a["qs"], a["ks"], a["vs"], a["H"] * a["dv"], a["l"], a["S"],
                              None, a["o"], a["o"], a["o"], a["F"], a["B"], a["H"], a["Hkv"], a["L"], a["d"], a["dv"],
                              a["scale"], a["cu"], a["ws"], a["n"], stream=0),
            b.attn_linear_step(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["l"], 4096 if a["S"] is None else a["S"],
                               a["o"], a["B"], a["H"], a["Hkv"], a["d"], a["dv"], a["scale"], stream=0))


@pytest.fixture(scope="module")
def built():
    from exact_attention_blackwell_tma_gb300 import build
    return build.build()


@pytest.mark.parametrize("bad", [dict(B=-1), dict(H=3), dict(Hkv=0), dict(d=96, dv=96), dict(d=128, dv=64), dict(scale=0.0),
                                 dict(scale=math.inf), dict(scale=math.nan), dict(q=None), dict(l=None), dict(o=None),
                                 dict(qs=120), dict(ks=132), dict(vs=64), dict(B=1 << 30, L=64)])
def test_refuses_arguments(built, bad):
    codes = _codes(**bad)
    assert codes[0] == codes[1] == binding.ATTN_ERR_ARG
    if bad.get("L") is None:
        assert codes[2] == binding.ATTN_ERR_ARG
    assert binding.attn_last_error() != ""


def test_refuses_sizes_and_workspaces(built):
    assert _codes(L=-1)[:2] == (binding.ATTN_ERR_ARG,) * 2
    assert _codes(cu=4096, B=1025)[:2] == (binding.ATTN_ERR_ARG,) * 2
    assert _codes(cu=4096, B=0)[:2] == (binding.ATTN_ERR_ARG,) * 2
    assert _codes(q=4104) == (binding.ATTN_ERR_ALIGN,) * 3
    assert _codes(S=4100) == (binding.ATTN_ERR_ALIGN,) * 3
    need = binding.attn_linear_workspace_size(1, 2, 2, 4096, False, 64, 64, False)
    assert need > 0
    assert _codes(L=4096)[:2] == (binding.ATTN_ERR_WORKSPACE,) * 2
    assert _codes(L=4096, ws=4096, n=need - 1)[:2] == (binding.ATTN_ERR_WORKSPACE,) * 2
    assert _codes(L=4096, ws=4112, n=need)[:2] == (binding.ATTN_ERR_ALIGN,) * 2
    assert _codes(B=0) == (binding.ATTN_OK,) * 3
    assert binding.attn_linear_workspace_size(1, 3, 2, 4096, False, 64, 64, True) == 0
    # one segment: for a final state alone
    assert _codes(L=64, F=4096)[:2] == (binding.ATTN_ERR_WORKSPACE,) * 2
    assert binding.attn_linear_workspace_size(1, 2, 2, 64, False, 64, 64, True) == 2 * 64 * 64 * 4
    assert binding.attn_linear_workspace_size(1, 2, 2, 64, False, 64, 64, False) == 0


@gpu
def test_binding_refuses_tensors():
    def args(**kw):
        x = torch.zeros((2, 8, 2, 64), dtype=torch.bfloat16, device="cuda")
        a = dict(q=x, k=x, v=x, log_decay=torch.zeros(2, device="cuda"))
        a.update(kw)
        return a

    z = torch.zeros
    bad = [dict(q=z((2, 8, 2, 64), device="cuda")), dict(k=z((2, 8, 2, 64), dtype=torch.bfloat16)),
           dict(k=z((2, 7, 2, 64), dtype=torch.bfloat16, device="cuda")), dict(v=z((2, 8, 1, 64), dtype=torch.bfloat16, device="cuda")),
           dict(log_decay=z(3, device="cuda")), dict(log_decay=z(2, device="cuda", dtype=torch.float64)), dict(log_decay=z(2)),
           dict(state=z((2, 2, 64, 32), device="cuda")), dict(state=z((2, 2, 64, 64))),
           dict(q=z((16, 2, 64), dtype=torch.bfloat16, device="cuda")),
           dict(q=z((2, 8, 64, 2), dtype=torch.bfloat16, device="cuda").transpose(2, 3)),
           dict(cu_seqlens=torch.tensor([0, 8], dtype=torch.int32).cuda())]
    for kw in bad:
        with pytest.raises(ValueError):
            binding.linear_forward(**args(**kw))
        with pytest.raises(ValueError):
            binding.linear_backward(**args(**kw), dout=args()["q"])
    with pytest.raises(ValueError):
        binding.linear_backward(**args(), dout=z((2, 7, 2, 64), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        binding.linear_backward(**args(), dout=args()["q"], dstate=z((1, 2, 64, 64), device="cuda"))
    with pytest.raises(ValueError):
        binding.linear_forward(**args(), final_state=z((2, 2, 64, 64), device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        binding.linear_forward(**args(), workspace=z(1 << 20, dtype=torch.uint8))
    x = z((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    l, S = z(2, device="cuda"), z((3, 2, 64, 64), device="cuda")
    for kw in (dict(state=S[:2]), dict(state=S.half()), dict(k=x[:2]), dict(q=x.float()), dict(log_decay=l[:1]),
               dict(v=x[:, :1]), dict(q=x[None])):
        with pytest.raises(ValueError):
            binding.linear_step(**{**dict(q=x, k=x, v=x, log_decay=l, state=S), **kw})
    with pytest.raises(binding.AttnError):   # head dims
        binding.linear_step(x[..., :32].contiguous(), x[..., :32].contiguous(), x, l, z((3, 2, 32, 64), device="cuda"))
