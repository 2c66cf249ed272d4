"""Local windows with sinks (forward and backward) against plain float64 attention,
element by element within bounds that count the bf16 roundings."""
import math

import pytest
import torch

from exact_attention_blackwell_tma_gb300 import binding, inputs
from _plain import assert_lse, assert_within, attention, gradients, visible


def _seqs(t, cu, cuk):
    """Per-sequence (query rows, key rows) of a dense or packed problem as index pairs."""
    if cu is None:
        return [((b,), (b,)) for b in range(t["q"].shape[0])]
    cuk = cu if cuk is None else cuk
    return [((slice(int(cu[b]), int(cu[b + 1])),), (slice(int(cuk[b]), int(cuk[b + 1])),)) for b in range(len(cu) - 1)]


def check(t, causal, window, sinks, what, scale=None, cu=None, cuk=None, deterministic=False, grad=True):
    d = t["q"].shape[-1]
    scale = float(torch.tensor(1 / math.sqrt(d), dtype=torch.float32)) if scale is None else scale
    g = {n: x.cuda() for n, x in t.items()}
    kw = dict(causal=causal, scale=scale, window=window, sinks=sinks, cu_seqlens=None if cu is None else cu.cuda(),
              cu_seqlens_k=None if cuk is None else cuk.cuda())
    o, lse = binding.forward(g["q"], g["k"], g["v"], **kw)
    grads = binding.backward(g["q"], g["k"], g["v"], o, lse, g["do"], deterministic=deterministic, **kw) if grad else ()
    binding.check_status()
    for b, (rq, rk) in enumerate(_seqs(t, cu, cuk)):
        q, k, v, do = (t[n][r].double() for n, r in (("q", rq), ("k", rk), ("v", rk), ("do", rq)))
        ok = visible(q.shape[0], k.shape[0], causal, window, sinks)
        f = attention(q, k, v, ok, scale)
        name = f"{what} sequence {b}"
        assert_within(o[rq], f["o"], f["bound"], f"{name} O")
        assert_lse(lse[rq] if cu is None else lse[:, rq[0]], f["lse"], name)
        if grad:
            r = gradients(q, k, v, do, ok, scale)
            for n, x, at in zip(("dq", "dk", "dv"), grads, (rq, rk, rk)):
                assert_within(x[at], r[n], r[n + "_bound"], f"{name} {n}")
    return o, lse, grads


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [((0, 0), 1), ((5, 0), 4), ((127, 0), 128), ((128, 0), 129), ((200, 0), 300),
                                          ((64, 64), 3), ((300, -1), 7), ((1000, 0), 5), ((50, 0), 10 ** 9),
                                          ((2 ** 31 - 1, 2 ** 31 - 1), 4)])
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (192, 192), (256, 256), (192, 128)])
def test_window_with_sinks(d, dv, window, sinks):
    t = inputs.small(B=2, H=2, L=513, d=d, dv=dv, seed=171)
    check(t, False, window, sinks, f"d={d}/{dv} window={window} sinks={sinks}")


@pytest.mark.gpu
@pytest.mark.parametrize("sinks", [1, 130])
@pytest.mark.parametrize("L", [1, 2, 77, 129, 255, 257, 900])
def test_lengths(L, sinks):
    t = inputs.small(B=2, H=2, L=L, d=128, seed=172)
    check(t, True, (100, 0), sinks, f"L={L} sinks={sinks}", scale=0.09)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Lq,Lk", [(300, 77), (77, 300), (513, 129), (1, 700), (3, 1)])
@pytest.mark.parametrize("d", [64, 256])
def test_rectangular(d, Lq, Lk, causal):
    """More queries than keys leaves causal rows without a key: O = 0, LSE = -inf, dQ = 0."""
    t = inputs.small(B=1, H=2, L=Lq, Lk=Lk, d=d, seed=173)
    check(t, causal, (40, 3), 9, f"Lq={Lq} Lk={Lk} causal={causal}")


@pytest.mark.gpu
@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (192, 128), (256, 256)])
@pytest.mark.parametrize("H,Hkv", [(8, 2), (3, 1)])
def test_grouped_heads(H, Hkv, d, dv, deterministic):
    t = inputs.small(B=1, H=H, L=800, d=d, dv=dv, seed=174, Hkv=Hkv)
    check(t, True, (200, 0), 20, f"grouped d={d} det={deterministic}", deterministic=deterministic)


@pytest.mark.gpu
@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("d", [64, 128, 192])
def test_packed_sequences(d, deterministic):
    """Sequences of their own query and key lengths, empty ones among them; sinks count from each sequence's start."""
    lq, lk = [1, 128, 200, 513, 0, 300, 700], [300, 1, 200, 129, 77, 256, 700]
    cu, cuk = inputs.cu_seqlens(lq), inputs.cu_seqlens(lk)
    g = torch.Generator("cpu").manual_seed(175)
    r = lambda rows, h: torch.randn(rows, h, d, generator=g).to(torch.bfloat16)  # noqa: E731
    t = {"q": r(int(cu[-1]), 4), "k": r(int(cuk[-1]), 2), "v": r(int(cuk[-1]), 2), "do": r(int(cu[-1]), 4)}
    check(t, True, (60, 0), 70, f"packed d={d} det={deterministic}", cu=cu, cuk=cuk, deterministic=deterministic)


@pytest.mark.gpu
@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (192, 128), (256, 256)])
def test_sink_blocks_in_many_parts(d, dv, deterministic):
    """A short window over a long sequence: each sink block's queries are worked on in several parts, dense and
    grouped, and packed with sequences that have fewer key blocks than sinks."""
    t = inputs.small(B=1, H=4, L=2500, d=d, dv=dv, seed=182, Hkv=2)
    check(t, True, (20, 0), 200, f"parts d={d} det={deterministic}", deterministic=deterministic)
    lens = [1900, 0, 90, 1300]
    cu = inputs.cu_seqlens(lens)
    g = torch.Generator("cpu").manual_seed(183)
    r = lambda h, w: torch.randn(int(cu[-1]), h, w, generator=g).to(torch.bfloat16)  # noqa: E731
    t = {"q": r(2, d), "k": r(2, d), "v": r(2, dv), "do": r(2, dv)}
    check(t, True, (30, 0), 150, f"packed parts d={d} det={deterministic}", cu=cu, deterministic=deterministic)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_deterministic_backward_repeats(d):
    t = {n: x.cuda() for n, x in inputs.small(B=1, H=4, L=2048, d=d, seed=176).items()}
    o, lse = binding.forward(t["q"], t["k"], t["v"], causal=True, window=(500, 0), sinks=5)
    runs = [binding.backward(t["q"], t["k"], t["v"], o, lse, t["do"], causal=True, window=(500, 0), sinks=5,
                             deterministic=True) for _ in range(3)]
    binding.check_status()
    for again in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], again))


@pytest.mark.gpu
@pytest.mark.parametrize("d,dv", [(64, 64), (192, 192), (192, 128)])
@pytest.mark.parametrize("packed", [False, True])
def test_rows_with_few_keys_keep_their_precision(d, dv, packed):
    """Two and three keys per row: the cancellation in dS = P (dP - D) does not bring out the rounding of O.
    dQ then errs by dS's rounding to bf16 (rms U / 2, uniform over half a step either way of at most U, so below
    U / sqrt(3)) and its own; together less than sqrt(2 / 3) U = 3.2e-3 relative L2, taken with a quarter to spare."""
    lens = [3] * 40 if packed else [600]
    cu = inputs.cu_seqlens(lens) if packed else None
    g = torch.Generator("cpu").manual_seed(184)
    r = lambda h, w: torch.randn(*((sum(lens),) if packed else (1, 600)), h, w, generator=g).to(torch.bfloat16)  # noqa: E731
    t = {"q": r(4, d), "k": r(2, d), "v": r(2, dv), "do": r(4, dv)}
    window = (50, 0) if packed else (0, 0)
    _, _, grads = check(t, True, window, 1, "few keys", cu=cu)
    ok = visible(lens[0], lens[0], True, window, 1)
    scale = float(torch.tensor(1 / math.sqrt(d), dtype=torch.float32))
    refs = [gradients(*(t[n][x].double() for n in ("q", "k", "v", "do")), ok, scale)
            for x in ([slice(i, i + 3) for i in range(0, 120, 3)] if packed else [0])]
    for n, got in zip(("dq", "dk"), grads):
        ref = torch.cat([x[n] for x in refs])
        rel = ((got.double().cpu().reshape(ref.shape) - ref).norm() / ref.norm()).item()
        assert rel <= 4.0e-3, f"{n}: {rel:.2e}"


@pytest.mark.gpu
def test_no_left_bound_ignores_sinks():
    t = {n: x.cuda() for n, x in inputs.small(B=1, H=2, L=600, d=128, seed=177).items()}
    a = binding.forward(t["q"], t["k"], t["v"], causal=True)
    b = binding.forward(t["q"], t["k"], t["v"], causal=True, sinks=9)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
def test_window_and_sinks_over_everything_match_causal():
    """sinks covering every key give the causal result whatever the window."""
    t = inputs.small(B=1, H=2, L=700, d=64, seed=178)
    check(t, True, (3, 0), 700, "sinks everywhere")
    g = {n: x.cuda() for n, x in t.items()}
    a, _ = binding.forward(g["q"], g["k"], g["v"], causal=True)
    b, _ = binding.forward(g["q"], g["k"], g["v"], causal=True, window=(3, 0), sinks=700)
    assert (a.float() - b.float()).abs().max() <= 2 * 2.0 ** -8 * a.float().abs().max()


@pytest.mark.gpu
def test_gradients_against_differences():
    """Directional differences of the float64 loss (central, step 1e-4: error ~1e-8) against the kernel's gradients."""
    t = inputs.small(B=1, H=2, L=150, d=64, seed=179)
    _, _, grads = check(t, True, (20, 0), 3, "differences")
    ok, scale = visible(150, 150, True, (20, 0), 3), float(torch.tensor(1 / 8.0))
    x = {n: t[n][0].double() for n in ("q", "k", "v", "do")}
    g = torch.Generator("cpu").manual_seed(180)

    def loss(**kw):
        y = dict(x, **kw)
        return (attention(y["q"], y["k"], y["v"], ok, scale)["o"] * x["do"]).sum()

    r = gradients(x["q"], x["k"], x["v"], x["do"], ok, scale)
    for n, grad in zip(("q", "k", "v"), grads):
        step = torch.randn(x[n].shape, generator=g, dtype=torch.float64)
        diff = (loss(**{n: x[n] + 1e-4 * step}) - loss(**{n: x[n] - 1e-4 * step})) / 2e-4
        dot = (grad[0].double().cpu() * step).sum()
        assert abs(diff - dot) <= (r[f"d{n}_bound"] * step.abs()).sum() + 1e-4


@pytest.mark.gpu
def test_captured_forward_and_backward_replay():
    t = {n: x.cuda() for n, x in inputs.small(B=1, H=4, L=500, d=128, seed=181, Hkv=2).items()}
    kw = dict(causal=True, window=(90, 0), sinks=6)
    o, lse = binding.forward(t["q"], t["k"], t["v"], **kw)
    ref = binding.backward(t["q"], t["k"], t["v"], o, lse, t["do"], deterministic=True, **kw)
    out, l2 = torch.empty_like(o), torch.empty_like(lse)
    grads = [torch.empty_like(x) for x in ref]
    ws = torch.empty(binding.attn_bwd_sinks_workspace_size(1, 4, 2, 500, 500, 128, 128, 1, 90, 0, 6, 1), dtype=torch.uint8,
                     device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.forward(t["q"], t["k"], t["v"], out=out, lse=l2, **kw)
        binding.backward(t["q"], t["k"], t["v"], out, l2, t["do"], deterministic=True, workspace=ws, dq=grads[0],
                         dk=grads[1], dv=grads[2], **kw)
    for _ in range(2):
        for x in (out, *grads):
            x.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o) and torch.equal(l2, lse)
    assert all(torch.equal(a, b) for a, b in zip(grads, ref))


def test_refusals():
    """Arguments are checked on the host, before the device is touched."""
    from exact_attention_blackwell_tma_gb300 import build
    build.build()
    lib, x = binding.load(), 1 << 20
    fwd = lambda sinks, wl=5, cuq=None, cuk=None, d=64, p=x: lib.attn_fwd_sinks(  # noqa: E731
        p, x, x, x, x, 1, 2, 1, 64, 64, d, d, 0.1, 1, wl, -1, sinks, cuq, cuk, None)
    assert fwd(-1) == binding.ATTN_ERR_ARG and "sinks" in binding.last_error()
    assert fwd(4, wl=-2) == binding.ATTN_ERR_ARG
    assert fwd(4, cuk=x) == binding.ATTN_ERR_ARG
    assert fwd(4, d=96) == binding.ATTN_ERR_ARG
    assert fwd(4, p=x + 2) == binding.ATTN_ERR_ALIGN
    assert fwd(4, p=None) == binding.ATTN_ERR_ARG
    need = lib.attn_bwd_sinks_workspace_size(1, 2, 1, 64, 64, 64, 64, 1, 5, -1, 4, 0)
    bwd = lambda sinks, ws: lib.attn_bwd_sinks(*([x] * 9), 1, 2, 1, 64, 64, 64, 64, 0.1, 1, 5, -1, sinks,  # noqa: E731
                                               None, None, 0, x, ws, None)
    assert bwd(-3, need) == binding.ATTN_ERR_ARG
    assert bwd(4, need - 1) == binding.ATTN_ERR_WORKSPACE
    t = torch.zeros(1)
    with pytest.raises(ValueError):
        binding._no_block_mask(t)


def test_mask_arithmetic_on_the_host(tmp_path):
    import os
    import subprocess
    from exact_attention_blackwell_tma_gb300 import build
    here = os.path.dirname(os.path.abspath(__file__))
    exe = str(tmp_path / "sinks_host")
    subprocess.run([build.nvcc(), "-std=c++17", "-O2", "-I", build.CSRC, "-I", build.INCLUDE,
                    os.path.join(here, "sinks_host.cu"), "-o", exe], check=True, capture_output=True)
    assert subprocess.run([exe], capture_output=True, text=True).stdout == "0 disagreements\n"
