"""Windows with sinks in batches of very different sequences, and the workspace of the backward."""
import math

import pytest
import torch

from exact_attention_blackwell_tma_gb300 import binding, inputs
from _plain import gradients, visible


@pytest.mark.gpu
@pytest.mark.parametrize("d,dv", [(64, 64), (192, 128)])
def test_few_keys_beside_a_long_sequence(d, dv):
    """Sequences of two tokens keep the precision that test_rows_with_few_keys_keep_their_precision derives when a long
    sequence is packed with them: dS's rounding to bf16 and the output's, each below U / sqrt(3) rms (U = 2^-8)."""
    lens = [2] * 20 + [8000] + [2] * 20
    cu = inputs.cu_seqlens(lens)
    g = torch.Generator("cpu").manual_seed(185)
    r = lambda h, w: torch.randn(sum(lens), h, w, generator=g).to(torch.bfloat16)  # noqa: E731
    t = {"q": r(4, d), "k": r(2, d), "v": r(2, dv), "do": r(4, dv)}
    x = {n: y.cuda() for n, y in t.items()}
    scale = float(torch.tensor(1 / math.sqrt(d), dtype=torch.float32))
    kw = dict(causal=True, scale=scale, window=(50, 0), sinks=1, cu_seqlens=cu.cuda())
    o, lse = binding.forward(x["q"], x["k"], x["v"], **kw)
    grads = binding.backward(x["q"], x["k"], x["v"], o, lse, x["do"], **kw)
    binding.check_status()
    short = [slice(int(cu[b]), int(cu[b + 1])) for b in range(len(lens)) if lens[b] == 2]
    ok = visible(2, 2, True, (50, 0), 1)
    refs = [gradients(*(t[n][s].double() for n in ("q", "k", "v", "do")), ok, scale) for s in short]
    for n, got in zip(("dq", "dk"), grads):
        ref = torch.cat([y[n] for y in refs])
        got = torch.cat([got[s] for s in short]).double().cpu()
        rel = ((got - ref).norm() / ref.norm()).item()
        assert rel <= math.sqrt(2 / 3) * 2.0 ** -8, f"{n}: {rel:.2e}"


@pytest.fixture(scope="module")
def host_lib():
    from exact_attention_blackwell_tma_gb300 import build
    build.build()
    return binding.load()


@pytest.mark.parametrize("B,L,H,Hkv,d,dv,window,sinks", [(64, 2048, 32, 8, 128, 128, 512, 4), (16, 4096, 16, 16, 64, 64, 512, 4),
                                                        (1024, 30, 8, 2, 192, 128, 50, 1), (64, 2048, 32, 8, 128, 128, -1, 0),
                                                        (7, 333, 4, 4, 256, 256, 1000, 70)])
def test_packed_workspace_goes_by_the_rows(host_lib, B, L, H, Hkv, d, dv, window, sinks):
    """A packed batch of T rows needs the fp32 dQ of T rows, D, semaphores, the map and at most as much again in
    partials, not B times that; the call asks for exactly this."""
    T = B * L
    need = host_lib.attn_bwd_packed_workspace_size(B, H, Hkv, T, T, d, dv, 1, window, 0, sinks, 0)
    dq = 4 * T * H * d
    assert dq <= need <= 2 * dq + (64 << 20)
    x = 1 << 20   # never used: the workspace is refused first
    rc = host_lib.attn_bwd_sinks(*([x] * 9), B, H, Hkv, T, T, d, dv, 0.1, 1, window, 0, sinks, x, None, 0, x, need - 1, None)
    assert rc == binding.ATTN_ERR_WORKSPACE and f"{need} bytes needed" in binding.last_error()
    assert host_lib.attn_bwd_packed_workspace_size(B, 3, 2, T, T, d, dv, 1, window, 0, sinks, 0) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [((60, 0), 200), ((-1, -1), 0)])
@pytest.mark.parametrize("H,Hkv,d", [(4, 4, 64), (4, 2, 192)])
def test_packed_backward_stays_inside_its_workspace(H, Hkv, d, window, sinks):
    """With exactly the bytes asked for, whatever they hold, the gradients are the same and the bytes behind stay."""
    lens = [900, 1, 0, 300, 1500] + [40] * 30
    cu = inputs.cu_seqlens(lens)
    T = sum(lens)
    g = torch.Generator("cpu").manual_seed(186)
    q, k, v, do = (torch.randn(T, h, d, generator=g).to(torch.bfloat16).cuda() for h in (H, Hkv, Hkv, H))
    kw = dict(causal=True, window=window, sinks=sinks, cu_seqlens=cu.cuda())
    o, lse = binding.forward(q, k, v, **kw)
    ref = binding.backward(q, k, v, o, lse, do, deterministic=True, **kw)
    need = binding.attn_bwd_packed_workspace_size(len(lens), H, Hkv, T, T, d, d, 1, *window, sinks, 1)
    for fill in (0, 255):
        buf = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
        got = binding.backward(q, k, v, o, lse, do, deterministic=True, workspace=buf[:need], **kw)
        binding.check_status()
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
        assert (buf[need:] == fill).all()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("B,L,H,Hkv,d,window", [(1, 32768, 32, 32, 128, 128), (2, 8192, 16, 16, 128, 100), (8, 32768, 8, 8, 64, 128),
                                                (1, 5001, 8, 2, 192, 64), (1, 100000, 1, 1, 256, 10), (64, 2048, 32, 8, 128, 0)])
def test_sink_partials_are_bounded(host_lib, B, L, H, Hkv, d, window, packed):
    """However many keys are sinks, their partial dK and dV take at most 2 x 640 tiles of 128 rows (kernels.h)."""
    rows = B * L if packed else L
    size = host_lib.attn_bwd_packed_workspace_size if packed else host_lib.attn_bwd_sinks_workspace_size
    base = size(B, H, Hkv, rows, rows, d, d, 1, window, 0, 0, 0)
    for sinks in (1, 4, 129, 1000, 5000, L, 2 ** 31 - 1):
        more = size(B, H, Hkv, rows, rows, d, d, 1, window, 0, sinks, 0) - base
        assert 0 <= more <= 2 * 640 * 128 * 2 * d * 4 + 256, (sinks, more)
    if L // 128 > window // 128 + 2 and B * Hkv * H // Hkv < 320:   # few sinks of a long sequence: cut into parts
        assert size(B, H, Hkv, rows, rows, d, d, 1, window, 0, 4, 0) > base
