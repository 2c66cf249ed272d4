"""Windows with sinks in batches of very different sequences."""
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
