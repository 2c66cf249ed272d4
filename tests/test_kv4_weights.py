"""Key weights that several calls accumulate, with decay, and the budget that they leave (bounds: test_kv4.py)."""
import math

import numpy as np
import pytest
import torch

from exact_attention_blackwell_tma_gb300 import binding
from test_kv4 import Pool, bf16, offsets, plain_evict


def weights_of(pool, b, q, scale):
    """float64 [Hkv, keys]: the attention weight that sequence b's keys get from rows q [n, H, d] (its last tokens)."""
    k = pool.values(b, 0)[0]
    n, H, N = q.shape[0], q.shape[1], k.shape[0]
    s = torch.einsum("ihd,jhd->hij", q.double(), k.repeat_interleave(H // pool.Hkv, 1)) * scale
    s = s.masked_fill(torch.arange(N) > torch.arange(n)[:, None] + N - n, -math.inf)
    return torch.softmax(s, -1).reshape(pool.Hkv, -1, N).sum(1)


@pytest.mark.gpu
@pytest.mark.parametrize("decay", [0.9, 0.5, 1.0])
@pytest.mark.parametrize("H,Hkv,d", [(8, 2, 64), (4, 4, 128)])
def test_decay_over_several_calls(H, Hkv, d, decay):
    """Five steps that append and attend, each decaying what the ones before left; every addition is within 2^-13 of
    itself and every decayed term within another 2^-23, so the sum within 2^-13 + 5 x 2^-23 of itself: 2^-12."""
    start, steps = [150, 63, 700], [[1, 1, 1], [3, 2, 1], [1, 0, 5], [1, 1, 1], [8, 1, 2]]
    pool = Pool([n + 20 for n in start], Hkv, d, seed=51)
    pool.lens = list(start)
    w = torch.zeros((3, Hkv, pool.width * 64), device="cuda")
    want = [torch.zeros(Hkv, n + 20, dtype=torch.float64) for n in start]
    scale = 1 / math.sqrt(d)
    for new in steps:
        pool.lens = [a + b for a, b in zip(pool.lens, new)]
        lens, cu = torch.tensor(pool.lens, dtype=torch.int32).cuda(), offsets(new).cuda()
        k, v, q = (bf16(pool.g, sum(new), h, d) for h in (Hkv, Hkv, H))
        binding.kv4_append(pool.cache, k.cuda(), v.cuda(), pool.table, lens, cu_seqlens=cu)
        binding.kv4_forward(q.cuda(), pool.cache, pool.table, lens, scale=scale, cu_seqlens=cu, key_weights=w,
                            weight_decay=decay)
        pool.download()
        at = 0
        for b, n in enumerate(new):
            N = pool.lens[b]
            want[b][:, :N] *= decay
            if n:
                want[b][:, :N] += weights_of(pool, b, q[at:at + n], scale)
            at += n
    binding.check_status()
    for b, n in enumerate(pool.lens):
        got = w[b, :, :n].double().cpu()
        assert ((got - want[b][:, :n]).abs() <= 2.0 ** -12 * want[b][:, :n] + 1e-12).all(), b
        assert (w[b, :, n:] == 0).all()


@pytest.mark.gpu
def test_budget_kept_over_decaying_steps():
    """Decode, evict, decode, evict: the second eviction goes by the weights that the first one kept, decayed and
    added to, in the kept order."""
    H, Hkv, d, budget, decay = 4, 2, 64, 100, 0.75
    pool = Pool([230, 140], Hkv, d, seed=52, extra=20)
    pages = [torch.tensor(pool.spare[i:i + 4].reshape(2, 2).astype(np.int32)).cuda() for i in (0, 4)]
    tables, lens = (pool.table, *pages), pool.lens_t
    w = torch.zeros((2, Hkv, pool.width * 64), device="cuda")
    cu = offsets([1, 1]).cuda()
    for step in range(2):
        table = tables[step]
        q = bf16(pool.g, 2, H, d).cuda()
        before = w.clone()
        binding.kv4_forward(q, pool.cache, table, lens, cu_seqlens=cu, key_weights=w, weight_decay=decay)
        alone = torch.zeros_like(w)
        binding.kv4_forward(q, pool.cache, table, lens, cu_seqlens=cu, key_weights=alone)
        assert torch.allclose(w, decay * before + alone, rtol=2.0 ** -22, atol=0)   # two roundings of fp32
        size = budget - 30 * step
        new_w = torch.zeros((2, Hkv, 128), device="cuda")
        new_lens, kept, _ = binding.kv4_evict(pool.cache, table, lens, w, tables[step + 1], budget=size, sinks=2, recent=10,
                                              new_key_weights=new_w)
        for b, n in enumerate(lens.tolist()):
            for h in range(Hkv):
                want = plain_evict(w[b, h].cpu().numpy(), n, size, 2, 10)
                assert kept[b, h].tolist() == want and torch.equal(new_w[b, h, :size], w[b, h, want])
        w, lens = new_w, new_lens
    binding.check_status()
