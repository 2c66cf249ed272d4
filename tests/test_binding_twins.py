"""The binding's C entry points under the same names, for sinks and the 4-bit cache: what they return and refuse,
and that a step made of them gives the bits of the tensor-level calls. Bounds may be any integers."""
import numpy as np
import pytest
import torch

from exact_attention_blackwell_tma_gb300 import binding, inputs
from test_kv4 import Pool, bf16, offsets

X = 1 << 20   # an address that is never used: the checks come first


def test_twins_return_the_codes():
    from exact_attention_blackwell_tma_gb300 import build
    build.build()
    bad, arg = binding._Kv4Struct(X, X, X, X, 4, 2, 96, 96), binding.ATTN_ERR_ARG
    assert binding.attn_kv4_append(X, X, 512, 512, bad, X, 3, X, None, 1, 1, stream=0) == arg
    assert binding.attn_kv4_read(X, X, bad, X, 3, X, None, 1, 1, stream=0) == arg
    assert binding.attn_kv4_fwd(X, 1024, bad, X, 3, X, None, X, X, 1, 4, 1, 0.1, True, -1, -1, 0, None, 0, 1.0, X, 1 << 40,
                                stream=0) == arg
    assert binding.attn_kv4_evict(bad, X, 3, X, X, 192, X + 64, 1, 1, 10, 0, 0, X + 128, X, X + 64, 10, stream=0) == arg
    assert binding.attn_fwd_sinks(X, X, X, X, X, 1, 2, 1, 64, 64, 64, 64, 0.1, True, 5, -1, -1, stream=0) == arg
    assert binding.attn_bwd_sinks(*([X] * 9), 1, 2, 1, 64, 64, 64, 64, 0.1, True, 5, -1, -1, None, None, False, X, 1 << 40,
                                  stream=0) == arg
    assert "sinks" in binding.last_error()
    good = binding._Kv4Struct(X, X, X, X, 4, 2, 64, 64)
    assert binding.attn_kv4_append(X, X, 128, 128, good, X, 3, X, None, 0, 1, stream=0) == binding.ATTN_OK


@pytest.mark.gpu
def test_a_cache_step_of_twins():
    lens, new, H, Hkv, d = [300, 90], [2, 1], 4, 2, 64
    pools = [Pool(lens, Hkv, d, seed=41, extra=4) for _ in range(2)]
    g = np.random.default_rng(42)
    q, k, v, cu = bf16(g, 3, H, d).cuda(), bf16(g, 3, Hkv, d).cuda(), bf16(g, 3, Hkv, d).cuda(), offsets(new).cuda()
    width = pools[0].width
    new_table = torch.tensor(pools[0].spare[:4].reshape(2, 2).astype(np.int32)).cuda()
    w = [torch.zeros(2, Hkv, width * 64, device="cuda") for _ in range(2)]
    a, b = pools
    binding.kv4_append(a.cache, k, v, a.table, a.lens_t, cu_seqlens=cu)
    o, lse = binding.kv4_forward(q, a.cache, a.table, a.lens_t, cu_seqlens=cu, window=(80, -1), sinks=3, key_weights=w[0])
    kept = binding.kv4_evict(a.cache, a.table, a.lens_t, w[0], new_table, 100, 4, 20)
    rk, rv = binding.kv4_read(a.cache, new_table, kept[0], 190, cu_seqlens=offsets([100, 90]).cuda())
    c = b.cache._struct
    assert binding.attn_kv4_append(k, v, Hkv * d, Hkv * d, c, b.table, width, b.lens_t, cu, 2, 3) == 0
    need = binding.attn_kv4_fwd_workspace_size(2, H, Hkv, 3, True, width, d, d, True)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    assert binding.attn_kv4_fwd(q, H * d, c, b.table, width, b.lens_t, cu, o2, lse2, 2, H, 3, 1 / 8, True, 80, -1, 3, w[1],
                                width * 64, 1.0, ws, need) == 0
    got = [torch.empty_like(x) for x in kept]
    assert binding.attn_kv4_evict(c, b.table, width, b.lens_t, w[1], width * 64, new_table, 2, 2, 100, 4, 20, got[0], got[1],
                                  got[2], 100) == 0
    k2, v2 = torch.empty_like(rk), torch.empty_like(rv)
    assert binding.attn_kv4_read(k2, v2, c, new_table, 2, got[0], offsets([100, 90]).cuda(), 2, 190) == 0
    binding.check_status()
    pairs = [(o, o2), (lse, lse2), (w[0], w[1]), (rk, k2), (rv, v2), *zip(kept, got)]
    assert all(torch.equal(x, y) for x, y in pairs) and (o != 0).any()


@pytest.mark.gpu
def test_sinks_of_twins_and_other_integers():
    t = {n: x.cuda() for n, x in inputs.small(B=1, H=4, L=400, d=64, seed=192, Hkv=2).items()}
    q, k, v, do = (t[n] for n in ("q", "k", "v", "do"))
    o, lse = binding.forward(q, k, v, causal=True, window=(60, 0), sinks=5, scale=0.125)
    grads = binding.backward(q, k, v, o, lse, do, causal=True, window=(60, 0), sinks=5, scale=0.125, deterministic=True)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    assert binding.attn_fwd_sinks(q, k, v, o2, lse2, 1, 4, 2, 400, 400, 64, 64, 0.125, True, 60, 0, 5) == 0
    need = binding.attn_bwd_sinks_workspace_size(1, 4, 2, 400, 400, 64, 64, True, 60, 0, 5, True)
    ws, got = torch.empty(need, dtype=torch.uint8, device="cuda"), [torch.empty_like(x) for x in grads]
    assert binding.attn_bwd_sinks(q, k, v, o2, lse2, do, *got, 1, 4, 2, 400, 400, 64, 64, 0.125, True, 60, 0, 5, None, None,
                                  True, ws, need) == 0
    numpy = dict(causal=True, window=np.array([60, 0]), sinks=np.int32(5), scale=0.125)
    o3, lse3 = binding.forward(q, k, v, **numpy)
    other = binding.backward(q, k, v, o3, lse3, do, deterministic=True, **numpy)
    binding.check_status()
    for x in ((o2, lse2, *got), (o3, lse3, *other)):
        assert all(torch.equal(a, b) for a, b in zip((o, lse, *grads), x))
    pool = Pool([200], 2, 64, seed=43)
    args, cu = (pool.cache, pool.table, pool.lens_t), offsets([1]).cuda()
    a = binding.kv4_forward(q[0, :1], *args, cu_seqlens=cu, window=(50, -1), sinks=4)
    b = binding.kv4_forward(q[0, :1], *args, cu_seqlens=cu, window=np.array([50, -1]), sinks=np.int64(4))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 31 - 1, 10 ** 20])
def test_integers_that_do_not_fit_are_refused(big):
    """Their low 32 bits would be another bound (2^32 sinks: none)."""
    x = torch.ones(1, 200, 2, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = binding.forward(x, x, x, causal=True, window=(5, 0), sinks=2)
    pool = Pool([200], 2, 64, seed=44)
    args, cu = (pool.cache, pool.table, pool.lens_t), offsets([1]).cuda()
    w = torch.zeros(1, 2, 256, device="cuda")
    for window, sinks in (((5, 0), big), ((big, 0), 2), ((5, big), 2)):
        with pytest.raises(ValueError, match="fit"):
            binding.forward(x, x, x, causal=True, window=window, sinks=sinks)
        with pytest.raises(ValueError, match="fit"):
            binding.backward(x, x, x, o, lse, x, causal=True, window=window, sinks=sinks)
        with pytest.raises(ValueError, match="fit"):
            binding.kv4_forward(x[0, :1], *args, cu_seqlens=cu, window=window, sinks=sinks)
    for kw in (dict(budget=big), dict(budget=64, sinks=big), dict(budget=64, recent=big)):
        with pytest.raises(ValueError, match="fit"):
            binding.kv4_evict(*args, w, pool.table, **kw)
    binding.check_status()
