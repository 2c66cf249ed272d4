"""The 4-bit cache at the ends of its types' ranges (bounds: test_kv4.py)."""
import math

import numpy as np
import pytest
import torch

from exact_attention_blackwell_tma_gb300 import binding
from _plain import assert_within
from test_kv4 import Pool, bf16, check_appended, offsets


@pytest.mark.gpu
@pytest.mark.parametrize("step", [2.0 ** -133, 3 * 2.0 ** -133, 2.0 ** -131, 2.0 ** -128, 2.0 ** -126, 2.0 ** 100, 2.0 ** 120])
def test_append_codes_at_the_ends_of_the_range(step):
    """Groups whose scale is subnormal (its reciprocal infinite) or huge: codes as defined, exactly."""
    g = np.random.default_rng(31)
    unit = np.arange(64) % 16
    rows = [unit, 15 - unit, np.minimum(unit, 7), unit - 15] + [g.integers(-7, 9, 64) for _ in range(40)]
    x = torch.tensor(np.stack(rows) * step, dtype=torch.float32).to(torch.bfloat16)[:, None]
    assert torch.equal(x[:, 0].double(), torch.tensor(np.stack(rows) * step))   # all representable
    pool = Pool([len(rows)], 1, 64, seed=32)
    before = pool.host
    binding.kv4_append(pool.cache, x.cuda(), x.flip(0).contiguous().cuda(), pool.table, pool.lens_t,
                       cu_seqlens=offsets([len(rows)]).cuda())
    binding.check_status()
    check_appended(pool, [len(rows)], x, x.flip(0), before)


def check_values_of_size(size, d, n, lens, H):
    """O for values around `size`; the floor is what fp32 and bf16 resolve at the bottom of their range."""
    pool = Pool(lens, 1, d, seed=33)
    pool.host[3] = (pool.host[3].double() * size).to(torch.bfloat16)
    pool.upload()
    q = bf16(pool.g, sum(n), H, d)
    o, _ = binding.kv4_forward(q.cuda(), pool.cache, pool.table, pool.lens_t, scale=0.1, cu_seqlens=offsets(n).cuda())
    binding.check_status()
    o, at = o.double().cpu() / size, 0
    for b, rows in enumerate(n):
        k, (v, ac, spread) = pool.values(b, 0)[0], (x / size for x in pool.values(b, 1))
        s = torch.einsum("ihd,jhd->hij", q[at:at + rows].double(), k.expand(-1, H, -1)) * 0.1
        i, j = torch.arange(rows)[:, None], torch.arange(lens[b])[None]
        p = torch.softmax(s.masked_fill(j > i + lens[b] - rows, -math.inf), -1)
        ref, c, x = (torch.einsum("hij,jhd->ihd", p, y.expand(-1, H, -1)) for y in (v, ac, spread))
        # 2^-134: half a step of the smallest bf16; sums of 2^-149-sized fp32 roundings stay far below another
        assert_within(o[at:at + rows], ref, 2.0 ** -11 * c + 2.0 ** -13 * x + 2.0 ** -8 * ref.abs() + 2.0 ** -133 / size,
                      f"size {size} sequence {b}", floor=0.0)
        at += rows


@pytest.mark.gpu
@pytest.mark.parametrize("size", [2.0 ** -110, 2.0 ** -120, 2.0 ** -122, 2.0 ** -124, 2.0 ** -126, 2.0 ** -128])
@pytest.mark.parametrize("d", [64, 256])
def test_forward_tiny_values(size, d):
    """Value scales down to the subnormals keep the codes' share of O."""
    check_values_of_size(size, d, [1, 3], [700, 33], 2)


@pytest.mark.gpu
@pytest.mark.parametrize("size", [2.0 ** 90, 2.0 ** 106, 2.0 ** 112])
@pytest.mark.parametrize("d", [64, 256])
def test_forward_huge_values(size, d):
    """Value scales past 2^107, where 2^24 times the scale leaves the fp32 range."""
    check_values_of_size(size, d, [1, 3], [700, 33], 2)


@pytest.mark.gpu
def test_offsets_that_run_backwards_do_no_work():
    """Offsets 0, T, 0, T, .. pass every sequence's own check but give 512 sequences the same rows, whose work list
    (512 sequences x 16384 row blocks x 32768 units = 2^38) no int counts: reported, nothing written."""
    T, H, width = 4096, 64, 1 << 16
    pool = Pool([64], 1, 64, seed=34)
    table = torch.full((1023, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.full((1023,), width * 64, dtype=torch.int32, device="cuda")
    cu = torch.tensor([T * (i % 2) for i in range(1024)], dtype=torch.int32).cuda()
    q = torch.ones(T, H, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full((T, H, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, T), 7.0, device="cuda")
    binding.kv4_forward(q, pool.cache, table, lens, cu_seqlens=cu, out=out, lse=lse)
    with pytest.raises(binding.AttnError):
        binding.check_status()
    assert (out == 7).all() and (lse == 7).all()
    # the next call is not affected
    q = bf16(pool.g, 1, 2, 64)
    o, _ = binding.kv4_forward(q.cuda(), pool.cache, pool.table, pool.lens_t, cu_seqlens=offsets([1]).cuda())
    binding.check_status()
    assert torch.isfinite(o).all()


@pytest.mark.gpu
def test_refuses_a_workspace_that_is_not_on_the_device():
    pool = Pool([100], 1, 64, seed=35)
    q, cu = bf16(pool.g, 1, 2, 64).cuda(), offsets([1]).cuda()
    args = (q, pool.cache, pool.table, pool.lens_t)
    need = binding.attn_kv4_fwd_workspace_size(1, 2, 1, 1, 1, pool.width, 64, 64, 0)
    for bad in (torch.empty(need, dtype=torch.uint8), torch.empty(need, dtype=torch.uint8, pin_memory=True),
                torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            binding.kv4_forward(*args, cu_seqlens=cu, workspace=bad)
    o, lse = binding.kv4_forward(*args, cu_seqlens=cu)
    o2, lse2 = binding.kv4_forward(*args, cu_seqlens=cu, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    x = torch.ones(1, 9, 2, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = binding.forward(x, x, x, causal=True, window=(3, 0), sinks=1)
    with pytest.raises(ValueError):
        binding.backward(x, x, x, o, lse, x, causal=True, window=(3, 0), sinks=1,
                         workspace=torch.empty(1 << 20, dtype=torch.uint8))
    binding.check_status()


def test_workspace_check():
    with pytest.raises(ValueError):
        binding._check_workspace(torch.empty(8, dtype=torch.uint8), 0)


@pytest.mark.parametrize("d,dv", [(96, None), (100, 64), (128, 72), (32, 32)])
def test_empty_cache_refuses_head_dims(d, dv):
    with pytest.raises(ValueError, match="multiples of 64"):
        binding.Kv4Cache.empty(3, 1, d, dv, device="cpu")
