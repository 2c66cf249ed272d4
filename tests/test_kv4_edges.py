"""The 4-bit cache at the ends of its types' ranges (bounds: test_kv4.py)."""
import numpy as np
import pytest
import torch

from exact_attention_blackwell_tma_gb300 import binding
from test_kv4 import Pool, check_appended, offsets


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
