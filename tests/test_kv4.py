"""The 4-bit key/value cache (append, read, attention, eviction) against float64.

Bounds. Codes and kept slots are compared exactly. Attention: p a' is rounded to
fp16 (half a step: 2^-11) before it multiplies a code, the output to bf16 (2^-8);
scores, statistics and sums are fp32, which for scores below about 100 moves p by
less than 2^-14 of itself; so |O - ref| <= 2^-11 sum p a' c + 2^-13 sum p (15 a' +
|b'|) + 2^-8 |ref|, and a key weight is off by at most 2^-13 of itself.
"""
import math

import numpy as np
import pytest
import torch

from exact_attention_blackwell_tma_gb300 import binding
from _plain import assert_lse, assert_within, visible

PAGE, GROUP = binding.KV4_PAGE, binding.KV4_GROUP


def codes_and_params(x):
    """The definition in float64: x [..., 64] -> codes, scale, minimum."""
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    with np.errstate(over="ignore"):
        scale = torch.tensor((hi - lo) / 15.0).to(torch.bfloat16).double().numpy()
    q = np.divide(x - lo, scale, out=np.zeros_like(x), where=scale > 0)
    return np.clip(np.rint(q), 0, 15).astype(np.uint8), scale[..., 0], lo[..., 0]


class Pool:
    """A cache with pages handed out in a shuffled order, random contents, on the GPU."""

    def __init__(self, lens, Hkv, d, dv=None, seed=0, extra=0, width=None):
        self.Hkv, self.d, self.dv, self.lens = Hkv, d, d if dv is None else dv, list(lens)
        g = np.random.default_rng(seed)
        need = [-(-n // PAGE) for n in lens]
        total = max(1, sum(need) + extra)
        self.g, self.total = g, total
        ids = g.permutation(total)
        self.width = max([1] + need) if width is None else width
        table = np.full((len(lens), self.width), -7, np.int32)   # entries past a sequence's pages are never read
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
        self.spare = ids[at:]
        self.table_host = table
        self.table, self.lens_t = torch.tensor(table).cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda()
        parts = []
        for w in (self.d, self.dv):
            codes = torch.tensor(g.integers(0, 256, (total, Hkv, w // GROUP, PAGE, GROUP // 2), dtype=np.uint8))
            scale = 0.3 * np.exp(0.3 * g.standard_normal((total, Hkv, w // GROUP, PAGE)))
            low = -7.5 * scale + 0.3 * g.standard_normal(scale.shape)
            parts += [codes, torch.tensor(np.stack((scale, low), -1)).to(torch.bfloat16)]
        self.host = parts
        self.upload()

    def upload(self):
        self.cache = binding.Kv4Cache(*(x.cuda() for x in self.host))

    def download(self):
        c = self.cache
        self.host = [x.cpu() for x in (c.k_codes, c.k_params, c.v_codes, c.v_params)]

    def values(self, b, which, table=None, n=None):
        """Sequence b's keys (which = 0) or values (1) in float64: value, scale * code and 15 |scale| + |minimum|,
        each [tokens, Hkv, width]."""
        codes, params = self.host[2 * which], self.host[2 * which + 1].double()
        n = self.lens[b] if n is None else n
        j = np.arange(n)
        page = (self.table_host if table is None else table)[b][j // PAGE].astype(np.int64)
        c, p = codes[page, :, :, j % PAGE], params[page, :, :, j % PAGE]
        c = torch.stack((c & 15, c >> 4), -1).flatten(-2).double()
        s, m = p[..., :1], p[..., 1:]
        return tuple(x.flatten(2) for x in (s * c + m, (s * c).abs(), (15 * s.abs() + m.abs()).expand_as(c)))


def offsets(ns):
    return torch.tensor([0] + list(np.cumsum(ns)), dtype=torch.int32)


def bf16(g, *shape):
    return torch.tensor(g.standard_normal(shape), dtype=torch.float32).to(torch.bfloat16)


# ------------------------------------------------------------------ append and read

def check_appended(pool, new, k, v, before):
    """The new rows' codes and parameters follow the definition; every other token of the pool is as before."""
    pool.download()
    at, touched = 0, [x.clone() for x in before]
    for b, n in enumerate(new):
        for which, x in enumerate((k, v)):
            rows = x[at:at + n].double().numpy().reshape(n, pool.Hkv, x.shape[-1] // GROUP, GROUP)
            c, s, m = codes_and_params(rows)
            j = np.arange(pool.lens[b] - n, pool.lens[b])
            page = pool.table_host[b][j // PAGE].astype(np.int64)
            touched[2 * which][page, :, :, j % PAGE] = torch.tensor(c[..., 0::2] | c[..., 1::2] << 4)
            touched[2 * which + 1][page, :, :, j % PAGE] = torch.tensor(np.stack((s, m), -1)).to(torch.bfloat16)
        at += n
    for name, got, want in zip(("k codes", "k params", "v codes", "v params"), pool.host, touched):
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8)), name


@pytest.mark.gpu
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (192, 128), (256, 256)])
@pytest.mark.parametrize("new,lens", [([1], [1]), ([1, 1, 1], [64, 65, 500]), ([130, 0, 64, 3], [130, 77, 200, 66]),
                                      ([5, 700], [5, 701])])
def test_append_packed(d, dv, new, lens):
    pool = Pool(lens, 2, d, dv, seed=1, extra=2)
    before = pool.host
    k, v = bf16(pool.g, sum(new), 2, d), bf16(pool.g, sum(new), 2, dv)
    binding.kv4_append(pool.cache, k.cuda(), v.cuda(), pool.table, pool.lens_t, cu_seqlens=offsets(new).cuda())
    binding.check_status()
    check_appended(pool, new, k, v, before)
    rk, rv = binding.kv4_read(pool.cache, pool.table, pool.lens_t, sum(new), cu_seqlens=offsets(new).cuda())
    at = 0
    for b, n in enumerate(new):
        for which, got in enumerate((rk, rv)):
            want = pool.values(b, which)[0][lens[b] - n:]
            # fp32 rounding, then bf16
            assert_within(got[at:at + n], want, 2.0 ** -8 * want.abs() + 2.0 ** -22 * pool.values(b, which)[2][lens[b] - n:],
                          f"read {which}")
        at += n


@pytest.mark.gpu
def test_append_hard_values():
    """Ties, borders, constant groups, outliers, mixed exponents, the smallest and largest values."""
    g = np.random.default_rng(2)
    rows = []
    grid = np.arange(64, dtype=np.float64)
    rows += [np.zeros(64), np.full(64, -3.25), grid % 31 * 0.5, (grid % 31) * 0.5 - 7, grid, -grid, grid * 2.0 ** -130,
             np.where(grid == 5, 1e30, grid), np.where(grid == 5, 2.0 ** -60, grid % 8 + 100)]
    rows += [np.round(g.standard_normal(64) * 8) / 8 for _ in range(60)]
    rows += [g.standard_normal(64) * np.exp(4 * g.standard_normal(64)) for _ in range(60)]
    rows += [g.integers(-15, 16, 64) * 0.25 for _ in range(60)]
    rows += [g.standard_normal(64) * 2.0 ** g.integers(-60, 60) for _ in range(60)]
    x = torch.tensor(np.stack(rows), dtype=torch.float32).to(torch.bfloat16)[:, None]
    pool = Pool([len(rows)], 1, 64, seed=3)
    before = pool.host
    binding.kv4_append(pool.cache, x.cuda(), x.flip(0).contiguous().cuda(), pool.table, pool.lens_t,
                       cu_seqlens=offsets([len(rows)]).cuda())
    binding.check_status()
    check_appended(pool, [len(rows)], x, x.flip(0), before)


@pytest.mark.gpu
def test_append_dense_strided_and_neighbours():
    """Rows of a fused projection (strided views), a dense batch; infinities and NaN stay in their group."""
    B, L, Hkv, d = 3, 70, 2, 128
    pool = Pool([70, 170, 99], Hkv, d, seed=4)
    fused = bf16(pool.g, B, L, 2 * Hkv + 4, d)
    fused[1, 3, 4, 70] = math.inf
    fused[2, 5, 7, 1] = math.nan
    gpu = fused.cuda()
    k, v = gpu[:, :, 4:6], gpu[:, :, 6:8]
    binding.kv4_append(pool.cache, k, v, pool.table, pool.lens_t)
    binding.check_status()
    rk, rv = binding.kv4_read(pool.cache, pool.table, pool.lens_t, L)
    assert rk.shape == (B, L, Hkv, d)
    for got, x, bad in ((rk, k, (1, 3, 0, 1)), (rv, v, (2, 5, 1, 0))):
        got = got.reshape(B, L, Hkv, 2, GROUP).float().cpu()
        x = x.reshape(B, L, Hkv, 2, GROUP).float().cpu()
        assert torch.isnan(got[bad]).all()
        ok = torch.ones(B, L, Hkv, 2, dtype=torch.bool)
        ok[bad] = False
        step = (x.amax(-1) - x.amin(-1))[..., None] / 15
        # half a step, a scale off by 2^-8 over 15 steps, bf16 rounding of the value
        bound = step * (0.5 + 15 * 2.0 ** -8) + x.abs() * 2.0 ** -8
        assert ((got - x).abs()[ok] <= bound[ok]).all()


@pytest.mark.gpu
def test_read_padded_batch_and_rows_behind_the_last():
    pool = Pool([3, 0, 100], 1, 64, seed=5)
    k, v = binding.kv4_read(pool.cache, pool.table, pool.lens_t, 5)
    assert (k[0, :2] == 0).all() and (k[1] == 0).all() and (k[0, 2:] != 0).any()
    want = pool.values(2, 1)[0][95:]
    assert_within(v[2], want, 2.0 ** -8 * want.abs() + 1e-6, "last rows")
    out = torch.full((9, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out2 = out.clone()
    binding.kv4_read(pool.cache, pool.table, pool.lens_t, 9, cu_seqlens=offsets([2, 0, 4]).cuda(), k=out, v=out2)
    binding.check_status()
    assert (out[6:] == 7).all() and (out2[6:] == 7).all() and (out[:6] != 7).any()
    before = pool.host
    x = bf16(pool.g, 9, 1, 64)
    binding.kv4_append(pool.cache, x.cuda(), x.cuda(), pool.table, pool.lens_t, cu_seqlens=offsets([2, 0, 4]).cuda())
    binding.check_status()
    check_appended(pool, [2, 0, 4], x, x, before)


# ------------------------------------------------------------------ attention

def check_forward(pool, new, H, causal=True, window=(-1, -1), sinks=0, decay=None, q=None, packed=True, scale=None,
                  what=""):
    T = sum(new)
    q = bf16(pool.g, T, H, pool.d) if q is None else q
    scale = 1 / math.sqrt(pool.d) if scale is None else scale
    old = None
    if decay is not None:
        old = torch.tensor(pool.g.random((len(new), pool.Hkv, pool.width * PAGE)), dtype=torch.float32)
    w = None if old is None else old.clone().cuda()
    cu = offsets(new).cuda() if packed else None
    gq = q.cuda() if packed else q.reshape(len(new), -1, H, pool.d).cuda()
    o, lse = binding.kv4_forward(gq, pool.cache, pool.table, pool.lens_t, causal=causal, scale=scale, cu_seqlens=cu,
                                 window=window, sinks=sinks, key_weights=w, weight_decay=0.0 if decay is None else decay)
    binding.check_status()
    o2 = o.reshape(T, H, pool.dv)
    lse2 = lse if packed else lse.transpose(0, 1).reshape(H, T)
    r, at = H // pool.Hkv, 0
    for b, n in enumerate(new):
        k, (v, ac, spread) = pool.values(b, 0)[0], pool.values(b, 1)
        N = pool.lens[b]
        ok = visible(n, N, causal, window, sinks)
        kx, vx, acx, sx = (x.repeat_interleave(r, 1).nan_to_num(0.0, 0.0, 0.0) for x in (k, v, ac, spread))
        s = torch.einsum("ihd,jhd->hij", q[at:at + n].double(), kx) * scale
        s = s.masked_fill(~ok, -math.inf)
        ref_lse = torch.logsumexp(s, -1) if N else torch.full((H, n), -math.inf, dtype=torch.float64)
        p = torch.where(ok, torch.exp(s - torch.where(torch.isfinite(ref_lse), ref_lse, 0.0)[..., None]), 0.0)
        ref = torch.einsum("hij,jhd->ihd", p, vx)
        bound = (2.0 ** -11 * torch.einsum("hij,jhd->ihd", p, acx) + 2.0 ** -13 * torch.einsum("hij,jhd->ihd", p, sx)
                 + 2.0 ** -8 * ref.abs())
        assert_within(o2[at:at + n], ref, bound, f"{what} sequence {b} O")
        assert_lse(lse2[:, at:at + n], ref_lse, f"{what} sequence {b}", scores=100.0)
        if old is not None:
            got = w[b].double().cpu()
            want = p.reshape(pool.Hkv, r * n, N).sum(1) if n else torch.zeros(pool.Hkv, N, dtype=torch.float64)
            want = want + decay * old[b, :, :N].double()
            assert_within(got[:, :N], want, 2.0 ** -13 * want, f"{what} sequence {b} weights", floor=1e-12)
            assert torch.equal(w[b, :, N:].cpu(), old[b, :, N:]), "weights past the cache"
        at += n
    return o, lse, w


DIMS = [(64, 64), (128, 128), (192, 192), (192, 128), (256, 256)]


@pytest.mark.gpu
@pytest.mark.parametrize("d,dv", DIMS)
@pytest.mark.parametrize("H,Hkv", [(1, 1), (2, 2), (8, 2), (6, 2), (16, 1), (12, 1)])
def test_forward_one_token(d, dv, H, Hkv):
    lens = [1, 63, 64, 65, 200, 1000]
    check_forward(Pool(lens, Hkv, d, dv, seed=6), [1] * len(lens), H, decay=0.0, what=f"d={d}/{dv} H={H}/{Hkv}")


@pytest.mark.gpu
@pytest.mark.parametrize("d,dv", DIMS)
@pytest.mark.parametrize("window,sinks", [((-1, -1), 0), ((0, -1), 0), ((10, -1), 4), ((64, -1), 64), ((100, -1), 70),
                                          ((300, -1), 1), ((2 ** 31 - 1, -1), 2 ** 31 - 1)])
def test_forward_window_and_sinks(d, dv, window, sinks):
    """1 to 16 tokens, empty sequences, a cache shorter than its rows."""
    lens, new = [700, 64, 5, 0, 333, 129, 3], [16, 3, 5, 0, 0, 1, 2]
    check_forward(Pool(lens, 2, d, dv, seed=7), new, 6, window=window, sinks=sinks, decay=1.0,
                  what=f"d={d} window={window} sinks={sinks}")


@pytest.mark.gpu
@pytest.mark.parametrize("causal,window", [(False, (-1, -1)), (False, (30, 20)), (False, (-1, 5)), (True, (7, 9))])
def test_forward_other_masks(causal, window):
    lens, new = [400, 90, 130], [9, 2, 70]
    check_forward(Pool(lens, 1, 64, seed=8), new, 3, causal=causal, window=window, sinks=3, decay=0.5,
                  what=f"causal={causal} window={window}")


@pytest.mark.gpu
def test_forward_rows_without_keys():
    """More rows than cached tokens: the first rows see nothing (O = 0, LSE = -inf); so does an empty cache."""
    o, lse, _ = check_forward(Pool([4, 0, 70], 1, 128, seed=9), [9, 3, 2], 2, decay=0.0)
    assert (o[:5] == 0).all() and torch.isneginf(lse[:, :5]).all() and (o[9:12] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d,n,H,Hkv", [(64, 40, 8, 1), (128, 33, 4, 2), (256, 20, 2, 1), (128, 200, 2, 2)])
def test_forward_many_rows(d, n, H, Hkv):
    """Several row blocks per head."""
    check_forward(Pool([300, n, 2000], Hkv, d, seed=10), [n, n, n], H, decay=0.0, what=f"{n} rows")


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [((-1, -1), 0), ((300, -1), 4)])
def test_key_weights_of_many_caches(window, sinks):
    """Enough (sequence, head) pairs that a block takes four tiles of keys: their borders, and none at all."""
    lens = [2100, 513, 0, 512, 1537, 2048, 2049] + [3 + i % 90 for i in range(133)]
    new = [3, 1, 0, 2, 5, 1, 1] + [1] * 133
    check_forward(Pool(lens, 8, 64, seed=23), new, 16, decay=0.5, window=window, sinks=sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("L", [1, 4])
def test_forward_dense_batch(L):
    check_forward(Pool([100, 250, 64, 4], 2, 128, seed=11), [L] * 4, 8, packed=False, decay=0.0)


@pytest.mark.gpu
def test_forward_long_and_ragged():
    """One long cache shared by many CTAs beside short ones."""
    check_forward(Pool([40000, 17, 3000, 9000], 1, 128, seed=12), [1, 2, 1, 4], 4, decay=0.0)


@pytest.mark.gpu
def test_forward_strided_queries():
    pool = Pool([300, 200], 2, 64, seed=13)
    fused = bf16(pool.g, 5, 12, 64).cuda()
    cu = offsets([2, 3]).cuda()
    a = binding.kv4_forward(fused[:, :8], pool.cache, pool.table, pool.lens_t, cu_seqlens=cu)
    b = binding.kv4_forward(fused[:, :8].contiguous(), pool.cache, pool.table, pool.lens_t, cu_seqlens=cu)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [((-1, -1), 0), ((50, -1), 4)])
def test_forward_ignores_what_it_masks(window, sinks):
    """NaN and infinities in unwritten slots of the last page and in keys left of the window change nothing."""
    lens = [130, 200, 77]
    pool = Pool(lens, 2, 128, seed=14)
    for b, n in enumerate(lens):
        dead = list(range(n, -(-n // PAGE) * PAGE))
        if window[0] >= 0:
            dead += list(range(sinks, n - 1 - window[0] - 1))   # two rows: the first one's window reaches furthest
        j = np.array(dead)
        page = pool.table_host[b][j // PAGE].astype(np.int64)
        for part in (1, 3):
            pool.host[part][page, :, :, j % PAGE] = torch.tensor([math.nan, math.inf], dtype=torch.bfloat16)
        pool.host[3][page[::2], :, :, j[::2] % PAGE, 0] = math.inf
    pool.upload()
    check_forward(pool, [2, 2, 2], 4, window=window, sinks=sinks, decay=0.0)


@pytest.mark.gpu
def test_forward_masks_per_row():
    """A value that is infinite in a key only the last row sees leaves the rows before it alone."""
    pool = Pool([100], 1, 64, seed=15)
    page = int(pool.table_host[0][99 // PAGE])
    pool.host[3][page, 0, 0, 99 % PAGE, 0] = math.inf
    pool.upload()
    q = bf16(pool.g, 3, 2, 64).cuda()
    o, lse = binding.kv4_forward(q, pool.cache, pool.table, pool.lens_t, cu_seqlens=offsets([3]).cuda())
    assert torch.isfinite(o[:2]).all() and not torch.isfinite(o[2]).all() and torch.isfinite(lse).all()


@pytest.mark.gpu
@pytest.mark.parametrize("size", [2.0 ** -40, 2.0 ** -14, 1.0, 2.0 ** 14, 2.0 ** 40])
def test_forward_value_sizes(size):
    """V of any size, growing and shrinking along the cache by 2^12: p a' keeps its precision."""
    pool = Pool([700], 1, 128, seed=16)
    ramp = torch.tensor(2.0 ** pool.g.uniform(-6, 6, pool.host[3].shape[:-1]))[..., None]
    pool.host[3] = (pool.host[3].double() * ramp * size).to(torch.bfloat16)
    pool.upload()
    check_forward(pool, [2], 4, what=f"size {size}")


@pytest.mark.gpu
@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** -8, 2.0 ** 8])
def test_forward_query_sizes(size):
    """Rows of very different size in one block; the scale undoes the size."""
    pool = Pool([300], 1, 64, seed=17)
    q = (bf16(pool.g, 4, 3, 64).float() * size * 2.0 ** torch.arange(-4, 8).reshape(4, 3, 1)).to(torch.bfloat16)
    check_forward(pool, [4], 3, q=q, scale=min(2.0 ** -9 / size, 2.0 ** 30), what=f"queries {size}")


@pytest.mark.gpu
@pytest.mark.parametrize("junk", [3e38, 1e10, math.inf, math.nan, 0.0])
def test_forward_unused_rows_hold_anything(junk):
    """A padded dense batch: rows before a short sequence's tokens see no key, and neither they nor a neighbour's
    bad row reach the rows beside them."""
    pool = Pool([2, 100], 2, 128, seed=28)
    q = bf16(pool.g, 2, 4, 4, 128)
    q[0, :2] = junk   # sequence 0 has two tokens, its first two rows are padding
    q[1, 1, 2] = junk
    o, lse = binding.kv4_forward(q.cuda(), pool.cache, pool.table, pool.lens_t)
    assert (o[0, :2] == 0).all() and torch.isneginf(lse[0, :, :2]).all()
    clean = q.clone()
    clean[0, :2] = 1
    clean[1, 1, 2] = 1
    o2, lse2 = binding.kv4_forward(clean.cuda(), pool.cache, pool.table, pool.lens_t)
    keep = torch.ones(2, 4, 4, dtype=torch.bool)
    keep[1, 1, 2] = False
    assert torch.equal(o.cpu()[keep], o2.cpu()[keep]) and torch.equal(lse.cpu().transpose(1, 2)[keep], lse2.cpu().transpose(1, 2)[keep])
    binding.check_status()


@pytest.mark.gpu
def test_forward_a_maximum_that_climbs():
    """Scores that grow along the cache move the running maximum again and again."""
    pool = Pool([2000], 1, 64, seed=18)
    j = np.arange(2000)
    page = pool.table_host[0][j // PAGE].astype(np.int64)
    pool.host[1][page, 0, 0, j % PAGE, 1] = torch.tensor(j * 0.01).to(torch.bfloat16)
    pool.upload()
    q = bf16(pool.g, 1, 2, 64).abs()
    check_forward(pool, [1], 2, q=q, scale=0.1, decay=0.0)


@pytest.mark.gpu
def test_forward_shared_pages_and_repeats():
    """Two sequences with a common prefix of pages; the same call twice gives the same bits."""
    pool = Pool([500, 500], 2, 128, seed=19)
    pool.table_host[1, :5] = pool.table_host[0, :5]
    pool.table = torch.tensor(pool.table_host).cuda()
    q = bf16(pool.g, 4, 8, 128)
    a = check_forward(pool, [2, 2], 8, q=q, decay=0.0)
    b = check_forward(pool, [2, 2], 8, q=q, decay=0.0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(a[2][..., :500], b[2][..., :500])   # (past the cache: what each call found there)


@pytest.mark.gpu
def test_forward_largest_batch():
    lens = [(37 * i) % 150 for i in range(1024)]
    check_forward(Pool(lens, 1, 64, seed=20), [min(1, n) for n in lens], 2)


@pytest.mark.gpu
def test_forward_captured_and_on_other_streams():
    """A captured call replays on new contents; calls on two streams at once have workspaces of their own."""
    pool = Pool([3000, 70], 2, 128, seed=21)
    q = bf16(pool.g, 2, 8, 128).cuda()
    cu = offsets([1, 1]).cuda()
    args = (pool.cache, pool.table, pool.lens_t)
    want, lse = binding.kv4_forward(q, *args, cu_seqlens=cu)
    graph = torch.cuda.CUDAGraph()
    static = torch.zeros_like(q)
    with torch.cuda.graph(graph):
        o, l2 = binding.kv4_forward(static, *args, cu_seqlens=cu)
    static.copy_(q)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(l2, lse)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[binding.kv4_forward(q, *args, cu_seqlens=cu, stream=s)[0] for s in streams] for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for pair in outs for x in pair)


@pytest.mark.gpu
def test_bad_pages_and_lengths_are_reported():
    """The kernels check every page id and length; keys of a bad page do not count."""
    pool = Pool([200, 100], 1, 64, seed=22)
    good = pool.table_host.copy()
    x = bf16(pool.g, 2, 1, 64).cuda()
    cu = offsets([1, 1]).cuda()
    for bad in (-1, pool.total, 2 ** 31 - 1, -2 ** 31):
        t = good.copy()
        t[0, 1] = bad
        t[1, 1] = bad
        t = torch.tensor(t).cuda()
        o, _ = binding.kv4_forward(x, pool.cache, t, pool.lens_t, cu_seqlens=cu)
        with pytest.raises(binding.AttnError):
            binding.check_status()
        assert torch.isfinite(o).all()
        with pytest.raises(binding.AttnError):
            binding.kv4_append(pool.cache, x, x, t, pool.lens_t, cu_seqlens=cu)
            binding.check_status()
        with pytest.raises(binding.AttnError):
            binding.kv4_read(pool.cache, t, pool.lens_t, 300, cu_seqlens=offsets([200, 100]).cuda())
            binding.check_status()
    for lens, c in (([257, 100], [1, 1]), ([-1, 100], [1, 1]), ([2 ** 31 - 1, 5], [1, 1]), ([200, 100], [-1, 3]),
                    ([200, 100], [5, -3]), ([200, 100], [2 ** 30, 1])):
        lt = torch.tensor(lens, dtype=torch.int32).cuda()
        ct = torch.tensor([0, c[0], c[0] + c[1]], dtype=torch.int32).cuda()
        w = torch.zeros((2, 1, 256), device="cuda")
        for call in (lambda: binding.kv4_forward(x, pool.cache, pool.table, lt, cu_seqlens=ct, key_weights=w),):
            with pytest.raises(binding.AttnError):
                call()
                binding.check_status()
    binding.check_status()   # reported once, then clear


# ------------------------------------------------------------------ eviction

def plain_evict(w, n, budget, sinks, recent):
    if n <= budget:
        return list(range(n))
    key = [-math.inf if math.isnan(x) else x for x in w.tolist()]
    middle = sorted(range(sinks, n - recent), key=lambda j: (-key[j], j))[:budget - sinks - recent]
    return sorted(list(range(sinks)) + middle + list(range(n - recent, n)))


@pytest.mark.gpu
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (192, 128), (256, 256)])
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (64, 4, 20), (100, 0, 0), (100, 40, 60),
                                                 (333, 7, 100), (5000, 3, 3)])
def test_evict(d, dv, budget, sinks, recent):
    lens = [0, 1, 64, budget, budget + 1, 700, 3000]
    new_pages = -(-budget // PAGE)
    pool = Pool(lens, 2, d, dv, seed=23, extra=len(lens) * new_pages)
    g = pool.g
    w = g.random((len(lens), 2, pool.width * PAGE)).astype(np.float32)
    w[3:5, 0] = np.round(w[3:5, 0] * 4) / 4            # many equal weights
    w[5, 1] = 0.5                                      # all equal
    w[6, 0, ::3] = np.nan
    w[6, 1] *= np.where(g.random(w[6, 1].shape) < 0.5, -1, 1)
    w[6, 1, ::5] = 0.0
    w[6, 1, 1::5] = -0.0
    w[5, 0, 10:20] = [np.inf, -np.inf] * 5
    new_table = pool.spare[:len(lens) * new_pages].reshape(len(lens), new_pages).astype(np.int32)
    before = [x.clone() for x in pool.host]
    wide = torch.full((len(lens), 2, budget + 5), 9.0, device="cuda")
    new_lens, kept, new_w = binding.kv4_evict(pool.cache, pool.table, pool.lens_t, torch.tensor(w).cuda(),
                                              torch.tensor(new_table).cuda(), budget=budget, sinks=sinks,
                                              recent=recent, new_key_weights=wide)
    binding.check_status()
    pool.download()
    assert new_lens.tolist() == [min(n, budget) for n in lens]
    for b, n in enumerate(lens):
        for h in range(2):
            want = plain_evict(w[b, h], n, budget, sinks, recent)
            m = len(want)
            assert kept[b, h].tolist() == want + [-1] * (budget - m), (b, h)
            assert np.array_equal(new_w[b, h, :m].cpu().numpy(), w[b, h, want], equal_nan=True)
            assert (new_w[b, h, m:] == 0).all()
            src, dst = np.array(want, dtype=np.int64), np.arange(m)
            sp = pool.table_host[b][src // PAGE].astype(np.int64) if m else src
            dp = new_table[b][dst // PAGE].astype(np.int64)
            for part in range(4):
                assert torch.equal(pool.host[part][dp, h][:, :][np.arange(m), :, dst % PAGE].view(torch.uint8),
                                   before[part][sp, h][np.arange(m), :, src % PAGE].view(torch.uint8))
    for part in range(4):   # the old pages are as they were
        old = np.unique(pool.table_host[pool.table_host >= 0])
        assert torch.equal(pool.host[part][old].view(torch.uint8), before[part][old].view(torch.uint8))


@pytest.mark.gpu
def test_evict_long_cache():
    pool = Pool([100000], 1, 64, seed=24, extra=800)
    w = pool.g.random((1, 1, pool.width * PAGE)).astype(np.float32) ** 8
    table = torch.tensor(pool.spare[:800].reshape(1, 800).astype(np.int32)).cuda()
    _, kept, _ = binding.kv4_evict(pool.cache, pool.table, pool.lens_t, torch.tensor(w).cuda(), table, budget=50001,
                                   sinks=4, recent=1000)
    binding.check_status()
    assert kept[0, 0].tolist() == plain_evict(w[0, 0], 100000, 50001, 4, 1000)


@pytest.mark.gpu
def test_evict_reports_bad_pages():
    pool = Pool([200], 1, 64, seed=25, extra=4)
    w = torch.rand(1, 1, 256, device="cuda")
    for bad_old, bad_new in ((True, False), (False, True)):
        old, new = pool.table.clone(), torch.tensor(pool.spare[None, :2].astype(np.int32)).cuda()
        if bad_old:
            old[0, 0] = pool.total + 3
        if bad_new:
            new[0, 1] = -4
        binding.kv4_evict(pool.cache, old, pool.lens_t, w, new, budget=100, sinks=70)
        with pytest.raises(binding.AttnError):
            binding.check_status()
    binding.kv4_evict(pool.cache, pool.table, torch.tensor([2 ** 31 - 1], dtype=torch.int32).cuda(), w, new * 0, budget=100)
    with pytest.raises(binding.AttnError):
        binding.check_status()


@pytest.mark.gpu
def test_pages_past_32_bit_offsets():
    """A cache of more than 4 GB per tensor: its last pages work like its first ones."""
    n_pages, Hkv, d = 70000, 8, 256
    cache = binding.Kv4Cache.empty(n_pages, Hkv, d)
    assert cache.k_codes.numel() > 2 ** 32
    g = np.random.default_rng(27)
    k, v, q = (bf16(g, 300, h, d).cuda() for h in (Hkv, Hkv, 16))
    lens, cu = torch.tensor([300], dtype=torch.int32).cuda(), offsets([300]).cuda()
    got = []
    for first in (0, n_pages - 12):
        table = torch.arange(first, first + 5, dtype=torch.int32).cuda()[None]
        new = torch.arange(first + 6, first + 9, dtype=torch.int32).cuda()[None]
        binding.kv4_append(cache, k, v, table, lens, cu_seqlens=cu)
        w = torch.zeros(1, Hkv, 320, device="cuda")
        o, lse = binding.kv4_forward(q[-2:], cache, table, lens, cu_seqlens=offsets([2]).cuda(), key_weights=w)
        new_lens, kept, _ = binding.kv4_evict(cache, table, lens, w, new, budget=150, sinks=4, recent=30)
        rk, rv = binding.kv4_read(cache, new, new_lens, 150, cu_seqlens=offsets([150]).cuda())
        got.append((o, lse, w, kept, rk, rv))
    binding.check_status()
    assert all(torch.equal(a, b) for a, b in zip(*got)) and (got[0][0] != 0).any()


# ------------------------------------------------------------------ together

@pytest.mark.gpu
@pytest.mark.parametrize("d,H,Hkv", [(64, 4, 4), (128, 8, 2)])
def test_serving_loop(d, H, Hkv):
    """Prefill into the cache, decode with accumulated weights, evict, decode on: every step against float64 on
    what the cache holds, and the prefill's read-back run through the dense forward gives the same output."""
    lens, budget, window = [300, 150], 128, (90, -1)
    pool = Pool([n + 70 for n in lens], Hkv, d, seed=26, extra=8)
    pool.lens = list(lens)

    def step(new):
        k, v = bf16(pool.g, sum(new), Hkv, d), bf16(pool.g, sum(new), Hkv, d)
        pool.lens_t = torch.tensor(pool.lens, dtype=torch.int32).cuda()
        binding.kv4_append(pool.cache, k.cuda(), v.cuda(), pool.table, pool.lens_t, cu_seqlens=offsets(new).cuda())
        pool.download()

    step(lens)
    q = bf16(pool.g, sum(lens), H, d)
    o, _, _ = check_forward(pool, lens, H, q=q, window=window, sinks=4, what="prefill")
    cu = offsets(lens).cuda()
    k, v = binding.kv4_read(pool.cache, pool.table, pool.lens_t, sum(lens), cu_seqlens=cu)
    dense, _ = binding.forward(q.cuda(), k, v, causal=True, cu_seqlens=cu, window=window, sinks=4)
    assert (dense.float() - o.float()).abs().max() <= 2.0 ** -5 * o.float().abs().max()
    w = torch.zeros((2, Hkv, pool.width * PAGE), device="cuda")
    total = torch.zeros((2, Hkv), dtype=torch.float64)
    for n in ([1, 1], [3, 2]):
        pool.lens = [a + b for a, b in zip(pool.lens, n)]
        step(n)
        q = bf16(pool.g, sum(n), H, d)
        binding.kv4_forward(q.cuda(), pool.cache, pool.table, pool.lens_t, cu_seqlens=offsets(n).cuda(), key_weights=w)
        check_forward(pool, n, H, q=q, what="decode")
        total += torch.tensor(n, dtype=torch.float64)[:, None] * (H // Hkv)
    # every row's weights sum to one
    assert (w.double().sum(-1).cpu() - total).abs().max() <= 2.0 ** -13 * total.max()
    table = torch.tensor(pool.spare[:6].reshape(2, 3).astype(np.int32)).cuda()
    w2 = torch.zeros((2, Hkv, 192), device="cuda")
    new_lens, kept, _ = binding.kv4_evict(pool.cache, pool.table, pool.lens_t, w, table, budget=budget, sinks=4,
                                          recent=32, new_key_weights=w2)
    for b in range(2):
        for h in range(Hkv):
            assert kept[b, h].tolist() == plain_evict(w[b, h].cpu().numpy(), pool.lens[b], budget, 4, 32)
    pool.lens, pool.table, pool.table_host, pool.width = new_lens.tolist(), table, table.cpu().numpy(), 3
    for n in ([1, 1], [2, 1]):
        pool.lens = [a + b for a, b in zip(pool.lens, n)]
        step(n)
        check_forward(pool, n, H, decay=1.0, window=window, sinks=4, what="after eviction")
    binding.check_status()


# ------------------------------------------------------------------ refusals (no GPU)

@pytest.fixture(scope="module")
def lib():
    from exact_attention_blackwell_tma_gb300 import build
    build.build()
    return binding.load()


X = 1 << 20   # an address that is never used: the checks come first


def struct(d=64, dv=64, pages=4, Hkv=2, at=X):
    return binding._Kv4Struct(at, X, X, X, pages, Hkv, d, dv)


@pytest.mark.parametrize("bad,code", [(dict(d=96, dv=96), -1), (dict(d=128, dv=64), -1), (dict(pages=0), -1),
                                      (dict(Hkv=0), -1), (dict(at=None), -1), (dict(at=X + 4), -2)])
def test_refuses_caches(lib, bad, code):
    c = struct(**bad)
    assert lib.attn_kv4_append(X, X, 512, 512, c, X, 3, X, None, 1, 1, None) == code
    assert lib.attn_kv4_read(X, X, c, X, 3, X, None, 1, 1, None) == code
    assert lib.attn_kv4_fwd(X, 1024, c, X, 3, X, None, X, X, 1, 4, 1, 0.1, 1, -1, -1, 0, None, 0, 1.0, X, 1 << 40,
                            None) == code
    assert lib.attn_kv4_evict(c, X, 3, X, X, 192, X + 64, 1, 1, 10, 0, 0, X + 128, X, X + 64, 10, None) == code
    assert binding.last_error()


def test_refuses_arguments(lib):
    c = struct()
    ap = lambda k=X, ks=128, vs=128, table=X, width=3, lens=X, B=1, L=1: lib.attn_kv4_append(  # noqa: E731
        k, X, ks, vs, c, table, width, lens, None, B, L, None)
    for kw in (dict(k=None), dict(ks=120), dict(vs=132), dict(table=None), dict(width=0), dict(lens=None), dict(B=-1),
               dict(B=1025), dict(L=-1), dict(B=1000, L=2 ** 31 - 1), dict(width=2 ** 31 - 1), dict(width=2 ** 24), dict(L=2 ** 30)):
        assert ap(**kw) == binding.ATTN_ERR_ARG, kw
    assert ap(k=X + 2) == binding.ATTN_ERR_ALIGN
    assert ap(B=0) == 0 and ap(L=0) == 0
    need = lib.attn_kv4_fwd_workspace_size(1, 4, 2, 1, 0, 3, 64, 64, 0)
    assert need > 0 and need % 256 == 0
    assert lib.attn_kv4_fwd_workspace_size(1, 4, 2, 1, 0, 3, 64, 64, 1) >= need + 4 * 4 * 192
    assert lib.attn_kv4_fwd_workspace_size(1, 4, 3, 1, 0, 3, 64, 64, 0) == 0

    def fwd(q=X, qs=256, H=4, scale=0.1, wl=-1, wr=-1, sinks=0, w=None, stride=0, decay=1.0, ws=X, size=need, o=X, L=1,
            B=1, width=3):
        return lib.attn_kv4_fwd(q, qs, c, X, width, X, None, o, X, B, H, L, scale, 1, wl, wr, sinks, w, stride, decay, ws,
                                size, None)
    for kw in (dict(q=None), dict(qs=128), dict(qs=260), dict(H=3), dict(H=0), dict(scale=0.0), dict(scale=math.inf),
               dict(scale=math.nan), dict(wl=-2), dict(wr=-5), dict(sinks=-1), dict(w=X, stride=0, size=1 << 40),
               dict(w=X, stride=9, decay=1.5, size=1 << 40), dict(w=X, stride=9, decay=math.nan, size=1 << 40),
               dict(o=None), dict(L=2 ** 27, width=2 ** 20)):
        assert fwd(**kw) == binding.ATTN_ERR_ARG, kw
    assert fwd(size=need - 1) == binding.ATTN_ERR_WORKSPACE and fwd(ws=None) == binding.ATTN_ERR_WORKSPACE
    assert fwd(ws=X + 16) == binding.ATTN_ERR_ALIGN and fwd(o=X + 8) == binding.ATTN_ERR_ALIGN
    assert fwd(L=0) == 0 and fwd(B=0) == 0

    def evict(w=X, stride=192, table=X + 64, width=1, budget=10, sinks=0, recent=0, lens=X + 128, nw=X + 64, ns=10):
        return lib.attn_kv4_evict(c, X, 3, X, w, stride, table, width, 1, budget, sinks, recent, lens, X, nw, ns, None)
    for kw in (dict(w=None), dict(stride=0), dict(table=None), dict(table=X), dict(width=0), dict(budget=0),
               dict(budget=65, ns=65), dict(sinks=-1), dict(recent=-1), dict(sinks=6, recent=5), dict(lens=X), dict(nw=X),
               dict(ns=9), dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1)):
        assert evict(**kw) == binding.ATTN_ERR_ARG, kw


def test_binding_refuses_tensors():
    codes, params = torch.zeros(3, 2, 1, 64, 32, dtype=torch.uint8), torch.zeros(3, 2, 1, 64, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError):   # not on a GPU
        binding.Kv4Cache(codes, params, codes, params)
    with pytest.raises(ValueError):
        binding.Kv4Cache(codes.int(), params, codes, params)
    with pytest.raises(ValueError):
        binding.Kv4Cache(codes, params[:, :, :, :, :1], codes, params)
    with pytest.raises(ValueError):
        binding.Kv4Cache(codes, params, codes[:2], params[:2])
    rows = lambda x, B=2, cu=None: binding._kv4_rows(x, 4, 64, B, cu is not None, "q", -1)  # noqa: E731
    x = torch.zeros(2, 5, 6, 64, dtype=torch.bfloat16)
    assert rows(x[:, :, 1:5]) == (5, 384) and rows(x[0, :, :4], 2, 1) == (5, 384)
    for bad in (x[:, :, :3], x.float()[:, :, :4], x[0, :, :4], x[:, ::2, :4][:, :, :, :32], x[:, :4, :4],
                x.transpose(1, 2)[:, :, :4]):
        with pytest.raises(ValueError):
            rows(bad)
