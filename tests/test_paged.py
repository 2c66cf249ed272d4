"""The paged key/value cache in bf16 and 8 bits (append, read, attention) against float64.

Bounds. Codes, scales and what is read back are compared exactly. Attention: P (with V's power of two) is
rounded to bf16 (half a step: 2^-8) before it multiplies a value, the output once more; scores, statistics and
sums are fp32, which for scores below about 100 moves p by less than 2^-13 of itself. So |O - ref| <=
(2^-8 + 2^-12) sum p |v| + 2^-8 |ref|.
"""
import math

import numpy as np
import pytest
import torch

from exact_attention_blackwell_tma_gb300 import binding
from _plain import U, SLACK, assert_lse, assert_within, visible

PAGE = binding.PAGED_PAGE
DIMS = [(64, 64), (128, 128), (192, 192), (192, 128), (256, 256)]
BITS = [16, 8]
gpu = pytest.mark.gpu


def e4m3_values():
    """The value of every byte, from the format's definition: sign, 4 bits of exponent (bias 7), 3 of mantissa; NaN: 7f, ff."""
    out = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
        out.append(math.nan if c & 127 == 127 else -x if c & 128 else x)
    return np.array(out)


VALUES = e4m3_values()


def quantised(x):
    """The definition, by looking for the nearest code: float64 [..., width] -> codes, scale bytes."""
    top = np.abs(x).max(-1)
    e = np.full(top.shape, -126)
    for i in range(-125, 121):
        e = np.where(top > 448.0 * 2.0 ** (i - 1), i, e)
    y = np.abs(x) / (2.0 ** e.astype(float))[..., None]
    sizes = VALUES[:127]
    hi = np.clip(np.searchsorted(sizes, y), 1, 126)
    a, b = y - sizes[hi - 1], sizes[hi] - y
    code = np.where((a < b) | ((a == b) & (hi % 2 == 1)), hi - 1, hi)   # a tie: the even code
    bad = ~np.isfinite(x).all(-1)
    code = np.where(np.signbit(x), code + 128, code)
    code[bad] = 0
    return code.astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def bf16(g, *shape):
    return torch.tensor(g.standard_normal(shape), dtype=torch.float32).to(torch.bfloat16)


def offsets(ns):
    return torch.tensor([0] + list(np.cumsum(ns)), dtype=torch.int32)


class Pool:
    """A cache with pages handed out in a shuffled order, random contents."""

    def __init__(self, bits, lens, Hkv, d, dv=None, seed=0, extra=0, width=None):
        self.bits, self.Hkv, self.d, self.dv, self.lens = bits, Hkv, d, d if dv is None else dv, list(lens)
        self.g = g = np.random.default_rng(seed)
        need = [-(-n // PAGE) for n in lens]
        total = max(1, sum(need) + extra)
        ids = g.permutation(total)
        self.width = max([1] + need) if width is None else width
        table, at = np.full((len(lens), self.width), -7, np.int32), 0   # entries past a sequence's pages are never read
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
        self.table_host = table
        self.table, self.lens_t = torch.tensor(table).cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.host = []   # k, its scales, v, its scales
        for w in (self.d, self.dv):
            if bits == 16:
                self.host += [bf16(g, total, Hkv, PAGE, w), None]
            else:
                code = g.integers(0, 127, (total, Hkv, PAGE, w)) + 128 * g.integers(0, 2, (total, Hkv, PAGE, w))
                # sizes of 2^-7 and less next to 2^-2 .. 2^1, scales over a factor of 16: values of about 1
                self.host += [torch.tensor(code.astype(np.uint8)), torch.tensor(g.integers(118, 122, (total, Hkv, PAGE)).astype(np.uint8))]
        self.upload()

    def upload(self):
        k, ks, v, vs = (None if x is None else x.cuda() for x in self.host)
        if self.bits == 8:
            k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
        self.cache = binding.PagedCache(k, v, ks, vs)

    def download(self):
        c = self.cache
        as_bytes = (lambda x: x.view(torch.uint8)) if self.bits == 8 else (lambda x: x)
        self.host = [None if x is None else x.cpu() for x in (as_bytes(c.k), c.k_scales, as_bytes(c.v), c.v_scales)]

    def values(self, b, which, n=None):
        """Sequence b's keys (which = 0) or values (1) in float64, [tokens, Hkv, width]."""
        j = np.arange(self.lens[b] if n is None else n)
        page = self.table_host[b][j // PAGE].astype(np.int64)
        rows, scales = self.host[2 * which], self.host[2 * which + 1]
        x = rows[page, :, j % PAGE]
        if self.bits == 16:
            return x.double()
        e = scales[page, :, j % PAGE].numpy().astype(int)
        f = np.where(e == 255, math.nan, 2.0 ** (e - 127.0))
        return torch.tensor(VALUES[x.numpy()] * f[..., None])

    def put(self, b, which, j, x):
        """Token j of every head of sequence b becomes x (bf16 caches)."""
        self.host[2 * which][int(self.table_host[b][j // PAGE]), :, j % PAGE] = x


# ------------------------------------------------------------------ append and read

def check_appended(pool, new, k, v, before):
    """The new rows follow the definition; every other token of the pool is as before."""
    pool.download()
    want, at = [None if x is None else x.clone() for x in before], 0
    for b, n in enumerate(new):
        j = np.arange(pool.lens[b] - n, pool.lens[b])
        page = pool.table_host[b][j // PAGE].astype(np.int64)
        for which, x in enumerate((k, v)):
            rows = x[at:at + n]
            if pool.bits == 16:
                want[2 * which][page, :, j % PAGE] = rows
            elif n:
                c, e = quantised(rows.double().numpy())
                want[2 * which][page, :, j % PAGE] = torch.tensor(c)
                want[2 * which + 1][page, :, j % PAGE] = torch.tensor(e)
        at += n
    for name, got, ref in zip(("k", "k scales", "v", "v scales"), pool.host, want):
        assert got is None or torch.equal(got.contiguous().view(torch.uint8), ref.contiguous().view(torch.uint8)), name


@gpu
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("d,dv", DIMS)
@pytest.mark.parametrize("new,lens", [([1], [1]), ([1, 1, 1], [64, 65, 500]), ([130, 0, 64, 3], [130, 77, 200, 66]),
                                      ([5, 700], [5, 701])])
@pytest.mark.parametrize("Hkv", [1, 5])
def test_append_and_read_packed(bits, d, dv, new, lens, Hkv):
    pool = Pool(bits, lens, Hkv, d, dv, seed=d + len(lens))
    before = pool.host
    # sizes over many powers of two, so that codes of every exponent occur
    k, v = ((bf16(pool.g, sum(new), Hkv, w).float() * 2.0 ** torch.tensor(pool.g.integers(-9, 3, (sum(new), Hkv, w)))).to(
        torch.bfloat16) for w in (d, dv))
    binding.paged_append(pool.cache, k.cuda(), v.cuda(), pool.table, pool.lens_t, cu_seqlens=offsets(new).cuda())
    binding.check_status()
    check_appended(pool, new, k, v, before)
    got = binding.paged_read(pool.cache, pool.table, pool.lens_t, sum(lens), cu_seqlens=offsets(lens).cuda())
    binding.check_status()
    at = 0
    for b, n in enumerate(lens):
        for which in (0, 1):
            assert torch.equal(got[which][at:at + n].cpu(), pool.values(b, which).to(torch.bfloat16)), (b, which)
        at += n


@gpu
def test_append_hard_values():
    """Ties, the border of a scale, zeros of both signs, subnormals, the largest values, NaN and infinities."""
    nan, inf = math.nan, math.inf
    rows = [[448.0], [449.0], [450.0, 1.0], [464.0, 465.0, 466.0], [0.0], [-0.0], [1.0, 1.0625, 1.1875, 1.3125, -1.0625],
            [448.0, 2.0 ** -10, 3 * 2.0 ** -10, 5 * 2.0 ** -10, 2.0 ** -9, -(2.0 ** -11)], [2.0 ** -126], [2.0 ** -133], [2.0 ** -117],
            [1.75 * 2.0 ** -118], [1.7578125 * 2.0 ** -118], [3.3895313892515355e38, 1.0], [-3.3895313892515355e38], [nan, 1.0],
            [1.0, inf], [-inf], [2.0 ** 100, 2.0 ** 80], [1.75, 1.7578125]]
    x = torch.zeros(len(rows), 1, 64)
    for i, r in enumerate(rows):
        x[i, 0, 7:7 + len(r)] = torch.tensor(r)
    x = x.to(torch.bfloat16)
    pool = Pool(8, [len(rows)], 1, 64)
    before = pool.host
    binding.paged_append(pool.cache, x.cuda(), x.cuda(), pool.table, pool.lens_t, cu_seqlens=offsets([len(rows)]).cuda())
    check_appended(pool, [len(rows)], x, x, before)
    k, _ = binding.paged_read(pool.cache, pool.table, pool.lens_t, len(rows), cu_seqlens=offsets([len(rows)]).cuda())
    want = pool.values(0, 0).to(torch.bfloat16)
    assert torch.equal(torch.isnan(k.cpu()), torch.isnan(want)) and torch.isnan(k[15:18]).all()
    assert torch.equal(k.cpu().nan_to_num(), want.nan_to_num())
    binding.check_status()


@gpu
@pytest.mark.parametrize("bits", BITS)
def test_append_dense_strided_and_rows_behind_the_last(bits):
    pool = Pool(bits, [130, 67], 2, 64, 64, seed=3)
    before = pool.host
    fused = bf16(pool.g, 2, 3, 5, 64).cuda()
    binding.paged_append(pool.cache, fused[:, :, 1:3], fused[:, :, 3:], pool.table, pool.lens_t)
    binding.check_status()
    check_appended(pool, [3, 3], fused[:, :, 1:3].flatten(0, 1).cpu(), fused[:, :, 3:].flatten(0, 1).cpu(), before)
    # packed rows behind the last sequence are neither appended nor written by a read
    before = pool.host
    x = bf16(pool.g, 9, 2, 64)
    binding.paged_append(pool.cache, x.cuda(), x.cuda(), pool.table, pool.lens_t, cu_seqlens=offsets([2, 4]).cuda())
    check_appended(pool, [2, 4], x, x, before)
    out = [torch.full((9, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    binding.paged_read(pool.cache, pool.table, pool.lens_t, 9, cu_seqlens=offsets([2, 4]).cuda(), k=out[0], v=out[1])
    assert all((t[6:] == 7).all() for t in out)
    assert torch.equal(out[0][2:6].cpu(), pool.values(1, 0)[-4:].to(torch.bfloat16))
    # a padded dense batch: zeros before a sequence's first token
    pool = Pool(bits, [2, 0, 5], 2, 64, seed=4)
    k, v = binding.paged_read(pool.cache, pool.table, pool.lens_t, 4)
    assert (k[0, :2] == 0).all() and (v[1] == 0).all() and torch.equal(k[2].cpu(), pool.values(2, 0)[1:].to(torch.bfloat16))
    binding.check_status()


# ------------------------------------------------------------------ attention

def check_forward(pool, new, H, causal=True, window=(-1, -1), sinks=0, q=None, packed=True, scale=None, what=""):
    T = sum(new)
    q = bf16(pool.g, T, H, pool.d) if q is None else q
    scale = 1 / math.sqrt(pool.d) if scale is None else scale
    gq = q.cuda() if packed else q.reshape(len(new), -1, H, pool.d).cuda()
    o, lse = binding.paged_forward(gq, pool.cache, pool.table, pool.lens_t, causal=causal, scale=scale,
                                   cu_seqlens=offsets(new).cuda() if packed else None, window=window, sinks=sinks)
    binding.check_status()
    o2 = o.reshape(T, H, pool.dv)
    lse2 = lse if packed else lse.transpose(0, 1).reshape(H, T)
    r, at = H // pool.Hkv, 0
    for b, n in enumerate(new):
        N = pool.lens[b]
        ok = visible(n, N, causal, window, sinks)
        k, v = (pool.values(b, which).repeat_interleave(r, 1).nan_to_num(0.0, 0.0, 0.0) for which in (0, 1))
        s = torch.einsum("ihd,jhd->hij", q[at:at + n].double(), k) * scale
        s = s.masked_fill(~ok, -math.inf)
        ref_lse = torch.logsumexp(s, -1) if N else torch.full((H, n), -math.inf, dtype=torch.float64)
        p = torch.where(ok, torch.exp(s - torch.where(torch.isfinite(ref_lse), ref_lse, 0.0)[..., None]), 0.0)
        ref, spread = torch.einsum("hij,jhd->ihd", p, v), torch.einsum("hij,jhd->ihd", p, v.abs())
        assert_within(o2[at:at + n], ref, (U + SLACK) * spread + U * ref.abs(), f"{what} sequence {b} O")
        assert_lse(lse2[:, at:at + n], ref_lse, f"{what} sequence {b}", scores=100.0)
        at += n
    return o, lse


@gpu
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("d,dv", DIMS)
@pytest.mark.parametrize("H,Hkv", [(1, 1), (2, 2), (8, 2), (6, 2), (16, 1), (12, 1)])
def test_forward_one_token(bits, d, dv, H, Hkv):
    lens = [1, 63, 64, 65, 200, 1000]
    check_forward(Pool(bits, lens, Hkv, d, dv, seed=6), [1] * len(lens), H, what=f"d={d}/{dv} H={H}/{Hkv}")


@gpu
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("d,dv", DIMS)
@pytest.mark.parametrize("window,sinks", [((-1, -1), 0), ((0, -1), 0), ((10, -1), 4), ((64, -1), 64), ((100, -1), 70),
                                          ((300, -1), 1), ((2 ** 31 - 1, -1), 2 ** 31 - 1)])
def test_forward_window_and_sinks(bits, d, dv, window, sinks):
    """1 to 16 tokens, empty sequences, a cache shorter than its rows."""
    lens, new = [700, 64, 5, 0, 333, 129, 3], [16, 3, 5, 0, 0, 1, 2]
    check_forward(Pool(bits, lens, 2, d, dv, seed=7), new, 6, window=window, sinks=sinks, what=f"{window} {sinks}")


@gpu
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("causal,window", [(False, (-1, -1)), (False, (30, 20)), (False, (-1, 5)), (True, (7, 9))])
def test_forward_other_masks(bits, causal, window):
    lens, new = [400, 90, 130], [9, 2, 70]
    check_forward(Pool(bits, lens, 1, 64, seed=8), new, 3, causal=causal, window=window, sinks=3, what=f"{causal} {window}")


@gpu
@pytest.mark.parametrize("bits", BITS)
def test_forward_rows_without_keys(bits):
    """More rows than cached tokens: the first rows see nothing (O = 0, LSE = -inf); so does an empty cache."""
    o, lse = check_forward(Pool(bits, [4, 0, 70], 1, 128, seed=9), [9, 3, 2], 2)
    assert (o[:5] == 0).all() and torch.isneginf(lse[:, :5]).all() and (o[9:12] == 0).all()


@gpu
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("d,n,H,Hkv", [(64, 40, 8, 1), (128, 33, 4, 2), (256, 20, 2, 1), (128, 200, 2, 2)])
def test_forward_many_rows(bits, d, n, H, Hkv):
    check_forward(Pool(bits, [300, n, 2000], Hkv, d, seed=10), [n, n, n], H, what=f"{n} rows")


@gpu
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_forward_row_blocks(bits, d):
    """Numbers of rows around those that a warp, and a thread block, holds at once."""
    new = [7, 8, 9, 15, 16, 17, 24, 31, 32, 33, 48, 63, 64, 65]
    check_forward(Pool(bits, [n + 100 + 13 * n for n in new], 1, d, seed=16), new, 1, window=(90, -1), sinks=3)
    check_forward(Pool(bits, [150] * 9, 1, d, seed=17), [1, 2, 3, 4, 5, 6, 7, 8, 9], 4)


@gpu
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("L", [1, 4])
def test_forward_dense_batch(bits, L):
    check_forward(Pool(bits, [100, 250, 64, 4], 2, 128, seed=11), [L] * 4, 8, packed=False)


@gpu
@pytest.mark.parametrize("bits", BITS)
def test_forward_long_and_ragged(bits):
    """One long cache shared by many thread blocks beside short ones; strided queries; the same bits again."""
    pool = Pool(bits, [40000, 17, 3000, 9000], 1, 128, seed=12)
    fused = bf16(pool.g, 8, 6, 128)
    o, lse = check_forward(pool, [1, 2, 1, 4], 4, q=fused[:, 1:5])
    again = binding.paged_forward(fused.cuda()[:, 1:5], pool.cache, pool.table, pool.lens_t, cu_seqlens=offsets([1, 2, 1, 4]).cuda())
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@gpu
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("window,sinks", [((-1, -1), 0), ((50, -1), 4)])
def test_forward_ignores_what_it_masks(bits, window, sinks):
    """NaN and infinities in unwritten slots of the last page and in keys left of the window change nothing."""
    lens = [130, 200, 77]
    pool = Pool(bits, lens, 2, 128, seed=14)
    for b, n in enumerate(lens):
        dead = list(range(n, -(-n // PAGE) * PAGE))
        if window[0] >= 0:
            dead += list(range(sinks, n - 1 - window[0] - 1))   # two rows: the first one's window reaches furthest
        for j in dead:
            page = int(pool.table_host[b][j // PAGE])
            for which in (0, 2):
                if bits == 16:
                    pool.host[which][page, :, j % PAGE] = math.nan if j % 2 else math.inf
                else:
                    pool.host[which][page, :, j % PAGE] = 127 if j % 2 else 0
                    pool.host[which + 1][page, :, j % PAGE] = 255
    pool.upload()
    check_forward(pool, [2, 2, 2], 4, window=window, sinks=sinks)


@gpu
def test_forward_codes_mask_per_row():
    """A row of NaN in the 8-bit cache that only the last query sees leaves the ones before it alone."""
    pool = Pool(8, [100], 1, 64, seed=15)
    page = int(pool.table_host[0][99 // PAGE])
    pool.host[2][page, 0, 99 % PAGE] = 0
    pool.host[3][page, 0, 99 % PAGE] = 255
    pool.upload()
    q = bf16(pool.g, 3, 2, 64).cuda()
    o, lse = binding.paged_forward(q, pool.cache, pool.table, pool.lens_t, cu_seqlens=offsets([3]).cuda())
    assert torch.isfinite(o[:2]).all() and torch.isnan(o[2]).all() and torch.isfinite(lse).all()


@gpu
@pytest.mark.parametrize("e", [8, 60, 127, 200, 239])
def test_forward_value_scales(e):
    """V's scales over a factor of 2^16 around any size."""
    pool = Pool(8, [700], 1, 128, seed=16)
    pool.host[3] = torch.tensor(pool.g.integers(e - 7, e + 9, pool.host[3].shape).astype(np.uint8))
    pool.upload()
    if e < 20:   # (below the smallest normal numbers bf16 has absolute steps of 2^-133)
        o, _ = binding.paged_forward(bf16(pool.g, 2, 4, 128).cuda(), pool.cache, pool.table, pool.lens_t, cu_seqlens=offsets([2]).cuda())
        assert torch.isfinite(o).all() and o.abs().max() > 0
    check_forward(pool, [2], 4, what=f"scales {e}")


@gpu
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("size", [2.0 ** -80, 2.0 ** -30, 2.0 ** -8, 2.0 ** 8, 2.0 ** 40])
def test_forward_query_sizes(bits, size):
    """Rows of very different size in one block; the scale undoes the size."""
    pool = Pool(bits, [300], 1, 64, seed=17)
    q = (bf16(pool.g, 4, 3, 64).float() * size * 2.0 ** torch.arange(-4, 8).reshape(4, 3, 1)).to(torch.bfloat16)
    check_forward(pool, [4], 3, q=q, scale=2.0 ** -9 / size, what=f"queries {size}")


@gpu
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("junk", [3e38, 1e10, math.inf, math.nan, 0.0])
def test_forward_unused_rows_hold_anything(bits, junk):
    """Rows before a short sequence's tokens see no key, and neither they nor a neighbour's bad row reach the others."""
    pool = Pool(bits, [2, 100], 2, 128, seed=28)
    q = bf16(pool.g, 2, 4, 4, 128)
    clean = q.clone()
    q[0, :2] = junk
    q[1, 1, 2] = junk
    o, lse = binding.paged_forward(q.cuda(), pool.cache, pool.table, pool.lens_t)
    o2, lse2 = binding.paged_forward(clean.cuda(), pool.cache, pool.table, pool.lens_t)
    assert (o[0, :2] == 0).all() and torch.isneginf(lse[0, :, :2]).all()
    keep = torch.ones(2, 4, 4, dtype=torch.bool)
    keep[1, 1, 2] = False
    assert torch.equal(o.cpu()[keep], o2.cpu()[keep]) and torch.equal(lse.cpu().transpose(1, 2)[keep], lse2.cpu().transpose(1, 2)[keep])
    binding.check_status()


@gpu
def test_forward_a_maximum_that_climbs():
    pool = Pool(16, [2000], 1, 64, seed=18)
    for j in range(2000):
        pool.put(0, 0, j, pool.host[0][0, 0, 0] * 0 + j * 0.01)
    pool.upload()
    check_forward(pool, [1], 2, q=bf16(pool.g, 1, 2, 64).abs(), scale=0.1)


@gpu
@pytest.mark.parametrize("bits", BITS)
def test_forward_largest_batch_and_shared_pages(bits):
    lens = [(37 * i) % 150 for i in range(1024)]
    check_forward(Pool(bits, lens, 1, 64, seed=20), [min(1, n) for n in lens], 2)
    pool = Pool(bits, [500, 500], 2, 128, seed=19)
    pool.table_host[1, :5] = pool.table_host[0, :5]
    pool.table = torch.tensor(pool.table_host).cuda()
    check_forward(pool, [2, 2], 8)


@gpu
@pytest.mark.parametrize("bits", BITS)
def test_forward_captured_and_on_other_streams(bits):
    pool = Pool(bits, [3000, 70], 2, 128, seed=21)
    q = bf16(pool.g, 2, 8, 128).cuda()
    cu = offsets([1, 1]).cuda()
    args = (pool.cache, pool.table, pool.lens_t)
    want, lse = binding.paged_forward(q, *args, cu_seqlens=cu)
    graph, static = torch.cuda.CUDAGraph(), torch.zeros_like(q)
    with torch.cuda.graph(graph):
        o, l2 = binding.paged_forward(static, *args, cu_seqlens=cu)
    static.copy_(q)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(l2, lse)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[binding.paged_forward(q, *args, cu_seqlens=cu, stream=s)[0] for s in streams] for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for pair in outs for x in pair)


@gpu
@pytest.mark.parametrize("bits", BITS)
def test_bad_pages_lengths_and_offsets_are_reported(bits):
    pool = Pool(bits, [200, 100], 1, 64, seed=22)
    q, x = bf16(pool.g, 2, 2, 64).cuda(), bf16(pool.g, 2, 1, 64).cuda()
    cu = offsets([1, 1]).cuda()

    def reported(table, lens, cu, out=True):
        before = pool.cache.k.view(torch.uint8).clone()
        o, lse = binding.paged_forward(q, pool.cache, table, lens, cu_seqlens=cu)
        with pytest.raises(binding.AttnError) as err:
            binding.check_status()
        assert err.value.code == binding.ATTN_ERR_ARG
        binding.paged_read(pool.cache, table, lens, 2, cu_seqlens=cu)
        return o, before

    bad = pool.table.clone()
    bad[0, 1] = 1 << 20
    o, _ = reported(bad, pool.lens_t, cu)
    keep = [j for j in range(200) if j // PAGE != 1]   # the keys of a bad page do not count
    k, v = (pool.values(0, i)[keep, 0] for i in (0, 1))
    p = torch.softmax(q[0].cpu().double() @ k.T / 8, -1)
    assert_within(o[0], p @ v, (U + SLACK) * (p @ v.abs()) + U * (p @ v).abs(), "keys of good pages")
    assert_within(o[1], *(lambda p, v: (p @ v, (U + SLACK) * (p @ v.abs()) + U * (p @ v).abs()))(
        torch.softmax(q[1].cpu().double() @ pool.values(1, 0)[:, 0].T / 8, -1), pool.values(1, 1)[:, 0]), "the other sequence")
    reported(pool.table, torch.tensor([-3, 100], dtype=torch.int32).cuda(), cu)
    reported(pool.table, torch.tensor([200, 1 << 30], dtype=torch.int32).cuda(), cu)
    reported(pool.table, pool.lens_t, torch.tensor([0, 1, 9], dtype=torch.int32).cuda())
    # appends into such places write nothing
    bad[0, 3] = -1
    before = [t.clone() for t in (pool.cache.k.view(torch.uint8), pool.cache.v.view(torch.uint8))]
    binding.paged_append(pool.cache, x[:1], x[:1], bad[:1], pool.lens_t[:1], cu_seqlens=offsets([1]).cuda())
    with pytest.raises(binding.AttnError):
        binding.check_status()
    assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(before, (pool.cache.k, pool.cache.v)))


@gpu
def test_pages_past_32_bit_offsets():
    """Rows whose byte offset in the cache passes 2^32."""
    pages = (1 << 32) // (PAGE * 256 * 2) + 40
    cache = binding.PagedCache.empty(pages, 1, 256)
    g = np.random.default_rng(30)
    table = torch.tensor([[pages - 1, 3, pages - 7]], dtype=torch.int32).cuda()
    lens = torch.tensor([150], dtype=torch.int32).cuda()
    k, v, q = bf16(g, 1, 150, 1, 256), bf16(g, 1, 150, 1, 256), bf16(g, 1, 2, 2, 256)
    binding.paged_append(cache, k.cuda(), v.cuda(), table, lens)
    rk, rv = binding.paged_read(cache, table, lens, 150)
    assert torch.equal(rk.cpu(), k) and torch.equal(rv.cpu(), v)
    o, _ = binding.paged_forward(q.cuda(), cache, table, lens)
    binding.check_status()
    want, _ = binding.forward(q.cuda(), rk, rv, causal=True)
    # two bf16 kernels: P and O rounded in each
    p = torch.softmax((q[0].double().transpose(0, 1) @ k[0, :, 0].double().T / 16).masked_fill(~visible(2, 150, True, (-1, -1), 0), -math.inf), -1)
    spread = (p @ v[0, :, 0].double().abs()).transpose(0, 1)
    assert ((o - want)[0].double().cpu().abs() <= 2 * (2 * U + SLACK) * spread).all()


@gpu
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("d,H,Hkv", [(128, 8, 2), (64, 4, 4)])
def test_hybrid_serving_loop(bits, d, H, Hkv):
    """Two layers of a hybrid decoder over prompts and single tokens: exact attention over the paged cache, whose
    prompts attend to what the cache gives back, then linear attention with its state, fed by the first layer's output."""
    lens = [200, 65]
    pool = Pool(bits, [n + 8 for n in lens], Hkv, d, seed=40)
    log_decay = torch.tensor([-0.01 * (h + 1) for h in range(Hkv)]).cuda()
    state = torch.zeros((2, Hkv, d, d), device="cuda")
    pool.lens = [0, 0]
    inputs = []
    for new in (lens, [1, 1], [2, 1], [1, 1]):
        pool.lens = [a + b for a, b in zip(pool.lens, new)]
        pool.lens_t = torch.tensor(pool.lens, dtype=torch.int32).cuda()
        T, cu = sum(new), offsets(new).cuda()
        qkv = bf16(pool.g, T, H + 2 * Hkv, d).cuda()
        q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        binding.paged_append(pool.cache, k, v, pool.table, pool.lens_t, cu_seqlens=cu)
        pool.download()
        o, _ = check_forward(pool, new, H, q=q.cpu(), what=f"{new}")
        if new is lens:   # a prompt may go through the whole-prompt kernel over what the cache holds
            kr, vr = binding.paged_read(pool.cache, pool.table, pool.lens_t, T, cu_seqlens=cu)
            whole, _ = binding.forward(q.contiguous(), kr, vr, causal=True, cu_seqlens=cu)
            assert (whole.float() - o.float()).abs().max() <= 2.0 ** -5 * o.float().abs().max()
        args = (o, k, v, log_decay)
        if T == 2:
            y = binding.linear_step(*args, state)
        else:
            y, state = binding.linear_forward(*args, cu_seqlens=cu, state=state, final_state=True)
        inputs.append((new, o.cpu().double(), k.cpu().double(), v.cpu().double(), y.cpu().double()))
    binding.check_status()
    l = log_decay.cpu().double()
    for b in range(2):   # the linear layer token by token, from the outputs of the first
        S, size = torch.zeros(Hkv, d, d, dtype=torch.float64), torch.zeros(Hkv, d, d, dtype=torch.float64)
        for new, o, k, v, y in inputs:
            at = sum(new[:b])
            for t in range(at, at + new[b]):
                kv = torch.einsum("hd,he->hde", k[t], v[t])
                S, size = torch.exp(l)[:, None, None] * S + kv, torch.exp(l)[:, None, None] * size + kv.abs()
                x = o[t].unflatten(0, (Hkv, -1))
                ref = torch.einsum("hgd,hde->hge", x, S).flatten(0, 1) / math.sqrt(d)
                # scores and states are rounded to bf16: 2^-8 of their sums of absolute values at most
                bound = U * torch.einsum("hgd,hde->hge", x.abs(), size).flatten(0, 1) / math.sqrt(d) * (1 + U) + U * ref.abs()
                assert_within(y[t], ref, bound, f"sequence {b} token {t}")
        assert_within(state[b], S, 2.0 ** -15 * size, f"state {b}")


# ------------------------------------------------------------------ refusals (no GPU)

@pytest.fixture(scope="module")
def lib():
    from exact_attention_blackwell_tma_gb300 import build
    build.build()
    return binding.load()


X = 1 << 20   # an address that is never used: the checks come first


def struct(d=64, dv=64, pages=4, Hkv=2, bits=16, at=X, scales=None):
    return binding._PagedStruct(at, X, scales, scales, pages, Hkv, d, dv, bits)


@pytest.mark.parametrize("bad,code", [(dict(d=96, dv=96), -1), (dict(d=128, dv=64), -1), (dict(pages=0), -1),
                                      (dict(Hkv=0), -1), (dict(at=None), -1), (dict(at=X + 4), -2), (dict(bits=4), -1),
                                      (dict(bits=8), -1), (dict(bits=8, scales=X + 8), -2)])
def test_refuses_caches(lib, bad, code):
    c = struct(**bad)
    assert lib.attn_paged_append(X, X, 512, 512, c, X, 3, X, None, 1, 1, None) == code
    assert lib.attn_paged_read(X, X, c, X, 3, X, None, 1, 1, None) == code
    assert lib.attn_paged_fwd(X, 1024, c, X, 3, X, None, X, X, 1, 4, 1, 0.1, 1, -1, -1, 0, X, 1 << 40, None) == code
    assert binding.last_error()


def test_refuses_arguments(lib):
    c = struct()
    ap = lambda k=X, ks=128, vs=128, table=X, width=3, lens=X, B=1, L=1: lib.attn_paged_append(  # noqa: E731
        k, X, ks, vs, c, table, width, lens, None, B, L, None)
    for kw in (dict(k=None), dict(ks=120), dict(vs=132), dict(table=None), dict(width=0), dict(lens=None), dict(B=-1),
               dict(B=1025), dict(L=-1), dict(B=1000, L=2 ** 31 - 1), dict(width=2 ** 31 - 1), dict(width=2 ** 24), dict(L=2 ** 30)):
        assert ap(**kw) == binding.ATTN_ERR_ARG, kw
    assert ap(k=X + 2) == binding.ATTN_ERR_ALIGN
    assert ap(B=0) == 0 and ap(L=0) == 0
    need = lib.attn_paged_fwd_workspace_size(1, 4, 2, 1, 0, 64, 64)
    assert need > 0 and need % 256 == 0 and lib.attn_paged_fwd_workspace_size(1, 4, 3, 1, 0, 64, 64) == 0

    def fwd(q=X, qs=256, H=4, scale=0.1, wl=-1, wr=-1, sinks=0, ws=X, size=need, o=X, L=1, B=1, width=3):
        return lib.attn_paged_fwd(q, qs, c, X, width, X, None, o, X, B, H, L, scale, 1, wl, wr, sinks, ws, size, None)
    for kw in (dict(q=None), dict(qs=128), dict(qs=260), dict(H=3), dict(H=0), dict(scale=0.0), dict(scale=math.inf),
               dict(scale=math.nan), dict(wl=-2), dict(wr=-5), dict(sinks=-1), dict(o=None), dict(L=2 ** 27, width=2 ** 20)):
        assert fwd(**kw) == binding.ATTN_ERR_ARG, kw
    assert fwd(size=need - 1) == binding.ATTN_ERR_WORKSPACE and fwd(ws=None) == binding.ATTN_ERR_WORKSPACE
    assert fwd(ws=X + 16) == binding.ATTN_ERR_ALIGN and fwd(o=X + 8) == binding.ATTN_ERR_ALIGN
    assert fwd(L=0) == 0 and fwd(B=0) == 0


def test_binding_refuses_caches():
    k = torch.zeros(3, 2, 64, 64, dtype=torch.bfloat16)
    c, e = k.to(torch.float8_e4m3fn), torch.zeros(3, 2, 64, dtype=torch.uint8)
    for args in ((k, k), (k.float(), k.float()), (k, k[:2]), (k, c), (k[:, :, :32], k[:, :, :32]), (c, c), (c, c, e, None),
                 (c, c, e, e[:2]), (c, c, e.int(), e.int()), (k, k, e, e), (c, c, e, e)):   # (the good ones are not on a GPU)
        with pytest.raises(ValueError):
            binding.PagedCache(*args)
