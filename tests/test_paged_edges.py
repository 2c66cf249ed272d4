"""The paged cache in bf16 and 8 bits where its contents are at the ends of their types (bounds: test_paged.py)."""
import math

import numpy as np
import pytest
import torch

from exact_attention_blackwell_tma_gb300 import binding
from _plain import SLACK, U, visible
from test_paged import BITS, DIMS, PAGE, Pool, bf16, offsets

gpu = pytest.mark.gpu


def put_byte(pool, b, which, j, head, byte, channel=None, scale=False):
    """A code (of every channel, or of one) or the scale of token j's row of a head."""
    at = (int(pool.table_host[b][j // PAGE]), head, j % PAGE)
    if scale:
        pool.host[2 * which + 1][at] = byte
    elif channel is None:
        pool.host[2 * which][at] = byte
    else:
        pool.host[2 * which][at][channel] = byte


def check_as_read(pool, new, H, q=None, window=(-1, -1), sinks=0, scale=None):
    """O and LSE are those of what paged_read gives, row by row over the keys a row sees: NaN in the same places, the
    rest within the bounds. Returns O and the mask of its NaN."""
    T, r, at, where = sum(new), H // pool.Hkv, 0, []
    q = bf16(pool.g, T, H, pool.d) if q is None else q
    scale = 1 / math.sqrt(pool.d) if scale is None else scale
    o, lse = binding.paged_forward(q.cuda(), pool.cache, pool.table, pool.lens_t, scale=scale, cu_seqlens=offsets(new).cuda(),
                                   window=window, sinks=sinks)
    read = binding.paged_read(pool.cache, pool.table, pool.lens_t, sum(pool.lens), cu_seqlens=offsets(pool.lens).cuda())
    binding.check_status()
    got, got_lse, key0 = o.double().cpu(), lse.double().cpu(), 0
    for b, n in enumerate(new):
        k, v = (x[key0:key0 + pool.lens[b]].double().cpu().repeat_interleave(r, 1) for x in read)
        ok = visible(n, pool.lens[b], True, window, sinks)
        for i in range(n):
            ks, vs = k[ok[i]], v[ok[i]]
            s = torch.einsum("hd,jhd->hj", q[at + i].double(), ks) * scale
            p = torch.softmax(s, -1)
            ref = torch.einsum("hj,jhd->hd", p, vs)
            spread = torch.einsum("hj,jhd->hd", p, vs.abs())
            bad = torch.isnan(ref)
            where.append(bad)
            assert torch.equal(torch.isnan(got[at + i]), bad), f"sequence {b} row {i}: NaN in other places"
            over = (got[at + i] - ref).abs() - (U + SLACK) * spread - U * ref.abs() - 1e-6
            assert over[~bad].numel() == 0 or over[~bad].max() <= 0, f"sequence {b} row {i}: {over[~bad].max():.3e} past the bound"
            assert torch.equal(torch.isnan(got_lse[:, at + i]), torch.isnan(s).any(-1)), f"sequence {b} row {i}: LSE"
        at += n
        key0 += pool.lens[b]
    return o, torch.stack(where)


# ------------------------------------------------------------------ codes that are NaN

@gpu
@pytest.mark.parametrize("d,dv", DIMS)
@pytest.mark.parametrize("new", [[1, 1], [3, 5], [40, 17]])
def test_nan_codes_are_nan(d, dv, new):
    """The codes 7f and ff, as paged_read has them: in K they make the rows that see the key, in V the channel they stand
    in of the rows that see it. Row blocks of one token, of a warp's rows and of two warps'; pages seen whole and in part."""
    pool = Pool(8, [330, 100], 3, d, dv, seed=40 + d + dv + new[0])
    for b, n in enumerate(pool.lens):
        for _ in range(20):   # V of head 0: anywhere
            put_byte(pool, b, 1, int(pool.g.integers(n)), 0, int(pool.g.choice([127, 255])), int(pool.g.integers(dv)))
        # K of head 1: keys that the last rows alone see; head 2 is clean
        for j in (n - 1, n - max(1, new[b] // 2)):
            put_byte(pool, b, 0, j, 1, int(pool.g.choice([127, 255])), int(pool.g.integers(d)))
    pool.upload()
    _, bad = check_as_read(pool, new, 6)
    assert bad[:, :2].any() and not bad[:, :2].all() and bad[-1, 2:4].all() and not bad[:, 4:].any()
    if new[0] > 1:
        assert not bad[0, 2:4].any()


@gpu
@pytest.mark.parametrize("which", [0, 1])
def test_every_place_of_a_nan_code(which):
    """One code at a time, in every token of a tile and every channel of a head."""
    lens = [33] * 64
    pool = Pool(8, lens, 1, 64, seed=41)
    for turn in range(33):
        pool.host[2 * which] &= 0x7f
        pool.host[2 * which][pool.host[2 * which] == 0x7f] = 0
        for b in range(64):
            put_byte(pool, b, which, (turn + b) % 33, 0, 127 + 128 * (b & 1), b)
        pool.upload()
        q = bf16(pool.g, 64, 1, 64).cuda()
        o, _ = binding.paged_forward(q, pool.cache, pool.table, pool.lens_t, cu_seqlens=offsets([1] * 64).cuda())
        want = torch.eye(64, dtype=torch.bool) if which else torch.ones(64, 64, dtype=torch.bool)
        assert torch.equal(torch.isnan(o[:, 0]).cpu(), want), turn
    binding.check_status()


@gpu
@pytest.mark.parametrize("window,sinks", [((50, -1), 4), ((0, -1), 0), ((200, -1), 70)])
def test_nan_codes_and_windows(window, sinks):
    """Between the sinks and the windows they count as nothing, within either as NaN."""
    pool = Pool(8, [500, 129], 2, 128, seed=42)
    for b, n in enumerate(pool.lens):
        for j in (2, 60, 69, 75, n // 2, n - 60, n - 40, n - 2):
            put_byte(pool, b, 1, j, 0, 127, int(pool.g.integers(128)))
        for j in (60, 75, n // 2, n - 3):
            put_byte(pool, b, 0, j, 1, 255, int(pool.g.integers(128)))
    pool.upload()
    check_as_read(pool, [9, 2], 4, window=window, sinks=sinks)


@gpu
def test_nan_codes_in_a_cache_of_many_blocks():
    """Shares of several thread blocks are joined with them."""
    pool = Pool(8, [30000, 70], 1, 128, seed=43)
    for j in (3, 17000, 29990):
        put_byte(pool, 0, 1, j, 0, 255, j % 128)
    pool.upload()
    _, bad = check_as_read(pool, [2, 1], 4)
    assert bad[0].sum() == 4 * 3 and not bad[2].any()


@gpu
@pytest.mark.parametrize("size", [2.0 ** -110, 2.0 ** 70, 2.0 ** 110])
@pytest.mark.parametrize("bits", BITS)
def test_query_sizes_at_the_ends(bits, size):
    """Rows of very different size in one block; the scale undoes the size."""
    pool = Pool(bits, [300], 1, 64, seed=47)
    q = (bf16(pool.g, 4, 3, 64).float() * size * 2.0 ** torch.arange(-4, 8).reshape(4, 3, 1)).to(torch.bfloat16)
    _, bad = check_as_read(pool, [4], 3, q=q, scale=2.0 ** -9 / size)
    assert not bad.any()


# ------------------------------------------------------------------ small values

@gpu
@pytest.mark.parametrize("e", [1, 4, 8, 16, 25, 40, 60])
@pytest.mark.parametrize("d,N", [(64, 100), (128, 700), (256, 100)])
def test_small_value_scales(e, d, N):
    """V's scales from the least one (2^-126) up: O to its own rounding and P's, as for any other size. What is added is half
    a step of the smallest bf16 (2^-134) for a value's and for O's rounding each, and for the sums, whose weights are 2^-16
    and more and which cannot hold less than 2^-149: 2^-150 / 2^-16 for each of a row's N products."""
    pool = Pool(8, [N], 1, d, seed=46 + e)
    pool.host[3] = torch.tensor(pool.g.integers(e, e + 8, pool.host[3].shape).astype(np.uint8))
    pool.upload()
    q = bf16(pool.g, 2, 4, d)
    o, _ = binding.paged_forward(q.cuda(), pool.cache, pool.table, pool.lens_t, cu_seqlens=offsets([2]).cuda())
    binding.check_status()
    k, v = (pool.values(0, which).repeat_interleave(4, 1) for which in (0, 1))
    s = torch.einsum("ihd,jhd->hij", q.double(), k) / math.sqrt(d)
    p = torch.softmax(s.masked_fill(~visible(2, N, True, (-1, -1), 0), -math.inf), -1)
    ref, spread = torch.einsum("hij,jhd->ihd", p, v), torch.einsum("hij,jhd->ihd", p, v.abs())
    bound = (U + SLACK) * spread + U * ref.abs() + 2.0 ** -133 + N * 2.0 ** -134
    size = v.abs().max()
    over = ((o.double().cpu() - ref).abs() - bound) / size
    assert torch.isfinite(o).all() and over.max() <= 0, f"{over.max():.3e} of the largest value past the bound"


# ------------------------------------------------------------------ rows marked as NaN

@gpu
@pytest.mark.parametrize("d,dv", DIMS)
def test_rows_marked_nan_hold_any_codes(d, dv):
    """A scale of 255 makes a row NaN, whatever its codes are: read back, as keys and as values."""
    pool = Pool(8, [200, 70], 2, d, dv, seed=45)
    for b, n in enumerate(pool.lens):
        for j in (0, n - 1):   # (their codes stay as they are: neither 0 nor NaN)
            put_byte(pool, b, 1, j, 0, 255, scale=True)
        put_byte(pool, b, 0, n - 2, 1, 255, scale=True)
    pool.upload()
    k, v = binding.paged_read(pool.cache, pool.table, pool.lens_t, 270, cu_seqlens=offsets([200, 70]).cuda())
    assert torch.isnan(v[[0, 199, 200, 269], 0]).all() and torch.isnan(k[[198, 268], 1]).all()
    assert torch.isnan(v).sum() == 4 * dv and torch.isnan(k).sum() == 2 * d
    _, bad = check_as_read(pool, [4, 3], 4)
    assert bad[:, :2].all() and not bad[0, 2:].any() and bad[3, 2:].all()


# ------------------------------------------------------------------ keys whose weight is nothing in fp32

@gpu
@pytest.mark.parametrize("bits,how", [(16, "value"), (8, "code"), (8, "scale")])
@pytest.mark.parametrize("N,new,window,light,j", [
    (9000, 1, -1, (0, 4500), 5), (9000, 1, -1, (0, 4500), 4400), (128, 1, -1, (64, 128), 70), (128, 20, -1, (0, 64), 33),
    (9000, 6, 4000, (4990, 8000), 4998), (9000, 6, 4000, (4990, 8000), 6000)])
def test_nan_of_a_key_without_weight(bits, how, N, new, window, light, j):
    """The NaN value of a key whose weight is below 2^-149 reaches the rows that see it, whichever warp or thread block
    the key falls to: 0 times NaN, wherever the sum over the keys is cut."""
    pool = Pool(bits, [N], 1, 64, seed=44)
    tokens = np.arange(N)
    page, slot = pool.table_host[0][tokens // PAGE].astype(np.int64), tokens % PAGE
    few = torch.tensor((tokens >= light[0]) & (tokens < light[1]))[:, None]
    # the light keys score 256 less than the others (b8 is the code of -1)
    pool.host[0][page, 0, slot] = torch.where(few, -32.0, 0.0).to(torch.bfloat16) if bits == 16 else few.to(torch.uint8) * 0xb8
    if bits == 8:
        pool.host[1][:] = 127 + 5
    if how == "value":
        pool.host[2][int(page[j]), 0, j % PAGE, 9] = math.nan
    elif how == "code":
        put_byte(pool, 0, 1, j, 0, 127, 9)
    else:
        put_byte(pool, 0, 1, j, 0, 0)
        put_byte(pool, 0, 1, j, 0, 255, scale=True)
    pool.upload()
    q = torch.ones(new, 2, 64, dtype=torch.bfloat16)
    o, lse = binding.paged_forward(q.cuda(), pool.cache, pool.table, pool.lens_t, scale=1 / 8, cu_seqlens=offsets([new]).cuda(),
                                   window=(window, -1))
    binding.check_status()
    sees = visible(new, N, True, (window, -1), 0)[:, j].cuda()
    assert torch.isnan(o[sees][..., 9]).all() and torch.isfinite(lse).all()
    if bits == 8:   # (a NaN in bf16 reaches the rows beside them, too)
        assert torch.isfinite(o[~sees]).all()
    if how == "scale":
        assert torch.isnan(o[sees]).all()
    elif bits == 8:
        assert torch.isfinite(o[..., :9]).all() and torch.isfinite(o[..., 10:]).all()
