"""Operators of long-context serving and training beside the exact attention, case by case.

Three families, all on the tensors that a user of the framework holds:

  sinks   attention with a sliding window and a few first keys that stay visible
          (prefill and training: forward, and forward + backward);
  kv4     attention of 1 to 16 new tokens per sequence over a paged key/value
          cache held in 4 bits, with the same masks, and optionally the attention
          weight that every cached key collected;
  append  quantise new keys and values into that cache and read rows of it back
          as bf16 (a prefill attends to what the cache will later give);
  evict   keep, per key/value head, the first keys, the latest keys and those with
          the largest accumulated weight, in new pages, and read them back.

The cache: pages of 64 tokens; per page, key/value head and group of 64 channels
a row of 32 bytes per token (channel 2i in the low half of byte i, 2i + 1 in the
high half) and two bf16 parameters per token, scale and minimum: a code c stands
for scale * c + minimum. `own` selects who computes: False, plain torch in 32
bits; True, the framework's calls.
"""
import math
import random

import torch

own = False

PAGE = 64    # tokens of a page
GROUP = 64   # channels that share a scale and a minimum


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the smallest training step: one short sequence of odd length, two heads
        dict(name="sinks_train_b1h2l301d64", kind="sinks", B=1, H=2, Hkv=2, d=64, dv=64, lo=301, hi=301, lens_seed=0,
             packed=False, window=100, sinks=4, grad=True, deterministic=False),
        # the long-context training step: a 1024-key window over 8192 tokens with 4 sinks
        dict(name="sinks_train_b2h16l8192d128", kind="sinks", B=2, H=16, Hkv=16, d=128, dv=128, lo=8192, hi=8192,
             lens_seed=0, packed=False, window=1024, sinks=4, grad=True, deterministic=False),
        # grouped heads with a wider query/key head, ragged sizes, reproducible gradients
        dict(name="sinks_train_b1h8kv2l5001d192", kind="sinks", B=1, H=8, Hkv=2, d=192, dv=128, lo=5001, hi=5001,
             lens_seed=0, packed=False, window=700, sinks=130, grad=True, deterministic=True),
        # prefill of a packed batch of prompts
        dict(name="sinks_prefill_packed8h16kv4d128", kind="sinks", B=8, H=16, Hkv=4, d=128, dv=128, lo=256, hi=4096,
             lens_seed=4, packed=True, window=512, sinks=16, grad=False, deterministic=False),
        # a decode step: one new token of each of 64 sequences enters the cache
        dict(name="append_decode_b64kv4d128", kind="append", B=64, Hkv=4, d=128, dv=128, lo=1024, hi=16384, new_lo=1,
             new_hi=1, read_all=False, lens_seed=6),
        # chunked prefill: chunks of up to 2048 tokens, the whole prefix read back for the chunk's attention
        dict(name="append_prefill_b16kv8d128", kind="append", B=16, Hkv=8, d=128, dv=128, lo=2048, hi=8192, new_lo=100,
             new_hi=2048, read_all=True, lens_seed=7),
        # one user's next token: latency
        dict(name="kv4_decode_b1h16kv4l1000d128", kind="kv4", B=1, H=16, Hkv=4, d=128, dv=128, lo=1000, hi=1000,
             q_lo=1, q_hi=1, lens_seed=0, window=-1, sinks=0, weights=False),
        # 1 to 16 tokens per sequence (decode and speculative steps in one batch) over ragged caches
        dict(name="kv4_mix_b32h16kv4d128", kind="kv4", B=32, H=16, Hkv=4, d=128, dv=128, lo=1024, hi=16384, q_lo=1,
             q_hi=16, lens_seed=6, window=-1, sinks=0, weights=False),
        # a full decode batch that also collects each key's attention weight
        dict(name="kv4_weights_b64h32kv8d128", kind="kv4", B=64, H=32, Hkv=8, d=128, dv=128, lo=4096, hi=16384, q_lo=1,
             q_hi=1, lens_seed=8, window=-1, sinks=0, weights=True),
        # a window with sinks over long caches, wide heads that all share one key/value head
        dict(name="kv4_window_b16h8kv1d256", kind="kv4", B=16, H=8, Hkv=1, d=256, dv=256, lo=10000, hi=65536, q_lo=1,
             q_hi=1, lens_seed=9, window=4096, sinks=4, weights=False),
        # one short cache shrinks to its budget
        dict(name="evict_b1kv4l1500d64", kind="evict", B=1, Hkv=4, d=64, dv=64, lo=1500, hi=1500, budget=512, sinks=4,
             recent=128, lens_seed=0),
        # a serving batch shrinks to a quarter
        dict(name="evict_b16kv8l32768d128", kind="evict", B=16, Hkv=8, d=128, dv=128, lo=20000, hi=32768, budget=8192,
             sinks=4, recent=1024, lens_seed=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["sinks", "sinks", "append", "kv4", "kv4", "kv4", "evict"])
    d, dv = rng.choice([(64, 64), (128, 128), (128, 128), (192, 192), (192, 128), (256, 256)])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4, 8])
    seed = rng.randrange(1 << 20)
    if kind == "sinks":
        B = rng.choice([1, 1, 2, 3, 5])
        # the pairs of all heads stay below the largest listed case's
        most = int(math.sqrt(1.6e9 / (B * H)))
        hi = _log(rng, 1, min(most, 6000))
        packed = rng.random() < 0.4
        return dict(kind=kind, B=B, H=H, Hkv=Hkv, d=d, dv=dv, lo=max(1, hi // 3) if packed else hi, hi=hi,
                    lens_seed=seed, packed=packed, window=rng.choice([0, _log(rng, 1, 2000), _log(rng, 1, 2000)]),
                    sinks=rng.choice([1, 4, _log(rng, 1, 300)]), grad=rng.random() < 0.7,
                    deterministic=rng.random() < 0.3)
    if kind == "append":
        B = _log(rng, 1, 64)
        hi = _log(rng, 8, min(16384, 500000 // (B * Hkv)))
        new = 1 if rng.random() < 0.4 else _log(rng, 1, hi)
        return dict(kind=kind, B=B, Hkv=Hkv, d=d, dv=dv, lo=max(new, hi // 4), hi=hi, new_lo=max(1, new // 5),
                    new_hi=new, read_all=rng.random() < 0.5, lens_seed=seed)
    if kind == "evict":
        B = _log(rng, 1, 16)
        hi = _log(rng, 8, min(65536, 2000000 // (B * Hkv)))
        budget = max(2, int(hi * rng.uniform(0.1, 0.9)))
        return dict(kind=kind, B=B, Hkv=Hkv, d=d, dv=dv, lo=max(1, hi // 3), hi=hi, budget=budget,
                    sinks=min(rng.choice([0, 4, 17]), budget // 2), recent=rng.randrange(budget // 2 + 1),
                    lens_seed=seed)
    B = _log(rng, 1, 64)
    q_hi = rng.choice([1, 1, 1, rng.randrange(2, 17)])
    hi = _log(rng, 20, min(131072, 3000000 // (B * Hkv)))
    window = rng.random() < 0.4
    return dict(kind=kind, B=B, H=H, Hkv=Hkv, d=d, dv=dv, lo=max(q_hi, hi // 5), hi=hi,
                q_lo=1 if rng.random() < 0.5 else q_hi, q_hi=q_hi, lens_seed=seed,
                window=_log(rng, 1, 8192) if window else -1, sinks=rng.choice([0, 4, 70]) if window else 0,
                weights=rng.random() < 0.4)


def _lens(n, lo, hi, seed):
    rng = random.Random(seed)
    return [rng.randint(lo, hi) for _ in range(n)]


def _lengths(case):
    """Keys per sequence."""
    return _lens(case["B"], case["lo"], case["hi"], case["lens_seed"])


def _new(case, lo, hi):
    """New tokens per sequence (never more than its keys)."""
    return [min(a, b) for a, b in zip(_lens(case["B"], case[lo], case[hi], case["lens_seed"] + 1), _lengths(case))]


# ------------------------------------------------------------------------------------------ inputs

def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32).cuda()


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _cache(g, pages, Hkv, d, dv):
    """Codes and parameters as min/max quantisation of normal values gives them: bell-shaped
    codes, a scale near 0.31, a minimum near -2.3."""
    out = []
    for width in (d, dv):
        codes = torch.empty((pages, Hkv, width // GROUP, PAGE, GROUP // 2), dtype=torch.uint8, device="cuda")
        for part in codes.split(max(1, (1 << 26) // max(1, codes[0].numel()))):
            c = torch.randn(part.shape + (2,), generator=g, device="cuda").mul_(3.2).add_(7.5).round_().clamp_(0, 15)
            part.copy_(c[..., 0] + 16 * c[..., 1])
        shape = (pages, Hkv, width // GROUP, PAGE)
        scale = 0.31 * torch.exp(0.15 * torch.randn(shape, generator=g, device="cuda"))
        low = -7.5 * scale + 0.2 * torch.randn(shape, generator=g, device="cuda")
        out += [codes, torch.stack((scale, low), -1).to(torch.bfloat16)]
    return tuple(out)


def _pages(lens):
    return [-(-n // PAGE) for n in lens]


def _table(g, need, first, total):
    """Page table [B, widest]: pages first .. total - 1 in a shuffled order, -1 where a sequence has no page."""
    ids = (torch.randperm(total - first, generator=g, device="cuda") + first).to(torch.int32)
    width, at, rows = max(1, max(need)), 0, []
    for n in need:
        rows.append(torch.cat((ids[at:at + n], torch.full((width - n,), -1, dtype=torch.int32, device="cuda"))))
        at += n
    return torch.stack(rows).contiguous()


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    s = dict(case)
    lens = _lengths(case)
    s["longest"] = max(lens)
    s["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
    B, Hkv, d, dv = case["B"], case["Hkv"], case["d"], case["dv"]
    if case["kind"] == "sinks":
        H = case["H"]
        rows = (sum(lens),) if case["packed"] else (B, case["hi"])
        s["cu"] = _offsets(lens) if case["packed"] else None
        s["q"], s["k"] = _randn(g, *rows, H, d), _randn(g, *rows, Hkv, d)
        s["v"], s["do"] = _randn(g, *rows, Hkv, dv), _randn(g, *rows, H, dv)
        return s
    need = _pages(lens)
    spare = _pages([case["budget"]] * B) if case["kind"] == "evict" else []
    total = sum(need) + sum(spare)
    s["cache"] = _cache(g, total, Hkv, d, dv)
    s["table"] = _table(g, need, 0, sum(need))
    if case["kind"] == "append":
        new = _new(case, "new_lo", "new_hi")
        s["cu"], s["longest_new"] = _offsets(new), max(new)
        s["k"], s["v"] = _randn(g, sum(new), Hkv, d), _randn(g, sum(new), Hkv, dv)
        # channels of a trained model's keys differ in size: some are several times the others
        s["k"] *= (1 + 4 * (torch.rand((Hkv, d), generator=g, device="cuda") > 0.95)).to(torch.bfloat16)
        s["cu_read"] = _offsets(lens) if case["read_all"] else s["cu"]
        s["read"] = sum(lens) if case["read_all"] else sum(new)
    elif case["kind"] == "kv4":
        new = _new(case, "q_lo", "q_hi")
        s["cu"], s["longest_new"] = _offsets(new), max(new)
        s["q"] = _randn(g, sum(new), case["H"], d)
        s["key_weights"] = None
        if case["weights"]:
            s["key_weights"] = torch.zeros((B, Hkv, s["table"].shape[1] * PAGE), device="cuda")
    else:
        s["new_table"] = _table(g, spare, sum(need), total)
        # accumulated weights: a few keys hold most of it
        w = torch.rand((B, Hkv, s["table"].shape[1] * PAGE), generator=g, device="cuda")
        s["key_weights"] = w.pow_(8).mul_(3.0)
        kept = [min(n, case["budget"]) for n in lens]
        s["cu_read"], s["read"] = _offsets(kept), sum(kept)
    return s


# ------------------------------------------------------------------------------------------ plain forms

def _padded(x, cu, longest):
    """Packed rows [T, ...] as [B, longest, ...]; places past a sequence's end hold some other row of the batch."""
    at = cu[:-1, None].long() + torch.arange(longest, device=x.device)
    return x[at.clamp(max=x.shape[0] - 1)]


def _packed(x, cu, total):
    """The inverse: [B, longest, ...] to [total, ...]."""
    row = torch.arange(total, device=x.device)
    seq = (row[:, None] >= cu[None, 1:].long()).sum(1)
    return x[seq, row - cu[seq].long()]


def _visible(nq, nk, lens_q, lens_k, window, sinks, device):
    """[B, nq, nk]: causal (aligned at the end), within the window or among the first keys."""
    i = torch.arange(nq, device=device)[None, :, None] + (lens_k - lens_q)[:, None, None]
    j = torch.arange(nk, device=device)[None, None, :]
    ok = (j <= i) & (j < lens_k[:, None, None])
    if window >= 0:
        ok &= (j >= i - window) | (j < sinks)
    return ok


def _plain_sinks(s):
    packed = s["packed"]
    q, k, v, do = ((_padded(s[n], s["cu"], s["longest"]) if packed else s[n]).float() for n in ("q", "k", "v", "do"))
    B, L, H, d = q.shape
    Hkv, group, scale = s["Hkv"], H // s["Hkv"], 1.0 / math.sqrt(d)
    q = q.permute(0, 2, 1, 3).reshape(B, Hkv, group, L, d)
    do = do.permute(0, 2, 1, 3).reshape(B, Hkv, group, L, -1)
    k, v = k.permute(0, 2, 1, 3)[:, :, None], v.permute(0, 2, 1, 3)[:, :, None]
    lens = s["lens"].long()
    ok = _visible(L, L, lens, lens, s["window"], s["sinks"], q.device)[:, None, None]
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(~ok, -math.inf)
    top = x.amax(-1, keepdim=True).clamp_(min=-1e30)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1).reshape(B, H, L)
    p /= total.clamp(min=1e-30)
    o = torch.matmul(p, v)

    def rows(x, heads):   # [B, heads.., L, width] to the layout of the inputs
        x = x.reshape(B, heads, L, -1).permute(0, 2, 1, 3).to(torch.bfloat16)
        return _packed(x, s["cu"], s["q"].shape[0]) if packed else x.contiguous()

    out = {"o": rows(o, H), "lse": _packed(lse.transpose(1, 2), s["cu"], s["q"].shape[0]).t() if packed else lse}
    if s["grad"]:
        if packed:   # rows past a sequence's end take no part
            do = do * (torch.arange(L, device=q.device) < lens[:, None])[:, None, None, :, None]
        dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
        ds = torch.matmul(do, v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        out["dq"] = rows(torch.matmul(ds, k), H)
        out["dk"] = rows(torch.matmul(ds.transpose(-1, -2), q).sum(2), Hkv)
        out["dv"] = rows(dv, Hkv)
    return out


def _plain_values(codes, params, table):
    """fp32 [B, Hkv, keys, channels] of the pages in a table (a place without a page: any page)."""
    at = table.long().clamp(min=0)
    c, p = codes[at], params[at].float()
    c = torch.stack((c & 15, c >> 4), -1).flatten(-2).float()
    x = c.mul_(p[..., :1]).add_(p[..., 1:])   # [B, pages, Hkv, groups, 64 tokens, 64 channels]
    return x.permute(0, 2, 1, 4, 3, 5).flatten(4, 5).flatten(2, 3)


def _plain_append(s, codes, params, x):
    """Quantises x [T, Hkv, width] into the pages: row t of a sequence with n new rows is key lens - n + t."""
    cu, T = s["cu"].long(), x.shape[0]
    row = torch.arange(T, device=x.device)
    seq = (row[:, None] >= cu[None, 1:]).sum(1)
    slot = s["lens"].long()[seq] - (cu[1:] - cu[:-1])[seq] + row - cu[seq]
    page = s["table"].long()[seq, slot // PAGE]
    x = x.reshape(T, x.shape[1], -1, GROUP).double()   # values next to a border between two codes are decided in 64 bits
    low = x.amin(-1, keepdim=True)
    scale = ((x.amax(-1, keepdim=True) - low) / 15).to(torch.bfloat16).double()
    c = torch.where(scale > 0, (x - low) / scale, 0.0).round_().clamp_(0, 15).to(torch.uint8)
    codes[page, :, :, slot % PAGE] = c[..., 0::2] | (c[..., 1::2] << 4)
    params[page, :, :, slot % PAGE] = torch.cat((scale, low), -1).to(torch.bfloat16)


def _plain_read(codes, params, table, lens, cu, total):
    """bf16 [total, Hkv, width]: the last cu[b + 1] - cu[b] keys of each sequence's cache."""
    cu = cu.long()
    row = torch.arange(total, device=codes.device)
    seq = (row[:, None] >= cu[None, 1:]).sum(1)
    slot = lens.long()[seq] - (cu[1:] - cu[:-1])[seq] + row - cu[seq]
    page = table.long()[seq, slot // PAGE]
    c, p = codes[page, :, :, slot % PAGE], params[page, :, :, slot % PAGE].float()
    c = torch.stack((c & 15, c >> 4), -1).flatten(-2).float()
    return (c * p[..., :1] + p[..., 1:]).flatten(2, 3).to(torch.bfloat16)


def _plain_kv4(s):
    kc, kp, vc, vp = s["cache"]
    k, v = _plain_values(kc, kp, s["table"]), _plain_values(vc, vp, s["table"])
    B, Hkv, N, d = k.shape
    H, cu, lens = s["H"], s["cu"], s["lens"].long()
    group, n = H // Hkv, s["longest_new"]
    new = (cu[1:] - cu[:-1]).long()
    q = _padded(s["q"], cu, n).float().reshape(B, n, Hkv, group, d).permute(0, 2, 3, 1, 4)
    ok = _visible(n, N, new, lens, s["window"], s["sinks"], q.device)
    ok &= (torch.arange(n, device=q.device)[None, :] < new[:, None])[:, :, None]
    x = torch.matmul(q.reshape(B, Hkv, group * n, d), k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    x = x.reshape(B, Hkv, group, n, N).masked_fill_(~ok[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp_(min=-1e30)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p /= total.clamp(min=1e-30)
    v = v.masked_fill((torch.arange(N, device=q.device) >= lens[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(p.reshape(B, Hkv, group * n, N), v).reshape(B, H, n, -1)
    lse = (top + total.log()).reshape(B, H, n)
    T = s["q"].shape[0]
    out = {"o": _packed(o.transpose(1, 2), cu, T).to(torch.bfloat16), "lse": _packed(lse.transpose(1, 2), cu, T).t()}
    if s["weights"]:
        held = (torch.arange(N, device=q.device) < lens[:, None])[:, None]
        s["key_weights"].copy_(torch.where(held, p.sum((2, 3)), s["key_weights"]))
        out["key_weights"] = s["key_weights"]
    return out


def _plain_evict(s):
    lens, budget, w = s["lens"].long(), s["budget"], s["key_weights"]
    B, Hkv, N = w.shape
    j = torch.arange(N, device=w.device)
    held = (j < lens[:, None])[:, None]
    always = (j < s["sinks"]) | (j >= (lens - s["recent"])[:, None])[:, None]
    rank = torch.where(held, torch.where(always, math.inf, w), -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices   # equal weights: the earlier key first
    new_lens = lens.clamp(max=budget)
    order = order[..., :budget] if N >= budget else torch.cat((order, order[..., :1].expand(B, Hkv, budget - N)), -1)
    empty = (torch.arange(budget, device=w.device) >= new_lens[:, None])[:, None].expand(B, Hkv, budget)
    kept = order.masked_fill(empty, N).sort(-1).values   # the keys' order stays
    safe = kept.clamp(max=N - 1)
    page = s["table"].long().clamp(min=0)[:, None].expand(B, Hkv, -1).gather(2, safe // PAGE)
    at = torch.arange(budget, device=w.device)
    new_page = s["new_table"].long().gather(1, (at // PAGE).expand(B, budget))[:, None].expand(B, Hkv, budget)
    head = torch.arange(Hkv, device=w.device)[None, :, None].expand(B, Hkv, budget)
    spot = (at % PAGE).expand(B, Hkv, budget)
    go = ~empty
    for part in s["cache"]:
        part[new_page[go], head[go], :, spot[go]] = part[page[go], head[go], :, (safe % PAGE)[go]]
    new_weights = w.gather(2, safe).masked_fill(empty, 0.0)
    return new_lens.int(), kept.masked_fill(empty, -1).int(), new_weights


# ------------------------------------------------------------------------------------------ one pass

def run(s):
    kind = s["kind"]
    if own:
        from exact_attention_blackwell_tma_gb300 import binding
    if kind == "sinks":
        if own:
            window = (s["window"], -1)
            o, lse = binding.forward(s["q"], s["k"], s["v"], causal=True, cu_seqlens=s["cu"], window=window,
                                     sinks=s["sinks"])
            out = {"o": o, "lse": lse}
            if s["grad"]:
                out["dq"], out["dk"], out["dv"] = binding.backward(
                    s["q"], s["k"], s["v"], o, lse, s["do"], causal=True, cu_seqlens=s["cu"], window=window,
                    sinks=s["sinks"], deterministic=s["deterministic"])
            return out
        return _plain_sinks(s)
    if kind == "append":
        kc, kp, vc, vp = s["cache"]
        if own:
            cache = binding.Kv4Cache(kc, kp, vc, vp)
            binding.kv4_append(cache, s["k"], s["v"], s["table"], s["lens"], cu_seqlens=s["cu"])
            k, v = binding.kv4_read(cache, s["table"], s["lens"], s["read"], cu_seqlens=s["cu_read"])
        else:
            _plain_append(s, kc, kp, s["k"])
            _plain_append(s, vc, vp, s["v"])
            k = _plain_read(kc, kp, s["table"], s["lens"], s["cu_read"], s["read"])
            v = _plain_read(vc, vp, s["table"], s["lens"], s["cu_read"], s["read"])
        return {"k": k, "v": v}
    if kind == "kv4":
        if own:
            o, lse = binding.kv4_forward(s["q"], binding.Kv4Cache(*s["cache"]), s["table"], s["lens"], causal=True,
                                         cu_seqlens=s["cu"], window=(s["window"], -1), sinks=s["sinks"],
                                         key_weights=s["key_weights"], weight_decay=0.0)
            out = {"o": o, "lse": lse}
            if s["weights"]:
                out["key_weights"] = s["key_weights"]
            return out
        return _plain_kv4(s)
    if own:
        cache = binding.Kv4Cache(*s["cache"])
        lens, kept, weights = binding.kv4_evict(cache, s["table"], s["lens"], s["key_weights"], s["new_table"],
                                                budget=s["budget"], sinks=s["sinks"], recent=s["recent"])
        k, v = binding.kv4_read(cache, s["new_table"], lens, s["read"], cu_seqlens=s["cu_read"])
    else:
        kc, kp, vc, vp = s["cache"]
        lens, kept, weights = _plain_evict(s)
        k = _plain_read(kc, kp, s["new_table"], lens, s["cu_read"], s["read"])
        v = _plain_read(vc, vp, s["new_table"], lens, s["cu_read"], s["read"])
    return {"lens": lens, "kept": kept, "key_weights": weights, "k": k, "v": v}


# ------------------------------------------------------------------------------------------ what a pass cannot do without

def _seen(nq, nk, window, sinks):
    """(visible pairs, keys that some query sees) of the last nq queries of nk keys, causal."""
    pairs, lo = 0, nk
    for i in range(nk - nq, nk):
        first = max(0, i - window) if window >= 0 else 0
        pairs += i + 1 - first + min(sinks, first)
        lo = min(lo, first)
    return pairs, nk - lo + min(sinks, lo)


def work(case):
    lens = _lengths(case)
    Hkv, d, dv = case["Hkv"], case["d"], case["dv"]
    row = (d + dv) // 2 + (d + dv) // GROUP * 4   # bytes of one key and value of one head in the cache
    if case["kind"] == "sinks":
        pairs = case["H"] * sum(_seen(n, n, case["window"], case["sinks"])[0] for n in lens)
        T = sum(lens)
        size = 2 * T * (case["H"] * (d + dv) + Hkv * (d + dv)) + 4 * T * case["H"]
        flops = 2 * (d + dv) * pairs
        if case["grad"]:
            size += 2 * T * (case["H"] * (d + dv) + Hkv * (d + dv))
            flops += 2 * (3 * d + 2 * dv) * pairs
        return {"bytes": size, "flops": flops}
    if case["kind"] == "append":
        new = sum(_new(case, "new_lo", "new_hi"))
        read = sum(lens) if case["read_all"] else new
        return {"bytes": Hkv * (new * (2 * (d + dv) + row) + (read - new) * row + read * 2 * (d + dv)), "flops": 0}
    if case["kind"] == "kv4":
        new = _new(case, "q_lo", "q_hi")
        seen = [_seen(a, n, case["window"], case["sinks"]) for a, n in zip(new, lens)]
        size = Hkv * row * sum(x[1] for x in seen) + sum(new) * case["H"] * (2 * (d + dv) + 4)
        if case["weights"]:
            size += 4 * Hkv * sum(lens)
        return {"bytes": size, "flops": 2 * (d + dv) * case["H"] * sum(x[0] for x in seen)}
    kept = sum(min(n, case["budget"]) for n in lens)
    size = Hkv * (4 * sum(lens) + kept * (2 * row + 2 * (d + dv) + 4) + 4 * case["budget"] * case["B"])
    return {"bytes": size, "flops": 0}


# ------------------------------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    lens, Hkv, d = _lengths(case), case["Hkv"], case["d"]

    def rows_of(part, params, b, keys, head):   # keys of one head of sequence b, as the values they stand for
        page = s["table"][b].long()[keys // PAGE]
        c, p = part[page, head, :, keys % PAGE].to(torch.int64), params[page, head, :, keys % PAGE].double()
        out = torch.empty(c.shape[:-1] + (GROUP,), dtype=torch.float64, device="cuda")
        out[..., 0::2], out[..., 1::2] = (c % 16).double(), (c // 16).double()
        return (p[..., 1:] + out * p[..., :1]).reshape(keys.numel(), -1)

    if case["kind"] == "sinks":
        H, T = case["H"], sum(lens)
        if 2 * (5 * d + 4 * case["dv"]) * H * sum(n * n for n in lens) > 5e12:
            return None
        flat = {n: s[n].reshape(T, -1, s[n].shape[-1]).double() for n in ("q", "k", "v", "do")}
        o, lse = torch.zeros_like(flat["do"]), torch.zeros((H, T), dtype=torch.float64, device="cuda")
        dq, dk, dv = (torch.zeros_like(flat[n]) for n in ("q", "k", "v"))
        at = 0
        for n in lens:
            place = torch.arange(n, device="cuda")
            gap = place[:, None] - place[None, :]
            keep = (gap >= 0) & ((gap <= case["window"]) | (place[None, :] < case["sinks"]))
            for h in range(H):
                kv = h // (H // Hkv)
                q, k, v = (flat[m][at:at + n, x].detach().requires_grad_(case["grad"])
                           for m, x in (("q", h), ("k", kv), ("v", kv)))
                score = torch.where(keep, q @ k.T / math.sqrt(d), -math.inf)
                got = torch.softmax(score, -1) @ v
                o[at:at + n, h], lse[h, at:at + n] = got.detach(), torch.logsumexp(score.detach(), -1)
                if case["grad"]:
                    a, b, c = torch.autograd.grad(got, (q, k, v), flat["do"][at:at + n, h])
                    dq[at:at + n, h] = a
                    dk[at:at + n, kv] += b
                    dv[at:at + n, kv] += c
            at += n
        out = {"o": o.reshape(s["do"].shape),
               "lse": lse if case["packed"] else lse.reshape(H, case["B"], -1).transpose(0, 1).contiguous()}
        if case["grad"]:
            out.update({"dq": dq.reshape(s["q"].shape), "dk": dk.reshape(s["k"].shape), "dv": dv.reshape(s["v"].shape)})
        return out
    if case["kind"] == "append":
        new = _new(case, "new_lo", "new_hi")
        out = {}
        for i, name in enumerate(("k", "v")):
            part, params = s["cache"][2 * i], s["cache"][2 * i + 1]
            got, at = [], 0
            for b, (n, total) in enumerate(zip(new, lens)):
                if case["read_all"] and total > n:
                    keys = torch.arange(total - n, device="cuda")
                    got.append(torch.stack([rows_of(part, params, b, keys, h) for h in range(Hkv)], 1))
                x = s[name][at:at + n].double().reshape(n, Hkv, -1, GROUP)
                at += n
                low, high = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
                scale = ((high - low) / 15.0).to(torch.bfloat16).double()
                code = torch.floor((x - low) / torch.where(scale > 0, scale, 1.0) + 0.5)
                tie = code - 0.5 == (x - low) / torch.where(scale > 0, scale, 1.0)   # a tie: the even code
                code = torch.where(tie & (code % 2 == 1), code - 1, code).clamp(0, 15)
                got.append((low + scale * code).reshape(n, Hkv, -1))
            out[name] = torch.cat(got)
        return out
    if case["kind"] == "kv4":
        H, new = case["H"], _new(case, "q_lo", "q_hi")
        group, T = H // Hkv, sum(new)
        o = torch.zeros((T, H, case["dv"]), dtype=torch.float64, device="cuda")
        lse = torch.zeros((H, T), dtype=torch.float64, device="cuda")
        weights = torch.zeros((case["B"], Hkv, s["table"].shape[1] * PAGE), dtype=torch.float64, device="cuda")
        at = 0
        for b, (n, total) in enumerate(zip(new, lens)):
            keys = torch.arange(total, device="cuda")
            gap = torch.arange(total - n, total, device="cuda")[:, None] - keys[None, :]
            keep = gap >= 0
            if case["window"] >= 0:
                keep &= (gap <= case["window"]) | (keys < case["sinks"])[None, :]
            for h in range(Hkv):
                k, v = (rows_of(s["cache"][2 * i], s["cache"][2 * i + 1], b, keys, h) for i in (0, 1))
                q = s["q"][at:at + n, h * group:(h + 1) * group].double().transpose(0, 1)
                score = torch.where(keep, q @ k.T / math.sqrt(d), -math.inf)
                p = torch.softmax(score, -1)
                o[at:at + n, h * group:(h + 1) * group] = (p @ v).transpose(0, 1)
                lse[h * group:(h + 1) * group, at:at + n] = torch.logsumexp(score, -1)
                weights[b, h, :total] = p.sum((0, 1))
            at += n
        return {"o": o, "lse": lse, "key_weights": weights} if case["weights"] else {"o": o, "lse": lse}
    budget, w = case["budget"], s["key_weights"].double().cpu()
    kept = torch.full((case["B"], Hkv, budget), -1, dtype=torch.int64)
    k, v = [], []
    for b, n in enumerate(lens):
        m = min(n, budget)
        tail = max(0, n - case["recent"])
        per_head = []
        for h in range(Hkv):
            chosen = set(range(min(case["sinks"], n))) | set(range(tail, n))
            if n <= budget:
                chosen = set(range(n))
            row = w[b, h].tolist()
            middle = sorted(range(min(case["sinks"], n), tail), key=lambda j: (-row[j], j))
            chosen |= set(middle[:m - len(chosen)])
            kept[b, h, :m] = torch.tensor(sorted(chosen))
            per_head.append(kept[b, h, :m].cuda())
        k.append(torch.stack([rows_of(s["cache"][0], s["cache"][1], b, x, h) for h, x in enumerate(per_head)], 1))
        v.append(torch.stack([rows_of(s["cache"][2], s["cache"][3], b, x, h) for h, x in enumerate(per_head)], 1))
    new_weights = torch.where(kept >= 0, w.gather(2, kept.clamp(min=0)), 0.0)
    return {"lens": torch.tensor([min(n, budget) for n in lens], dtype=torch.int32), "kept": kept.int(),
            "key_weights": new_weights, "k": torch.cat(k), "v": torch.cat(v)}
