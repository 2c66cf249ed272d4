"""What the layers of a hybrid decoder need beside whole-prompt attention, case by case.

Some layers of such a model are exact attention, whose keys and values lie in a
paged cache while it serves; the others are linear attention with a decay for each
head, which keeps one matrix per head instead. Four families:

  lin     linear attention over whole sequences, o_t = scale * q_t^T S_t with
          S_t = decay * S_(t-1) + k_t v_t^T: the forward with states in and out
          (prompts), and forward + backward (training);
  step    the same for one new token per sequence, the states updated in place;
  write   new keys and values enter the paged cache, in bf16 or quantised to
          8 bits, and rows of it are read back as bf16;
  decode  attention of 1 to 16 new tokens per sequence over that cache.

The cache: pages of 64 tokens, [pages, heads, 64, channels] in bf16 or e4m3. With
e4m3 a byte e per token and head stands for a scale of 2^(e - 127), the least from
2^-126 up with which the row's largest value stays within 448. `own` selects who computes:
False, plain torch in 32 bits; True, the framework's calls.
"""
import math
import random

import torch

own = False

PAGE = 64     # tokens of a page
CHUNK = 128   # tokens that the plain form of linear attention takes at once


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the smallest training step: one short sequence of odd length, two heads
        dict(name="lin_train_b1h2l301d64", kind="lin", B=1, H=2, Hkv=2, d=64, dv=64, lo=301, hi=301, lens_seed=0,
             packed=False, grad=True, states=False),
        # the training step of a long-context model
        dict(name="lin_train_b2h16l8192d128", kind="lin", B=2, H=16, Hkv=16, d=128, dv=128, lo=8192, hi=8192,
             lens_seed=0, packed=False, grad=True, states=False),
        # packed documents that continue from earlier states and pass gradients to them, grouped heads
        dict(name="lin_train_packed6h8kv2d192", kind="lin", B=6, H=8, Hkv=2, d=192, dv=128, lo=300, hi=5000,
             lens_seed=3, packed=True, grad=True, states=True),
        # one user's chunk of a prompt: latency
        dict(name="lin_prompt_b1h8l777d128", kind="lin", B=1, H=8, Hkv=8, d=128, dv=128, lo=777, hi=777,
             lens_seed=0, packed=False, grad=False, states=True),
        # a serving batch of prompts, packed
        dict(name="lin_prompt_packed16h16d128", kind="lin", B=16, H=16, Hkv=16, d=128, dv=128, lo=256, hi=8192,
             lens_seed=4, packed=True, grad=False, states=True),
        # one user's next token
        dict(name="step_b1h16d128", kind="step", B=1, H=16, Hkv=16, d=128, dv=128),
        # a full decode batch, grouped heads
        dict(name="step_b128h32kv16d128", kind="step", B=128, H=32, Hkv=16, d=128, dv=128),
        # a decode step: one new token of each of 64 sequences enters the 8-bit cache
        dict(name="write_decode_b64kv4d128_8", kind="write", B=64, Hkv=4, d=128, dv=128, lo=1024, hi=16384, new_lo=1,
             new_hi=1, read_all=False, lens_seed=6, bits=8),
        # chunked prefill into an 8-bit cache, the whole prefix read back for the chunk's attention
        dict(name="write_prompt_b16kv8d128_8", kind="write", B=16, Hkv=8, d=128, dv=128, lo=2048, hi=8192, new_lo=100,
             new_hi=2048, read_all=True, lens_seed=7, bits=8),
        # one user's next token over a bf16 cache
        dict(name="decode_b1h16kv4l1000d128_16", kind="decode", B=1, H=16, Hkv=4, d=128, dv=128, lo=1000, hi=1000,
             q_lo=1, q_hi=1, lens_seed=0, window=-1, sinks=0, bits=16),
        # 1 to 16 tokens per sequence (decode and speculative steps in one batch) over ragged bf16 caches
        dict(name="decode_mix_b32h16kv4d128_16", kind="decode", B=32, H=16, Hkv=4, d=128, dv=128, lo=1024, hi=16384,
             q_lo=1, q_hi=16, lens_seed=6, window=-1, sinks=0, bits=16),
        # a full decode batch over 8-bit caches
        dict(name="decode_b64h32kv8d128_8", kind="decode", B=64, H=32, Hkv=8, d=128, dv=128, lo=4096, hi=16384,
             q_lo=1, q_hi=1, lens_seed=8, window=-1, sinks=0, bits=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    kind = rng.choice(["lin", "lin", "lin", "step", "write", "decode", "decode", "decode"])
    d, dv = rng.choice([(64, 64), (128, 128), (128, 128), (192, 192), (192, 128), (256, 256)])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 1, 2, 3, 4])
    seed = rng.randrange(1 << 20)
    if kind == "lin":
        B = rng.choice([1, 1, 2, 3, 5, 16])
        # states and tokens of all heads stay below the largest listed case's
        hi = _log(rng, 1, min(16384, (1 << 31) // (B * H * d * dv)))
        packed = rng.random() < 0.5
        return dict(kind=kind, B=B, H=H, Hkv=Hkv, d=d, dv=dv, lo=max(1, hi // 4) if packed else hi, hi=hi,
                    lens_seed=seed, packed=packed, grad=rng.random() < 0.5, states=rng.random() < 0.5)
    if kind == "step":
        return dict(kind=kind, B=_log(rng, 1, (1 << 25) // (Hkv * d * dv)), H=H, Hkv=Hkv, d=d, dv=dv)
    if kind == "write":
        B = _log(rng, 1, 64)
        hi = _log(rng, 8, min(16384, 500000 // (B * Hkv)))
        new = 1 if rng.random() < 0.4 else _log(rng, 1, hi)
        return dict(kind=kind, B=B, Hkv=Hkv, d=d, dv=dv, lo=max(new, hi // 4), hi=hi, new_lo=max(1, new // 5),
                    new_hi=new, read_all=rng.random() < 0.5, lens_seed=seed, bits=rng.choice([8, 8, 16]))
    B = _log(rng, 1, 64)
    q_hi = rng.choice([1, 1, 1, rng.randrange(2, 17)])
    hi = _log(rng, 20, min(131072, 2000000 // (B * Hkv)))
    window = rng.random() < 0.4
    return dict(kind=kind, B=B, H=H, Hkv=Hkv, d=d, dv=dv, lo=max(q_hi, hi // 5), hi=hi,
                q_lo=1 if rng.random() < 0.5 else q_hi, q_hi=q_hi, lens_seed=seed,
                window=_log(rng, 1, 8192) if window else -1, sinks=rng.choice([0, 4, 70]) if window else 0,
                bits=rng.choice([8, 16]))


def _lens(n, lo, hi, seed):
    rng = random.Random(seed)
    return [rng.randint(lo, hi) for _ in range(n)]


def _lengths(case):
    """Tokens per sequence."""
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


def _states(g, case, size):
    return torch.randn((case["B"], case["Hkv"], case["d"], case["dv"]), generator=g, device="cuda").mul_(size)


def _decays(Hkv):
    """A decay per head, spread from the slowest (memory of some 250 tokens) to the fastest (under two)."""
    return torch.tensor([-2.0 ** (-8.0 * (h + 1) / Hkv) for h in range(Hkv)]).cuda()


def _fused(g, T, heads):
    """Tensors [T, heads, width] side by side in the rows of one projection."""
    x = _randn(g, T, sum(h * w for h, w in heads))
    out, at = [], 0
    for h, w in heads:
        out.append(x[:, at:at + h * w].unflatten(1, (h, w)))
        at += h * w
    return out


def _cache(g, pages, Hkv, d, dv, bits):
    """Keys and values as a served model left them: normal values, in bf16 or as 8-bit codes with their scales' exponents."""
    out = []
    for width in (d, dv):
        if bits == 16:
            rows = torch.empty((pages, Hkv, PAGE, width), dtype=torch.bfloat16, device="cuda")
            size, scales = 1.0, None
        else:
            rows = torch.empty((pages, Hkv, PAGE, width), dtype=torch.float8_e4m3fn, device="cuda")
            size = 110.0   # the largest of a row's 64 to 256 values lies near 320
            scales = torch.randint(118, 121, (pages, Hkv, PAGE), generator=g, device="cuda", dtype=torch.uint8)
        for part in rows.split(max(1, (1 << 27) // max(1, rows[0].numel()))):
            part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(size).clamp_(-4 * size, 4 * size))
        out += [rows, scales]
    return tuple(out)   # k, its scales, v, its scales


def _pages(lens):
    return [-(-n // PAGE) for n in lens]


def _table(g, need):
    """Page table [B, widest]: the pages in a shuffled order, -1 where a sequence has no page."""
    ids = torch.randperm(sum(need), generator=g, device="cuda").to(torch.int32)
    width, at, rows = max(1, max(need)), 0, []
    for n in need:
        rows.append(torch.cat((ids[at:at + n], torch.full((width - n,), -1, dtype=torch.int32, device="cuda"))))
        at += n
    return torch.stack(rows).contiguous()


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    s = dict(case)
    B, Hkv, d, dv = case["B"], case["Hkv"], case["d"], case["dv"]
    if case["kind"] == "step":
        s["q"], s["k"], s["v"] = _fused(g, B, ((case["H"], d), (Hkv, d), (Hkv, dv)))
        s["log_decay"], s["state"] = _decays(Hkv), _states(g, case, 3.0)
        return s
    lens = _lengths(case)
    s["longest"] = max(lens)
    s["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
    if case["kind"] == "lin":
        H = case["H"]
        rows = (sum(lens),) if case["packed"] else (B, case["hi"])
        s["cu"] = _offsets(lens) if case["packed"] else None
        s["q"], s["k"], s["v"] = _randn(g, *rows, H, d), _randn(g, *rows, Hkv, d), _randn(g, *rows, Hkv, dv)
        s["log_decay"] = _decays(Hkv)
        s["state"] = _states(g, case, 3.0) if case["states"] else None
        if case["grad"]:
            s["do"] = _randn(g, *rows, H, dv)
            s["dstate"] = _states(g, case, 1.0) if case["states"] else None
        return s
    need = _pages(lens)
    s["cache"] = _cache(g, sum(need), Hkv, d, dv, case["bits"])
    s["table"] = _table(g, need)
    if case["kind"] == "write":
        new = _new(case, "new_lo", "new_hi")
        s["cu"] = _offsets(new)
        s["k"], s["v"] = _fused(g, sum(new), ((Hkv, d), (Hkv, dv)))
        # channels of a trained model's keys differ in size: some are several times the others
        s["k"] *= (1 + 4 * (torch.rand((Hkv, d), generator=g, device="cuda") > 0.95)).to(torch.bfloat16)
        s["cu_read"] = _offsets(lens) if case["read_all"] else s["cu"]
        s["read"] = sum(lens) if case["read_all"] else sum(new)
    else:
        new = _new(case, "q_lo", "q_hi")
        s["cu"], s["longest_new"] = _offsets(new), max(new)
        s["q"] = _randn(g, sum(new), case["H"], d)
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


def _plain_lin(s):
    B, H, Hkv, d, dv, L, grad = s["B"], s["H"], s["Hkv"], s["d"], s["dv"], s["longest"], s["grad"]
    packed, group, scale = s["packed"], H // Hkv, 1.0 / math.sqrt(d)
    held = torch.arange(L, device="cuda") < s["lens"][:, None]   # [B, L]

    def heads(x):   # [B, Hkv, group (1 for keys and values), L, width], zero past a sequence's end
        x = (_padded(x, s["cu"], L) if packed else x).float() * held[:, :, None, None]
        return x.unflatten(2, (Hkv, -1)).permute(0, 2, 3, 1, 4)

    q, k, v = heads(s["q"]), heads(s["k"]), heads(s["v"])
    do = heads(s["do"]) if grad else None
    l = s["log_decay"].double()[:, None] * held[:, None].double()   # [B, Hkv, L]: a padded place changes no state
    state = torch.zeros((B, Hkv, d, dv), device="cuda") if s["state"] is None else s["state"]
    o = torch.empty((B, Hkv, group, L, dv), device="cuda")
    if grad:
        dq, dk, dvv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    starts = list(range(0, L, CHUNK))
    decays = []
    for c in starts:   # forward in time
        e = min(L, c + CHUNK)
        cum = l[..., c:e].cumsum(-1)
        gap = cum[..., :, None] - cum[..., None, :]
        later = torch.ones((e - c, e - c), dtype=torch.bool, device="cuda").tril_()
        D = torch.where(later, gap, -math.inf).exp().float()[:, :, None]       # decay from token j to token i
        into = cum.exp().float()[:, :, None, :, None]                          # ... from the chunk's start to i
        out = (cum[..., -1:] - cum).exp().float()[:, :, None, :, None]         # ... from j to its end
        over = cum[..., -1].exp().float()[..., None, None]
        qc, kc, vc = q[..., c:e, :], k[..., c:e, :], v[..., c:e, :]
        o[..., c:e, :] = (qc @ kc.transpose(-1, -2) * D @ vc + into * (qc @ state[:, :, None])) * scale
        if grad:
            dc = do[..., c:e, :]
            dq[..., c:e, :] = (dc @ vc.transpose(-1, -2) * D @ kc + into * (dc @ state[:, :, None].transpose(-1, -2))) * scale
            decays.append((D, into, out, over))
        state = over * state + ((kc * out).transpose(-1, -2) @ vc)[:, :, 0]

    def rows(x):   # back to the layout of the inputs, in their type
        x = x.flatten(1, 2).permute(0, 2, 1, 3).to(torch.bfloat16)
        return _packed(x, s["cu"], s["q"].shape[0]) if packed else x.contiguous()

    got = {"o": rows(o)}
    if s["states"]:
        got["state"] = state
    if grad:
        G = s["dstate"] if s["states"] else torch.zeros_like(state)
        for c, (D, into, out, over) in zip(reversed(starts), reversed(decays)):   # backward in time
            e = min(L, c + CHUNK)
            qc, kc, vc, dc = (x[..., c:e, :] for x in (q, k, v, do))
            P, dP = qc @ kc.transpose(-1, -2) * D * scale, dc @ vc.transpose(-1, -2) * D * scale
            dk[..., c:e, :] = (dP.transpose(-1, -2) @ qc).sum(2, keepdim=True) + out * (vc @ G[:, :, None].transpose(-1, -2))
            dvv[..., c:e, :] = (P.transpose(-1, -2) @ dc).sum(2, keepdim=True) + out * (kc @ G[:, :, None])
            G = over * G + ((qc * into).transpose(-1, -2) @ dc).sum(2) * scale
        got["dq"], got["dk"], got["dv"] = rows(dq), rows(dk), rows(dvv)
        if s["states"]:
            got["dstate"] = G
    return got


def _plain_step(s):
    q, k, v, S = s["q"].float(), s["k"].float(), s["v"].float(), s["state"]
    S.mul_(s["log_decay"].exp()[:, None, None]).add_(k[..., :, None] * v[..., None, :])
    o = q.unflatten(1, (s["Hkv"], -1)) @ S / math.sqrt(s["d"])
    return {"o": o.flatten(1, 2).to(torch.bfloat16), "state": S}


def _places(s, cu, T):
    """Page and slot of each packed row: row t of a sequence with n rows is token lens - n + t."""
    cu = cu.long()
    row = torch.arange(T, device="cuda")
    seq = (row[:, None] >= cu[None, 1:]).sum(1)
    slot = s["lens"].long()[seq] - (cu[1:] - cu[:-1])[seq] + row - cu[seq]
    return s["table"].long()[seq, slot // PAGE], slot % PAGE


def _plain_write(rows, scales, x, page, slot):
    if scales is None:
        rows[page, :, slot] = x
        return
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))   # amax = m 2^e with m in [1/2, 1); 448 = 7/8 2^9
    e = torch.where(m > 0, e - 9 + (m > 0.875), -126).clamp(min=-126)
    # 2^-e in 64 bits: the product is exact, so that the cast rounds once
    rows[page, :, slot] = (x.double() * ((1023 - e.long()) << 52).view(torch.float64)[..., None]).float().to(torch.float8_e4m3fn)
    scales[page, :, slot] = (e + 127).to(torch.uint8)


def _values(rows, scales):   # (a scale's exponent is that of a 32-bit float: 2^(e - 127), exactly)
    return rows.float() if scales is None else rows.float() * (scales.int() << 23).view(torch.float32)[..., None]


def _plain_read(rows, scales, page, slot):
    return _values(rows[page, :, slot], None if scales is None else scales[page, :, slot]).to(torch.bfloat16)


def _visible(nq, nk, lens_q, lens_k, window, sinks):
    """[B, nq, nk]: causal (aligned at the end), within the window or among the first keys."""
    i = torch.arange(nq, device="cuda")[None, :, None] + (lens_k - lens_q)[:, None, None]
    j = torch.arange(nk, device="cuda")[None, None, :]
    ok = (j <= i) & (j < lens_k[:, None, None])
    if window >= 0:
        ok &= (j >= i - window) | (j < sinks)
    return ok


def _plain_decode(s):
    kr, ks, vr, vs = s["cache"]
    at = s["table"].long().clamp(min=0)   # a place without a page: any page

    def gather(rows, scales):   # [B, Hkv, keys, channels]
        return _values(rows[at], None if scales is None else scales[at]).transpose(1, 2).flatten(2, 3)

    k, v = gather(kr, ks), gather(vr, vs)
    B, Hkv, N, d = k.shape
    H, cu, lens = s["H"], s["cu"], s["lens"].long()
    group, n = H // Hkv, s["longest_new"]
    new = (cu[1:] - cu[:-1]).long()
    q = _padded(s["q"], cu, n).float().reshape(B, n, Hkv, group, d).permute(0, 2, 3, 1, 4)
    ok = _visible(n, N, new, lens, s["window"], s["sinks"])
    ok &= (torch.arange(n, device="cuda")[None, :] < new[:, None])[:, :, None]
    x = torch.matmul(q.reshape(B, Hkv, group * n, d), k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    x = x.reshape(B, Hkv, group, n, N).masked_fill_(~ok[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp_(min=-1e30)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p /= total.clamp(min=1e-30)
    v = v.masked_fill((torch.arange(N, device="cuda") >= lens[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(p.reshape(B, Hkv, group * n, N), v).reshape(B, H, n, -1)
    lse = (top + total.log()).reshape(B, H, n)
    T = s["q"].shape[0]
    return {"o": _packed(o.transpose(1, 2), cu, T).to(torch.bfloat16), "lse": _packed(lse.transpose(1, 2), cu, T).t()}


# ------------------------------------------------------------------------------------------ one pass

def run(s):
    kind = s["kind"]
    if own:
        from exact_attention_blackwell_tma_gb300 import binding
    if kind == "lin":
        if not own:
            return _plain_lin(s)
        o, state = binding.linear_forward(s["q"], s["k"], s["v"], s["log_decay"], cu_seqlens=s["cu"], state=s["state"],
                                          final_state=s["states"])
        out = {"o": o}
        if s["states"]:
            out["state"] = state
        if s["grad"]:
            out["dq"], out["dk"], out["dv"], dstate = binding.linear_backward(
                s["q"], s["k"], s["v"], s["log_decay"], s["do"], cu_seqlens=s["cu"], state=s["state"],
                dstate=s["dstate"])
            if s["states"]:
                out["dstate"] = dstate
        return out
    if kind == "step":
        if not own:
            return _plain_step(s)
        return {"o": binding.linear_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"]), "state": s["state"]}
    kr, ks, vr, vs = s["cache"]
    if kind == "write":
        if own:
            cache = binding.PagedCache(kr, vr, ks, vs)
            binding.paged_append(cache, s["k"], s["v"], s["table"], s["lens"], cu_seqlens=s["cu"])
            k, v = binding.paged_read(cache, s["table"], s["lens"], s["read"], cu_seqlens=s["cu_read"])
        else:
            page, slot = _places(s, s["cu"], s["k"].shape[0])
            _plain_write(kr, ks, s["k"], page, slot)
            _plain_write(vr, vs, s["v"], page, slot)
            page, slot = _places(s, s["cu_read"], s["read"])
            k, v = _plain_read(kr, ks, page, slot), _plain_read(vr, vs, page, slot)
        return {"k": k, "v": v}
    if own:
        o, lse = binding.paged_forward(s["q"], binding.PagedCache(kr, vr, ks, vs), s["table"], s["lens"], causal=True,
                                       cu_seqlens=s["cu"], window=(s["window"], -1), sinks=s["sinks"])
        return {"o": o, "lse": lse}
    return _plain_decode(s)


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
    Hkv, d, dv = case["Hkv"], case["d"], case["dv"]
    if case["kind"] in ("lin", "step"):
        B, H = case["B"], case["H"]
        T, one = (B, 1) if case["kind"] == "step" else (sum(_lengths(case)), 4 * B * Hkv * d * dv)
        size = 2 * T * (H * (d + dv) + Hkv * (d + dv)) + 4 * Hkv
        flops = 2 * d * dv * (Hkv + H) * T   # the recurrence: states and outputs
        if case["kind"] == "step":
            return {"bytes": size + 8 * B * Hkv * d * dv, "flops": flops}
        if case["grad"]:
            size += 2 * T * (H * (d + dv) + Hkv * (d + dv))
            flops += 2 * d * dv * (2 * H + 2 * Hkv) * T
        if case["states"]:
            size += one * (4 if case["grad"] else 2)
        return {"bytes": size, "flops": flops}
    lens = _lengths(case)
    row = (d + dv) * case["bits"] // 8 + (2 if case["bits"] == 8 else 0)   # a key and value of one head in the cache
    if case["kind"] == "write":
        new = sum(_new(case, "new_lo", "new_hi"))
        read = sum(lens) if case["read_all"] else new
        return {"bytes": Hkv * (new * (2 * (d + dv) + row) + (read - new) * row + read * 2 * (d + dv)), "flops": 0}
    new = _new(case, "q_lo", "q_hi")
    seen = [_seen(a, n, case["window"], case["sinks"]) for a, n in zip(new, lens)]
    return {"bytes": Hkv * row * sum(x[1] for x in seen) + sum(new) * case["H"] * (2 * (d + dv) + 4),
            "flops": 2 * (d + dv) * case["H"] * sum(x[0] for x in seen)}


# ------------------------------------------------------------------------------------------ the definition in 64 bits

def _pow2(e):
    """2^e for whole e, exactly (powers by the device's exp2 or pow can be a bit off, which breaks ties)."""
    return torch.tensor([2.0 ** i for i in range(-200, 201)], dtype=torch.float64, device="cuda")[e.long() + 200]


def _e4m3(y):
    """Values of at most 448 in size to the nearest with four significant bits down to 2^-6 and steps of 2^-9 below, ties to even."""
    size = y.abs().clamp(min=2.0 ** -6)
    e = torch.floor(torch.log2(size))
    step = _pow2(torch.where(_pow2(e) > size, e - 1, torch.where(_pow2(e + 1) <= size, e + 1, e)) - 3)
    return torch.round(y / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    Hkv, d, dv = case["Hkv"], case["d"], case["dv"]
    if case["kind"] == "step":
        S = s["state"].double() * torch.exp(s["log_decay"].double())[:, None, None]
        S = S + torch.einsum("bhi,bhj->bhij", s["k"].double(), s["v"].double())
        q = s["q"].double().reshape(case["B"], Hkv, -1, d)
        return {"o": torch.einsum("bhgi,bhij->bhgj", q, S).reshape(case["B"], -1, dv) / math.sqrt(d), "state": S}
    lens = _lengths(case)
    if case["kind"] == "lin":
        H, T, grad, states = case["H"], sum(lens), case["grad"], case["states"]
        if 2 * (d + dv) * (3 if grad else 1) * H * sum(n * n for n in lens) > 6e12:
            return None
        flat = {n: s[n].reshape(T, -1, s[n].shape[-1]).double() for n in ("q", "k", "v") + (("do",) if grad else ())}
        out = {"o": torch.zeros((T, H, dv), dtype=torch.float64, device="cuda")}
        if states:
            out["state"] = torch.zeros((case["B"], Hkv, d, dv), dtype=torch.float64, device="cuda")
        if grad:
            out.update(dq=torch.zeros_like(flat["q"]), dk=torch.zeros_like(flat["k"]), dv=torch.zeros_like(flat["v"]))
            if states:
                out["dstate"] = torch.zeros_like(out["state"])
        at = 0
        for b, n in enumerate(lens):   # every pair of tokens, weighted by the decay over their distance
            place = torch.arange(n, device="cuda", dtype=torch.float64)
            gap = place[:, None] - place[None, :]
            for h in range(H):
                kv = h // (H // Hkv)
                l = s["log_decay"][kv].double()
                q, k, v = (flat[m][at:at + n, x].detach().requires_grad_(grad) for m, x in (("q", h), ("k", kv), ("v", kv)))
                S = (s["state"][b, kv].double() if states else torch.zeros((d, dv), dtype=torch.float64, device="cuda"))
                S = S.detach().requires_grad_(grad)
                w = torch.where(gap >= 0, torch.exp(l * gap.clamp(min=0)), 0.0)
                o = ((q @ k.T * w) @ v + torch.exp(l * (place + 1))[:, None] * (q @ S)) / math.sqrt(d)
                out["o"][at:at + n, h] = o.detach()
                last = torch.exp(l * n) * S + k.T @ (torch.exp(l * (n - 1 - place))[:, None] * v)
                if states:
                    out["state"][b, kv] = last.detach()
                if grad:
                    loss = (o * flat["do"][at:at + n, h]).sum()
                    if states and h % (H // Hkv) == 0:   # the query heads of a group share the state
                        loss = loss + (last * s["dstate"][b, kv].double()).sum()
                    a, c, e, f = torch.autograd.grad(loss, (q, k, v, S))
                    out["dq"][at:at + n, h] = a
                    out["dk"][at:at + n, kv] += c
                    out["dv"][at:at + n, kv] += e
                    if states:
                        out["dstate"][b, kv] += f
            at += n
        for name, x in (("o", "q"), ("dq", "q"), ("dk", "k"), ("dv", "v")):
            if name in out:
                out[name] = out[name].reshape(s[x].shape[:-1] + (out[name].shape[-1],))
        return out

    def rows_of(i, b, tokens):   # [n, Hkv, channels] of sequence b, as the values they stand for
        page, slot = s["table"][b].long()[tokens // PAGE], tokens % PAGE
        x = s["cache"][2 * i][page, :, slot].double()
        return x if case["bits"] == 16 else x * _pow2(s["cache"][2 * i + 1][page, :, slot].double() - 127)[..., None]

    if case["kind"] == "write":
        new, out = _new(case, "new_lo", "new_hi"), {}
        for i, name in enumerate(("k", "v")):
            got, at = [], 0
            for b, (n, total) in enumerate(zip(new, lens)):
                if case["read_all"] and total > n:
                    got.append(rows_of(i, b, torch.arange(total - n, device="cuda")))
                x = s[name][at:at + n].double()
                at += n
                if case["bits"] == 8:
                    top = x.abs().amax(-1, keepdim=True).clamp(min=1e-45)
                    e = torch.ceil(torch.log2(top / 448.0))
                    e = torch.where(448.0 * _pow2(e - 1) >= top, e - 1, torch.where(448.0 * _pow2(e) < top, e + 1, e))
                    e = e.clamp(min=-126)
                    x = _e4m3(x / _pow2(e)) * _pow2(e)
                got.append(x)
            out[name] = torch.cat(got)
        return out
    H, new = case["H"], _new(case, "q_lo", "q_hi")
    group, T = H // Hkv, sum(new)
    o = torch.zeros((T, H, dv), dtype=torch.float64, device="cuda")
    lse = torch.zeros((H, T), dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, total) in enumerate(zip(new, lens)):
        tokens = torch.arange(total, device="cuda")
        gap = torch.arange(total - n, total, device="cuda")[:, None] - tokens[None, :]
        keep = gap >= 0
        if case["window"] >= 0:
            keep &= (gap <= case["window"]) | (tokens < case["sinks"])[None, :]
        ks, vs = rows_of(0, b, tokens), rows_of(1, b, tokens)
        for h in range(Hkv):
            q = s["q"][at:at + n, h * group:(h + 1) * group].double().transpose(0, 1)
            score = torch.where(keep, q @ ks[:, h].T / math.sqrt(d), -math.inf)
            o[at:at + n, h * group:(h + 1) * group] = (torch.softmax(score, -1) @ vs[:, h]).transpose(0, 1)
            lse[h * group:(h + 1) * group, at:at + n] = torch.logsumexp(score, -1)
        at += n
    return {"o": o, "lse": lse}
