"""The token-cache operators as cases to measure: what a long-running token decode calls next to swa_decode.

    rope     rotary positions with several axes (time, height, width), and their gradient (swa_rope_nd)
    write    a run of new tokens quantised to 8 bits as it enters the rolling cache (swa_kv8_write)
    read     a run of cached tokens read back from 8 bits (swa_kv8_read)
    kv8      one decode step on the 8-bit cache: the new token quantised and attended to (swa_decode_kv8)
    prefix   one decode step of a batch that shares a long prefix (swa_decode_prefix)
    sparse   one decode step over the cache blocks that a score selects (swa_decode_sparse)

The plain forms below are elementary torch operations in 32 bits (64 for the angles and the block scores).
"""
import math

import torch

own = False

E_MIN, E_MAX = -40, 40  # exponents of a cached row's scale


# ------------------------------------------------------------------ cases
def listed():
    return [
        # every token of a 32-frame clip before a whole-clip prefill: (time, height, width) on 64-wide heads
        dict(name="rope_clip", op="rope", dtype="bf16", tokens=32128, heads=16, beside=0, D=64, nt=12, nh=10, nw=10,
             inverse=False),
        # its gradient in a training step, on the q and k heads of fused qkv rows
        dict(name="rope_gradient", op="rope", dtype="f32", tokens=4099, heads=40, beside=8, D=128, nt=22, nh=21, nw=21,
             inverse=True),
        # the new tokens of a batch in one decode step: latency
        dict(name="rope_step", op="rope", dtype="bf16", tokens=64, heads=40, beside=0, D=128, nt=22, nh=21, nw=21,
             inverse=False),
        # prompts of unequal length entering the cache
        dict(name="write_prompts", op="write", dtype="bf16", B=8, T=2048, W=4096, Hkv=8, D=128, lo=0.3, hi=1.0),
        # a cache handed on to code that wants 16 bits
        dict(name="read_back", op="read", dtype="bf16", B=16, T=1777, W=4096, Hkv=8, D=128, lo=0.5, hi=1.0),
        # the full rolling window at batch 64
        dict(name="kv8_window", op="kv8", dtype="bf16", B=64, W=4096, Hq=32, Hkv=8, D=128, lo=1.0, hi=40.0, idle=0),
        # a batch of unequal lengths with idle rows, 64-wide heads
        dict(name="kv8_ragged", op="kv8", dtype="bf16", B=33, W=8192, Hq=24, Hkv=8, D=64, lo=0.01, hi=1.0, idle=2),
        # one conversation: latency
        dict(name="kv8_single", op="kv8", dtype="bf16", B=1, W=1024, Hq=8, Hkv=2, D=128, lo=0.7, hi=0.7, idle=0),
        # a batch of answers over one long document
        dict(name="prefix_document", op="prefix", dtype="bf16", B=64, N=32768, W=1024, Hq=32, Hkv=8, D=128, lo=0.02,
             hi=0.5, idle=0),
        # a few samples after one prompt, three heads to a group
        dict(name="prefix_samples", op="prefix", dtype="bf16", B=5, N=5001, W=256, Hq=12, Hkv=4, D=64, lo=0.1, hi=3.0,
             idle=1),
        # long contexts of which a step reads a sixteenth
        dict(name="sparse_long", op="sparse", dtype="bf16", B=16, W=32768, Hq=32, Hkv=8, D=128, block=64, select=32,
             first=1, last=2, lo=0.5, hi=1.0, idle=0),
        # short contexts in 32 bits, a last block that is not whole
        dict(name="sparse_f32", op="sparse", dtype="f32", B=3, W=5000, Hq=8, Hkv=2, D=64, block=16, select=24, first=2,
             last=3, lo=0.1, hi=1.3, idle=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "kv8", "kv8", "prefix", "prefix", "sparse", "sparse"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    D = rng.choice([64, 128])
    if op == "rope":
        D = rng.choice([32, 64, 96, 128, 256])
        a, b = sorted(rng.randint(0, D // 2) for _ in range(2))
        nw = rng.randint(0, D // 2 - b)
        return dict(op=op, dtype=dtype, tokens=_log(rng, 1, 20000), heads=rng.randint(1, 24), beside=rng.choice([0, 0, 8]),
                    D=D, nt=a, nh=b - a, nw=nw, inverse=rng.random() < 0.5)
    Hkv = rng.choice([1, 2, 4, 8])
    if op in ("write", "read"):
        W = _log(rng, 16, 4096)
        return dict(op=op, dtype=dtype, B=rng.randint(1, 8), T=_log(rng, 1, min(W, 2000)), W=W, Hkv=Hkv, D=D,
                    lo=round(rng.uniform(0.0, 0.9), 3), hi=1.0)
    Hq = Hkv * rng.randint(1, 8)
    most = 4000000 // (Hkv * (1 if dtype == "bf16" else 8))  # cached tokens of the batch
    B = _log(rng, 1, 48)
    idle = rng.choice([0, 0, min(1, B - 1)])
    lo = round(rng.uniform(0.0, 1.0), 3)
    hi = round(lo + rng.uniform(0.0, 2.0), 3)
    case = dict(op=op, dtype=dtype, B=B, W=_log(rng, 16, min(16384, most // B)), Hq=Hq, Hkv=Hkv, D=D, lo=lo, hi=hi,
                idle=idle)
    if op == "prefix":
        case["N"] = _log(rng, 1, min(30000, most // B))
        case["W"] = min(case["W"], 2048)
    if op == "sparse":
        block = rng.choice([16, 32, 64, 128])
        first, last = rng.randint(0, 2), rng.randint(0, 3)
        case.update(block=block, first=first, last=last, select=max(1, first + last, _log(rng, 1, 64)))
    return case


def _lengths(case):
    """Tokens that each sequence has seen, the new one included: evenly from lo * W to hi * W; 0 for an idle row."""
    B, W = case["B"], case["W"]
    live = B - case.get("idle", 0)
    step = (case["hi"] - case["lo"]) / max(1, live - 1)
    return [max(1, int(W * (case["lo"] + i * step))) for i in range(live)] + [0] * (B - live)


def _counts(case):
    """Tokens of each sequence's run: evenly from lo * T to T."""
    B, T = case["B"], case["T"]
    return [min(T, round(T * (case["lo"] + (case["hi"] - case["lo"]) * (i + 1) / B))) for i in range(B)]


def work(case):
    op, D, e = case["op"], case["D"], 2 if case["dtype"] == "bf16" else 4
    if op == "rope":
        n = case["tokens"] * case["heads"] * D
        return {"bytes": 2 * n * e + case["tokens"] * 12, "flops": 3 * n}
    Hkv = case["Hkv"]
    if op in ("write", "read"):
        rows = 2 * sum(_counts(case)) * Hkv
        return {"bytes": rows * (D * e + D + 1), "flops": 2 * rows * D}
    B, Hq, W = case["B"], case["Hq"], case["W"]
    seen = [min(W, n) for n in _lengths(case)]
    io = (2 * B * Hq + 2 * B * Hkv) * D * e
    if op == "kv8":
        return {"bytes": io + 2 * sum(seen) * Hkv * (D + 1), "flops": 4 * sum(seen) * Hq * D}
    if op == "prefix":
        live = sum(n > 0 for n in seen)
        return {"bytes": io + 2 * (sum(seen) + case["N"]) * Hkv * D * e, "flops": 4 * (sum(seen) + live * case["N"]) * Hq * D}
    blocks = [-(-n // case["block"]) for n in seen]
    read = sum(min(n, case["select"] * case["block"]) for n in seen)
    return {"bytes": io + 2 * (read + sum(blocks)) * Hkv * D * e,
            "flops": 4 * read * Hq * D + 4 * sum(blocks) * Hkv * D}


# ------------------------------------------------------------------ inputs
def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _rows(shape, g, dtype):
    """Rows whose size varies from token to token, as keys and values do."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
    size = torch.randn(shape[:-1] + (1,), generator=g, device="cuda", dtype=dtype)
    return x.mul_(size.mul_(0.3).exp_())


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, op, D = _type(case), case["op"], case["D"]
    s = {"case": case}
    if op == "rope":
        n, H = case["tokens"], case["heads"]
        s["x"] = torch.randn(n, H + case["beside"], D, generator=g, device="cuda").to(dt)[:, :H]
        # a 37 x 27 grid of patches in each of many frames, from a frame far into the stream
        i = torch.arange(n, device="cuda")
        start = int(torch.randint(0, 100000, (1,), generator=g, device="cuda"))
        s["pos"] = torch.stack([start + i // 999, i % 999 // 37, i % 37], 1).to(torch.int32)
        s["out"] = torch.empty(n, H, D, device="cuda", dtype=dt)
        return s
    B, W, Hkv = case["B"], case["W"], case["Hkv"]
    order = torch.randperm(B, generator=g, device="cuda")
    if op in ("write", "read"):
        T = case["T"]
        s["count"] = torch.tensor(_counts(case), device="cuda", dtype=torch.int32)[order]
        s["pos"] = torch.randint(0, 3 * W, (B,), generator=g, device="cuda")
        k, v = (_rows((B, T if op == "write" else W, Hkv, D), g, dt) for _ in range(2))
        if op == "write":
            s["k"], s["v"] = k, v
            s["cache"] = [torch.zeros(B, W, Hkv, D, device="cuda").to(torch.float8_e4m3fn) if i % 2 == 0 else
                          torch.zeros(B, Hkv, W, device="cuda", dtype=torch.uint8) for i in range(4)]
        else:
            s["cache"] = [t for x in (k, v) for t in _cache8(x)]
            s["k"], s["v"] = (torch.zeros(B, T, Hkv, D, device="cuda", dtype=dt) for _ in range(2))
        return s
    s["pos"] = torch.tensor(_lengths(case), device="cuda", dtype=torch.int64)[order] - 1
    s["q"] = 1.5 * torch.randn(B, case["Hq"], D, generator=g, device="cuda")
    s["q"] = s["q"].to(dt)
    s["k_new"], s["v_new"] = (_rows((B, Hkv, D), g, dt) for _ in range(2))
    s["out"] = torch.empty(B, case["Hq"], D, device="cuda", dtype=dt)
    k, v = (_rows((B, W, Hkv, D), g, dt) for _ in range(2))
    if op == "kv8":
        s["cache"] = [t for x in (k, v) for t in _cache8(x)]
        return s
    if op == "sparse":  # neighbouring keys have a part in common
        block = case["block"]
        n = -(-W // block)
        k += torch.randn(B, n, Hkv, D, generator=g, device="cuda", dtype=dt).repeat_interleave(block, 1)[:, :W]
        s["bounds"] = _all_bounds(k, s["pos"], block)
        s["selected"] = torch.empty(B, Hkv, case["select"], device="cuda", dtype=torch.int32)
    s["cache"] = [k, v]
    if op == "prefix":
        s["prefix"] = [_rows((case["N"], Hkv, D), g, dt) for _ in range(2)]
    return s


# ------------------------------------------------------------------ plain forms
def _rope(x, pos, pairs, inverse):
    """Pair i (elements 2i and 2i + 1) of band a turns by pos[a] * 10000^(-j / pairs[a]), j its place in the band."""
    D = x.shape[-1]
    rate = torch.cat([10000.0 ** (-torch.arange(n, device=x.device, dtype=torch.float64) / max(n, 1)) for n in pairs])
    at = torch.cat([pos[:, a:a + 1].double().expand(-1, n) for a, n in enumerate(pairs)], 1)
    angle = at * rate
    angle = torch.nn.functional.pad(angle, (0, D // 2 - angle.shape[1]))
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if inverse:
        s = -s
    a, b = x[..., 0::2].float(), x[..., 1::2].float()
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2).to(x.dtype)


def _to8(x):
    """8-bit values of the rows of x and their scales' exponents: the least e with max|x| <= 448 * 2^e."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m == 0, E_MIN, torch.where(m <= 0.875, e - 9, e - 8)).clamp(E_MIN, E_MAX)
    x = torch.ldexp(x, -e[..., None]).clamp(-448.0, 448.0)
    return x.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _cache8(x):
    x8, e = _to8(x)
    return x8, e.transpose(1, 2).contiguous()


def _from8(x8, e):
    return torch.ldexp(x8.float(), e.int()[..., None] - 127)


def _put(cache, slot, keep, new):
    """cache[b, slot[b, t]] = new[b, t] where keep[b, t]; with the second axis of a cache in front."""
    b = torch.arange(cache.shape[0], device=cache.device)[:, None]
    old = cache[b, slot]
    keep = keep.reshape(keep.shape + (1,) * (old.dim() - 2))
    cache[b, slot] = torch.where(keep, new, old)


def _put8(cache8, exps, slot, keep, x):
    x8, e = _to8(x)
    _put(cache8.view(torch.uint8), slot, keep, x8.view(torch.uint8))
    _put(exps.transpose(1, 2), slot, keep, e)


def _append(s):
    W = s["cache"][0].shape[1]
    slot, live = (s["pos"].clamp(min=0) % W)[:, None], (s["pos"] >= 0)[:, None]
    if len(s["cache"]) == 4:
        _put8(s["cache"][0], s["cache"][1], slot, live, s["k_new"][:, None])
        _put8(s["cache"][2], s["cache"][3], slot, live, s["v_new"][:, None])
    else:
        _put(s["cache"][0], slot, live, s["k_new"][:, None])
        _put(s["cache"][1], slot, live, s["v_new"][:, None])
    return slot, live


def _valid(pos, W):
    return torch.arange(W, device=pos.device) < (pos[:, None] + 1).clamp(max=W)


def _weigh(scores, seen):
    """Softmax weights over the last axis where `seen`; all 0 in a row that sees nothing."""
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = (scores - torch.where(top == -math.inf, 0.0, top)).exp()
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, 1.0, total)


def _all_bounds(k, pos, block):
    """Smallest and largest element of each block's valid keys [B, Hkv, blocks, 2, D]."""
    B, W, Hkv, D = k.shape
    n = -(-W // block)
    seen = _valid(pos, W)[..., None, None]
    pad = (0, 0, 0, 0, 0, n * block - W)
    low = torch.nn.functional.pad(torch.where(seen, k, math.inf), pad, value=math.inf)
    high = torch.nn.functional.pad(torch.where(seen, k, -math.inf), pad, value=-math.inf)
    low, high = low.view(B, n, block, Hkv, D).amin(2), high.view(B, n, block, Hkv, D).amax(2)
    empty = (torch.arange(n, device=k.device) * block > pos[:, None])[..., None, None]
    low, high = (torch.where(empty, 0.0, x).to(k.dtype) for x in (low, high))
    return torch.stack([low, high], 3).permute(0, 2, 1, 3, 4).contiguous()


def _renew_bounds(k, pos, bounds, block):
    """The bounds of the block that the new token entered, from the cache."""
    B, W, Hkv, D = k.shape
    now = pos.clamp(min=0) % W // block
    slot = now[:, None] * block + torch.arange(block, device=k.device)
    seen = (slot < (pos[:, None] + 1).clamp(max=W)) & (slot < W)
    rows = k[torch.arange(B, device=k.device)[:, None], slot.clamp(max=W - 1)]
    seen = seen[..., None, None]
    low, high = torch.where(seen, rows, math.inf).amin(1), torch.where(seen, rows, -math.inf).amax(1)
    new = torch.stack([low, high], 2)[:, None]  # [B, 1, Hkv, 2, D]
    _put(bounds.transpose(1, 2), now[:, None], (pos >= 0)[:, None], new.to(bounds.dtype))
    return now


def _select(q, bounds, pos, now, W, block, select, first, last):
    """The blocks [B, Hkv, select] in ascending order, -1 behind them: `first` from the start, `last` back from the
    newest, then by the greatest sum over the group's heads and the elements of max(q * low, q * high)."""
    B, Hkv, n = bounds.shape[:3]
    q = q.view(B, Hkv, -1, q.shape[-1]).double()
    up, down = q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)
    score = ((bounds[..., 1, :].double() @ up[..., None]) + (bounds[..., 0, :].double() @ down[..., None]))[..., 0]
    j = torch.arange(n, device=q.device)
    used = -(-(pos + 1).clamp(max=W) // block)  # blocks that hold a token
    back = (now[:, None] - j) % torch.where(used > 0, used, 1)[:, None]
    forced = (j < first) | (back < last)
    score = torch.where(forced[:, None], math.inf, score)
    score = torch.where((j < used[:, None])[:, None], score, -math.inf)
    take = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :select]
    take = torch.where(take < used[:, None, None], take, n).sort(-1).values
    take = torch.nn.functional.pad(take, (0, select - take.shape[-1]), value=n)
    return torch.where(take < n, take, -1).int()


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import streaming_frame_causal_b200 as swa
    if op == "rope":
        pairs = (case["nt"], case["nh"], case["nw"])
        if own:
            return swa.swa_rope_nd(s["x"], s["pos"], pairs, inverse=case["inverse"], out=s["out"])
        return _rope(s["x"], s["pos"], pairs, case["inverse"])
    if op == "write":
        if own:
            swa.swa_kv8_write(s["k"], s["v"], *s["cache"], s["pos"], count=s["count"])
        else:
            t = torch.arange(case["T"], device="cuda")
            slot, keep = (s["pos"][:, None] + t) % case["W"], t < s["count"][:, None]
            _put8(s["cache"][0], s["cache"][1], slot, keep, s["k"])
            _put8(s["cache"][2], s["cache"][3], slot, keep, s["v"])
        return s["cache"]
    if op == "read":
        if own:
            swa.swa_kv8_read(*s["cache"], s["pos"], s["k"], s["v"], count=s["count"])
        else:
            t = torch.arange(case["T"], device="cuda")
            slot, keep = (s["pos"][:, None] + t) % case["W"], (t < s["count"][:, None])[..., None, None]
            b = torch.arange(case["B"], device="cuda")[:, None]
            for i, to in ((0, s["k"]), (2, s["v"])):
                x = _from8(s["cache"][i].view(torch.uint8)[b, slot].view(torch.float8_e4m3fn),
                           s["cache"][i + 1].transpose(1, 2)[b, slot])
                to.copy_(torch.where(keep, x.to(to.dtype), to))
        return s["k"], s["v"]
    if own and op == "kv8":
        swa.swa_decode_kv8(s["q"], s["k_new"], s["v_new"], *s["cache"], s["pos"], s["out"])
        return s["out"], s["cache"]
    if own and op == "prefix":
        swa.swa_decode_prefix(s["q"], s["k_new"], s["v_new"], *s["prefix"], *s["cache"], s["pos"], s["out"])
        return s["out"], s["cache"]
    if own and op == "sparse":
        swa.swa_decode_sparse(s["q"], s["k_new"], s["v_new"], *s["cache"], s["bounds"], s["pos"], s["out"],
                              s["selected"], case["block"], n_first=case["first"], n_last=case["last"])
        return s["out"], s["selected"], s["bounds"], s["cache"]
    B, Hkv, D, W = case["B"], case["Hkv"], case["D"], case["W"]
    _append(s)
    q = s["q"].float().view(B, Hkv, -1, D) / math.sqrt(D)
    pos = s["pos"]
    if op == "kv8":
        k, v = (_from8(s["cache"][i], s["cache"][i + 1].transpose(1, 2)) for i in (0, 2))
        p = _weigh(q @ k.permute(0, 2, 3, 1), _valid(pos, W)[:, None, None])
        return (p @ v.transpose(1, 2)).reshape(B, -1, D).to(s["q"].dtype), s["cache"]
    if op == "prefix":
        N = case["N"]
        k, v = (x.float() for x in s["cache"])
        kp, vp = (x.float().transpose(0, 1) for x in s["prefix"])  # [Hkv, N, D]
        G = q.shape[2]
        shared = (q.transpose(0, 1).reshape(Hkv, B * G, D) @ kp.transpose(1, 2)).view(Hkv, B, G, N).transpose(0, 1)
        seen = torch.cat([(pos >= 0)[:, None].expand(B, N), _valid(pos, W)], 1)[:, None, None]
        p = _weigh(torch.cat([shared, q @ k.permute(0, 2, 3, 1)], -1), seen)
        o = (p[..., :N].transpose(0, 1).reshape(Hkv, B * G, N) @ vp).view(Hkv, B, G, D).transpose(0, 1)
        return (o + p[..., N:] @ v.transpose(1, 2)).reshape(B, -1, D).to(s["q"].dtype), s["cache"]
    block = case["block"]
    now = _renew_bounds(s["cache"][0], pos, s["bounds"], block)
    chosen = _select(s["q"], s["bounds"], pos, now, W, block, case["select"], case["first"], case["last"])
    slot = (chosen[..., None] * block + torch.arange(block, device="cuda")).flatten(2)  # [B, Hkv, select * block]
    seen = (chosen >= 0).repeat_interleave(block, -1) & (slot < (pos + 1).clamp(max=W)[:, None, None])
    slot = slot.clamp(0, W - 1)
    b, h = (torch.arange(n, device="cuda").view(shape) for n, shape in ((B, (-1, 1, 1)), (Hkv, (1, -1, 1))))
    k, v = (x[b, slot, h].float() for x in s["cache"])
    p = _weigh(q @ k.transpose(2, 3), seen[:, :, None])
    return (p @ v).reshape(B, -1, D).to(s["q"].dtype), chosen, s["bounds"], s["cache"]


# ------------------------------------------------------------------ 64 bits
def _round8(x):
    """Rows of x as the 8-bit format (4 significant bits, least normal 2^-6, greatest 448) holds them, in 64 bits."""
    x = x.double()
    top = x.abs().max(-1, keepdim=True).values
    e = torch.ceil(torch.log2(top / 448.0))
    e = torch.where(448.0 * torch.exp2(e - 1) >= top, e - 1, torch.where(448.0 * torch.exp2(e) < top, e + 1, e))
    scale = torch.exp2(torch.where(top == 0, E_MIN, e).clamp(E_MIN, E_MAX))
    y = x / scale
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448), scale


def exact(case, seed):
    s = prepare(case, seed)
    op, D = case["op"], case["D"]
    if op == "rope":
        x = torch.view_as_complex(s["x"].double().unflatten(-1, (D // 2, 2)).contiguous())
        turn = torch.ones(x.shape[0], D // 2, device="cuda", dtype=torch.complex128)
        i = 0
        for a, n in enumerate((case["nt"], case["nh"], case["nw"])):
            for j in range(n):
                w = s["pos"][:, a].double() * math.pow(10000.0, -j / n)
                turn[:, i] = torch.complex(w.cos(), w.sin())
                i += 1
        y = x * (turn.conj() if case["inverse"] else turn)[:, None]
        return torch.view_as_real(y).flatten(-2)
    B, W, Hkv = case["B"], case["W"], case["Hkv"]
    if op == "write":
        out = []
        for x in (s["k"], s["v"]):
            y = torch.zeros(B, W, Hkv, D, device="cuda", dtype=torch.float64)
            for b in range(B):
                n, at = int(s["count"][b]), int(s["pos"][b])
                y[b, torch.arange(at, at + n, device="cuda") % W] = _round8(x[b, :n])[0]
            out += [y, None]
        return out
    if op == "read":
        out = []
        for x8, e in (s["cache"][0:2], s["cache"][2:4]):
            y = torch.zeros(B, case["T"], Hkv, D, device="cuda", dtype=torch.float64)
            for b in range(B):
                n, at = int(s["count"][b]), int(s["pos"][b])
                slot = torch.arange(at, at + n, device="cuda") % W
                y[b, :n] = x8[b].double()[slot] * torch.exp2(e[b].double().t()[slot] - 127.0)[..., None]
            out.append(y)
        return tuple(out)
    G = case["Hq"] // Hkv
    out = torch.zeros(B, case["Hq"], D, device="cuda", dtype=torch.float64)
    for b in range(B):
        at = int(s["pos"][b])
        if at < 0:
            continue
        n = min(at + 1, W)
        if op == "kv8":
            k, v = (s["cache"][i][b].double() * torch.exp2(s["cache"][i + 1][b].double().t() - 127.0)[..., None]
                    for i in (0, 2))
            for x, new in ((k, s["k_new"][b]), (v, s["v_new"][b])):
                y, scale = _round8(new)
                x[at % W] = y * scale
        else:
            k, v = s["cache"][0][b].double(), s["cache"][1][b].double()
            k[at % W], v[at % W] = s["k_new"][b].double(), s["v_new"][b].double()
        k, v = k[:n], v[:n]
        if op == "prefix":
            k, v = torch.cat([s["prefix"][0].double(), k]), torch.cat([s["prefix"][1].double(), v])
        for h in range(Hkv):
            q = s["q"][b, h * G:(h + 1) * G].double()
            kh, vh = k[:, h], v[:, h]
            if op == "sparse":
                block = case["block"]
                m = -(-n // block)
                kb = torch.nn.functional.pad(kh, (0, 0, 0, m * block - n), value=math.nan).view(m, block, D)
                low, high = kb.nan_to_num(nan=math.inf).amin(1), kb.nan_to_num(nan=-math.inf).amax(1)
                score = torch.zeros(m, device="cuda", dtype=torch.float64)
                for g in range(G):
                    score += torch.maximum(q[g] * low, q[g] * high).sum(1)
                now = at % W // block
                score[:case["first"]] = math.inf
                score[[(now - i) % m for i in range(min(case["last"], m))]] = math.inf
                best = sorted(range(m), key=lambda j, v=score.tolist(): (-v[j], j))[:case["select"]]
                slot = torch.tensor(best, device="cuda")[:, None] * block + torch.arange(block, device="cuda")
                slot = slot.flatten()
                slot = slot[slot < n]
                kh, vh = kh[slot], vh[slot]
            w = torch.softmax(q @ kh.t() / math.sqrt(D), -1)
            out[b, h * G:(h + 1) * G] = w @ vh
    if op == "sparse":
        return out, None, None, [None, None]
    return out, [None] * len(s["cache"])
