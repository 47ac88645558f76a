"""Measured cases of the paged-latent-cache operators: rows written with their norms and rotation
(16-bit or e4m3 cache), rows read back, and attention of a batch that shares a prefix.

A cache row is [c (d_c) ‖ k^R (d_rope)]; a page holds ``page`` rows. ``run`` computes an operator
in plain torch operations, or through the package's entry points where ``own`` is true.
"""
import math
import types

import torch

own = False

# The two cache shapes of the package's workloads: 8 heads over 160-wide rows, and 576-wide rows
# (128 heads, or the 16..64 heads that a rank of a tensor-parallel group holds).
WIDE = {"d_c": 512, "d_rope": 64, "d_head": 128}
SLIM = {"d_c": 128, "d_rope": 32, "d_head": 64}


def listed():
    return [
        # one new token of one sequence: the call's latency
        dict(name="append_1_slim_fp16", op="append", **SLIM, page=64, dtype="fp16", cache="elem", T=1, seqs=1, far=256,
             gains="c", pad=0),
        # a decode step of 64 sequences, the latent normalised as it is written
        dict(name="append_64_bf16", op="append", **WIDE, page=64, dtype="bf16", cache="elem", T=64, seqs=64, far=4096,
             gains="c", pad=0),
        # chunked prefill of 64 sequences into the e4m3 cache, rows cut from a wider fused projection
        dict(name="append_8192_fp8_bf16", op="append", **WIDE, page=64, dtype="bf16", cache="fp8", T=8192, seqs=64,
             far=32768, gains="cr", pad=1536),
        # a ragged handful of tokens fetched from the e4m3 cache
        dict(name="read_1021_fp8_bf16", op="read", **WIDE, page=64, dtype="bf16", cache="fp8", T=1021, seqs=7),
        # a whole long sequence turned from the e4m3 cache back into 16-bit rows
        dict(name="read_131072_fp8_bf16", op="read", **WIDE, page=64, dtype="bf16", cache="fp8", T=131072, seqs=1),
        # 16-bit rows of the slim cache moved out (a sequence leaving the batch)
        dict(name="read_16001_slim_fp16", op="read", **SLIM, page=64, dtype="fp16", cache="elem", T=16001, seqs=16),
        # a few sequences behind a short system prompt
        dict(name="prefix_512_b4_h16_bf16", op="prefix", **WIDE, page=64, dtype="bf16", heads=16, B=4, prefix=512,
             suffix=40, idle=0),
        # the 8-head model, 16 sequences over 4096 shared tokens
        dict(name="prefix_4096_b16_h8_slim", op="prefix", **SLIM, page=64, dtype="bf16", heads=8, B=16, prefix=4096,
             suffix=256, idle=0),
        # one of eight tensor-parallel ranks (16 heads), 64 sequences, some rows of the batch idle
        dict(name="prefix_8192_b64_h16_bf16", op="prefix", **WIDE, page=64, dtype="bf16", heads=16, B=64, prefix=8192,
             suffix=512, idle=3),
        # one of two ranks (64 heads), an odd batch, fp16
        dict(name="prefix_4096_b23_h64_fp16", op="prefix", **WIDE, page=64, dtype="fp16", heads=64, B=23, prefix=4096,
             suffix=200, idle=0),
        # all 128 heads on one GPU
        dict(name="prefix_4096_b64_h128_bf16", op="prefix", **WIDE, page=64, dtype="bf16", heads=128, B=64,
             prefix=4096, suffix=128, idle=0),
        # one of four ranks (32 heads), a large batch behind a long shared document
        dict(name="prefix_32768_b256_h32_bf16", op="prefix", **WIDE, page=64, dtype="bf16", heads=32, B=256,
             prefix=32768, suffix=1024, idle=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "prefix", "prefix"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "append":
        T = _log(rng, 1, 16384)
        return dict(op=op, **rng.choice([WIDE, SLIM]), page=rng.choice([16, 64]), dtype=dtype,
                    cache=rng.choice(["elem", "fp8"]), T=T, seqs=_log(rng, 1, min(T, 1024)), far=_log(rng, 64, 131072),
                    gains=rng.choice(["", "c", "cr"]), pad=rng.choice([0, 8, 1536]))
    if op == "read":
        T = _log(rng, 1, 100000)
        return dict(op=op, **rng.choice([WIDE, SLIM]), page=rng.choice([16, 64]), dtype=dtype,
                    cache=rng.choice(["elem", "fp8"]), T=T, seqs=_log(rng, 1, min(T, 256)))
    slim = rng.random() < 0.3
    heads = rng.randint(1, 16) if slim else rng.choice([rng.randint(1, 128), 16, 32, 64, 128])
    B = _log(rng, 1, 256)
    pages = _log(rng, 1, 512)
    while B * heads * pages > 256 * 32 * 512:
        pages = max(1, pages // 2)
    return dict(op=op, **(SLIM if slim else WIDE), page=64, dtype=dtype, heads=heads, B=B, prefix=64 * pages,
                suffix=_log(rng, 1, 1024), idle=rng.choice([0, 0, 1]) if B > 1 else 0)


def _dtype(case):
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[case["dtype"]]


def _spread(total, parts, rng):
    """``total`` tokens over ``parts`` sequences, at least one each, unevenly."""
    cuts = torch.randperm(total - 1, generator=rng)[:parts - 1] + 1 if parts > 1 else torch.zeros(0, dtype=torch.int64)
    ends = torch.cat([cuts.sort().values, torch.tensor([total])])
    return ends - torch.cat([torch.zeros(1, dtype=torch.int64), ends[:-1]])


def _table(used, first, width, pages, rng):
    """Block table [len(used), width] of pages drawn from ``pages``: row b has entries first[b] ..
    used[b] of its own, -1 elsewhere."""
    col = torch.arange(width)[None]
    mask = (col >= first[:, None]) & (col < used[:, None])
    table = torch.full((len(used), width), -1, dtype=torch.int32)
    table[mask] = pages[torch.randperm(len(pages), generator=rng)[:int(mask.sum())]].to(torch.int32)
    return table


def _values(shape, std, dtype, gen):
    return (torch.randn(shape, device="cuda", dtype=torch.float32, generator=gen) * std).to(dtype)


def _fp8_pages(n, page, D, gen):
    """Pages as a writer leaves them: e4m3 bytes (no NaN code) and two positive scales per row."""
    bits = torch.randint(0, 0x7F, (n, page * D), device="cuda", dtype=torch.uint8, generator=gen)
    sign = torch.randint(0, 2, (n, page * D), device="cuda", dtype=torch.uint8, generator=gen) * 0x80
    scales = torch.rand((n, page * 2), device="cuda", dtype=torch.float32, generator=gen) * 3e-3 + 1e-3
    return torch.cat([bits + sign, scales.view(torch.uint8)], 1).contiguous()


def prepare(case, seed):
    rng = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, page, D = _dtype(case), case["page"], case["d_c"] + case["d_rope"]
    heads = case.get("heads", 128 if case["d_c"] == 512 else 8)
    s = {"case": case, "dims": types.SimpleNamespace(
        d_model=5120 if case["d_c"] == 512 else 512, n_heads=heads, d_head=case["d_head"], d_c=case["d_c"],
        d_cq=1536 if case["d_c"] == 512 else 96, d_rope=case["d_rope"], page_size=page, dtype=case["dtype"],
        rope_base=10000.0)}
    if case["op"] == "append":
        T, n = case["T"], case["seqs"]
        new = _spread(T, n, rng)
        start = torch.randint(0, case["far"] + 1, (n,), generator=rng)
        seq = torch.repeat_interleave(torch.arange(n), new)
        at = torch.arange(T) - torch.repeat_interleave(new.cumsum(0) - new, new)
        pos = start[seq] + at
        used = (start + new + page - 1) // page
        # only the pages that the new tokens touch need memory: those before are another call's
        pages = T // page + 2 * n
        table = _table(used, start // page, int(used.max()), torch.arange(pages), rng)
        s["x"] = _values((T, D + case["pad"]), 0.43, dt, gen)[:, :D]
        s["gain_c"] = (1 + _values((case["d_c"],), 0.1, torch.float32, gen)).to(dt) if "c" in case["gains"] else None
        s["gain_r"] = (1 + _values((case["d_rope"],), 0.1, torch.float32, gen)).to(dt) if "r" in case["gains"] else None
        if case["cache"] == "fp8":
            s["pool"] = _fp8_pages(pages, page, D, gen)
        else:
            s["pool"] = _values((pages, page, D), 0.43, dt, gen)
        s["seq"], s["pos"], s["table"] = (t.to(torch.int32).cuda() for t in (seq, pos, table))
    elif case["op"] == "read":
        T, n = case["T"], case["seqs"]
        lens = _spread(T, n, rng)
        used = (lens + page - 1) // page
        pages = T // page + n
        table = _table(used, torch.zeros_like(used), int(used.max()), torch.arange(pages), rng)
        seq = torch.repeat_interleave(torch.arange(n), lens)
        pos = torch.arange(T) - torch.repeat_interleave(lens.cumsum(0) - lens, lens)
        s["pool"] = _fp8_pages(pages, page, D, gen) if case["cache"] == "fp8" else _values((pages, page, D), 0.43, dt, gen)
        s["seq"], s["pos"], s["table"] = (t.to(torch.int32).cuda() for t in (seq, pos, table))
    else:
        B, P = case["B"], case["prefix"]
        sp = P // page
        lens = P + torch.randint(1, case["suffix"] + 1, (B,), generator=rng)
        first = torch.full((B,), sp)
        idle = torch.randperm(B, generator=rng)[:case["idle"]]  # rows of a padded batch: one token of their own
        lens[idle], first[idle] = 1, 0
        used = (lens + page - 1) // page
        ids = torch.randperm(sp + B * ((case["suffix"] + page - 1) // page), generator=rng)
        shared = ids[:sp].to(torch.int32)
        table = _table(used, first, max(sp + 1, int(used.max())), ids[sp:], rng)
        table[:, :sp] = torch.where((first == sp)[:, None], shared[None], table[:, :sp])
        s["pool"] = _values((len(ids), page, D), 0.43, dt, gen)
        s["q"] = _values((B, heads, D), 2.0, dt, gen)
        s["lens"], s["table"], s["shared"] = lens.to(torch.int32).cuda(), table.cuda(), shared.cuda()
        s["longest"] = int(lens.max())
    return s


# ------------------------------------------------------------------------------ plain forms
def _slots(s):
    """Index of each token's row among the pool's rows."""
    page = s["dims"].page_size
    ids = s["table"][s["seq"].long(), (s["pos"] // page).long()].long()
    return ids * page + (s["pos"] % page).long()


def _fp8_parts(s):
    """(bytes as e4m3 [pages, page, D], scales [pages, page, 2]), both views of the pool."""
    d = s["dims"]
    n, rows = s["pool"].shape[0], d.page_size * (d.d_c + d.d_rope)
    codes = s["pool"][:, :rows].view(torch.float8_e4m3fn).unflatten(1, (d.page_size, d.d_c + d.d_rope))
    return codes, s["pool"][:, rows:].view(torch.float32).unflatten(1, (d.page_size, 2))


def _normed(x, gain):
    if gain is None:
        return x
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6) * gain.float()


def _append(s):
    d = s["dims"]
    x = s["x"].float()
    c, k = _normed(x[:, :d.d_c], s["gain_c"]), _normed(x[:, d.d_c:], s["gain_r"])
    freq = d.rope_base ** (-torch.arange(0, d.d_rope, 2, device="cuda", dtype=torch.float64) / d.d_rope)
    angle = s["pos"].double()[:, None] * freq
    cos, sin = angle.cos().float(), angle.sin().float()
    even, odd = k[:, 0::2], k[:, 1::2]
    k = torch.stack([even * cos - odd * sin, even * sin + odd * cos], 2).flatten(1)
    at = _slots(s)
    if s["case"]["cache"] == "elem":
        s["pool"].view(-1, d.d_c + d.d_rope)[at] = torch.cat([c, k], 1).to(s["pool"].dtype)
        return s["pool"]
    scale = torch.stack([c.abs().amax(1), k.abs().amax(1)], 1) / 448
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    row = torch.cat([c / scale[:, :1], k / scale[:, 1:]], 1).clamp(-448, 448).to(torch.float8_e4m3fn)
    codes, scales = _fp8_parts(s)
    n, r = at // d.page_size, at % d.page_size
    codes.view(torch.uint8)[n, r] = row.view(torch.uint8)
    scales[n, r] = scale
    return codes, scales


def _read(s):
    d = s["dims"]
    at = _slots(s)
    if s["case"]["cache"] == "elem":
        return s["pool"].view(-1, d.d_c + d.d_rope)[at]
    codes, scales = _fp8_parts(s)
    n, r = at // d.page_size, at % d.page_size
    v, sc = codes.view(torch.uint8)[n, r].view(torch.float8_e4m3fn).float(), scales[n, r]
    return torch.cat([v[:, :d.d_c] * sc[:, :1], v[:, d.d_c:] * sc[:, 1:]], 1).to(_dtype(s["case"]))


def _prefix(s):
    d, page = s["dims"], s["dims"].page_size
    q = s["q"].float()
    B, H, D = q.shape
    sp = s["shared"].numel()
    lens = s["lens"].long()
    uses = lens >= sp * page
    scale = 1 / math.sqrt(d.d_head + d.d_rope)
    # the shared rows, once for every query row
    rows = s["pool"][s["shared"].long()].view(-1, D).float()
    s1 = (q.view(B * H, D) @ rows.T).view(B, H, -1) * scale
    s1 = s1.masked_fill(~uses[:, None, None], -math.inf)
    # each sequence's own rows, padded to the longest
    start = torch.where(uses, sp * page, 0)
    longest = max(page, s["case"]["suffix"])
    col = torch.arange((longest + page - 1) // page, device="cuda") + (start // page)[:, None]
    ids = s["table"].gather(1, col.clamp(max=s["table"].shape[1] - 1)).clamp(min=0).long()
    mine = s["pool"][ids].view(B, -1, D).float()
    s2 = q @ mine.mT * scale
    live = torch.arange(mine.shape[1], device="cuda")[None] < (lens - start)[:, None]
    s2 = s2.masked_fill(~live[:, None], -math.inf)
    top = torch.maximum(s1.amax(2), s2.amax(2))[..., None]
    e1, e2 = (s1 - top).exp_(), (s2 - top).exp_()
    total = e1.sum(2, keepdim=True) + e2.sum(2, keepdim=True)
    o = (e1.view(B * H, -1) @ rows[:, :d.d_c]).view(B, H, -1) + e2 @ mine[..., :d.d_c]
    return (o / total).to(s["q"].dtype), (top + total.log())[..., 0]


def run(state):
    s = state
    op, cache = s["case"]["op"], s["case"].get("cache")
    if not own:
        return {"append": _append, "read": _read, "prefix": _prefix}[op](s)
    import mla_latent_kv_42_b200 as M
    if op == "append":
        call = M.norm_append_kv_fp8 if cache == "fp8" else M.norm_append_kv
        call(s["dims"], s["x"], s["seq"], s["pos"], s["table"], s["pool"], gain_c=s["gain_c"], gain_r=s["gain_r"],
             eps=1e-6)
        return _fp8_parts(s) if cache == "fp8" else s["pool"]
    if op == "read":
        call = M.read_kv_fp8 if cache == "fp8" else M.read_kv
        return call(s["dims"], s["pool"], s["seq"], s["pos"], s["table"])
    return M.shared_prefix_attention(s["dims"], s["q"], s["pool"], s["table"], s["lens"], s["longest"], s["shared"])


def work(case):
    D, d_c = case["d_c"] + case["d_rope"], case["d_c"]
    if case["op"] == "append":
        row = D + 8 if case["cache"] == "fp8" else 2 * D
        return {"bytes": case["T"] * (2 * D + row + 8), "flops": 6 * case["T"] * D}
    if case["op"] == "read":
        row = D + 8 if case["cache"] == "fp8" else 2 * D
        return {"bytes": case["T"] * (2 * D + row + 8), "flops": case["T"] * D if case["cache"] == "fp8" else 0}
    B, H = case["B"], case["heads"]
    live = B - case["idle"]
    mine = live * (case["suffix"] + 1) / 2 + case["idle"]  # own tokens: 1 .. suffix, evenly likely
    byts = 2 * D * (case["prefix"] + mine) + B * H * (2 * D + 2 * d_c + 4)
    return {"bytes": byts, "flops": 2 * H * (live * case["prefix"] + mine) * (D + d_c)}


# ------------------------------------------------------------------------------ from the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d, page, D = s["dims"], case["page"], case["d_c"] + case["d_rope"]
    table, pool = s["table"].long(), s["pool"]
    if case["op"] == "prefix":
        o = torch.empty((case["B"], case["heads"], d.d_c), device="cuda", dtype=torch.float64)
        lse = torch.empty((case["B"], case["heads"]), device="cuda", dtype=torch.float64)
        for b, n in enumerate(s["lens"].tolist()):  # each sequence for itself, over its whole table
            rows = pool[table[b, :(n + page - 1) // page]].reshape(-1, D)[:n].double()
            scores = torch.einsum("hd,nd->hn", s["q"][b].double(), rows) / (d.d_head + d.d_rope) ** 0.5
            lse[b] = scores.logsumexp(1)
            o[b] = torch.einsum("hn,nc->hc", (scores - lse[b][:, None]).exp(), rows[:, :d.d_c])
        return o, lse
    slot = s["pos"].long()
    ids, slot = table[s["seq"].long(), torch.div(slot, page, rounding_mode="floor")], slot % page
    if case["cache"] == "fp8":
        n_bytes = page * D
        codes = pool[:, :n_bytes].reshape(-1, page, D).view(torch.float8_e4m3fn).double()
        scales = pool[:, n_bytes:].contiguous().view(torch.float32).reshape(-1, page, 2).double()
    if case["op"] == "read":
        if case["cache"] == "elem":
            return pool[ids, slot].double()
        wide = scales[ids, slot].repeat_interleave(torch.tensor([d.d_c, d.d_rope], device="cuda"), 1)
        return codes[ids, slot] * wide
    x = s["x"].double()
    parts = []
    for part, gain in ((x[:, :d.d_c], s["gain_c"]), (x[:, d.d_c:], s["gain_r"])):
        if gain is not None:
            part = part / (part.pow(2).sum(1, keepdim=True) / part.shape[1] + 1e-6).sqrt() * gain.double()
        parts.append(part)
    theta = torch.pow(torch.tensor(d.rope_base, dtype=torch.float64, device="cuda"),
                      torch.arange(d.d_rope // 2, device="cuda").double() * (-2.0 / d.d_rope))
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["pos"].double()[:, None] * theta[None])
    parts[1] = torch.view_as_real(torch.view_as_complex(parts[1].reshape(len(x), -1, 2).contiguous()) * turn).flatten(1)
    if case["cache"] == "elem":
        out = pool.double()
        out[ids, slot] = torch.cat(parts, 1)
        return out
    peak = torch.stack([p.abs().max(1).values for p in parts], 1)
    peak = torch.where(peak > 0, peak / 448, 1.0)
    codes[ids, slot] = torch.cat([parts[0] / peak[:, 0:1], parts[1] / peak[:, 1:2]], 1)
    scales[ids, slot] = peak
    return codes, scales
