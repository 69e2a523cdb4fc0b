"""Measured cases of the serving and training operators around differential attention.

Four operators, as one serving step chains them, and the backward of one:

* page plan:   block table, slot map and positions of a step, built on the GPU;
* qk norm:     RMS norm of each query and key head with the position rotation, and its backward;
* 4-bit cache: quantising new K/V rows into pages, and reading rows back;
* decode:      single-token differential attention (V1 and V2) over the paged 4-bit cache.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits) where ``own`` is false, and calls the framework where it is true.

The 4-bit cache.  A row is the 128 channels of one token's K or V in one KV
head: 8 blocks of 16.  A block holds a scale byte b (the value of the fp16
number with bits b << 7: five exponent and three mantissa bits, no sign) and
sixteen 4-bit codes (sign, then the index into 0, 0.5, 1, 1.5, 2, 3, 4, 6).  A
tile is 16 tokens of one head, 2304 bytes: K codes, V codes, K scales, V
scales.  A page of one head is page_size / 16 tiles in a row.
"""
import math

import torch

own = False

D = 128           # row width of the cache
TILE = 16         # tokens of a tile
TILE_BYTES = 2304
MAX_SCALE = 10240.0   # 6 * MAX_SCALE is still an fp16 number
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# |x| / scale above which the next level is taken; on a border the even index wins
BORDERS = ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
           (5.0, False))


# ---- cases -------------------------------------------------------------------
def listed():
    return [
        # one decode step of a batch of 64: a few microseconds of work, latency counts
        dict(name="plan_decode_64", op="plan", requests=64, prompts=0, longest=32768, page=64,
             spare=0, tight=False),
        # admission of long prompts next to running requests, odd counts, padded slot buffer
        dict(name="plan_prompts_517", op="plan", requests=517, prompts=37, longest=9001, page=16,
             spare=1023, tight=True),
        # the 64 new tokens of a V2 decode step (64 query heads on 8 KV heads)
        dict(name="norm_v2_decode_64", op="norm", tokens=64, hq=64, hk=8, d=128, rot=128,
             pairs="halves", dtype="bf16", fused=True, far=32768),
        # V2 prefill of the benchmark: 2 x 8192 tokens, 32 query heads on 8 KV heads
        dict(name="norm_v2_prefill", op="norm", tokens=16384, hq=32, hk=8, d=128, rot=128,
             pairs="halves", dtype="bf16", fused=True, far=8192),
        # V1 training shape (both 64-wide branches of 16 heads): backward of 4 x 4096 tokens
        dict(name="norm_bwd_v1", op="norm_bwd", tokens=16384, hq=32, hk=32, d=64, rot=64,
             pairs="halves", dtype="bf16", fused=False, far=4096),
        # an odd number of fp32 tokens, adjacent pairs, half of the features rotated
        dict(name="norm_bwd_odd_fp32", op="norm_bwd", tokens=1237, hq=12, hk=2, d=128, rot=64,
             pairs="adjacent", dtype="fp32", fused=False, far=131072),
        # the K/V rows of one decode step go into the cache and are read back
        dict(name="cache_decode_64", op="cache", tokens=64, hk=8, page=64, dtype="bf16",
             fused=True, dropped=False),
        # a long prompt's K/V rows (a slice of the fused projection), with rows that have no slot
        dict(name="cache_prompt_16383", op="cache", tokens=16383, hk=8, page=64, dtype="bf16",
             fused=True, dropped=True),
        # V2 decode workload of the benchmark: 64 sequences of 32768 entries
        dict(name="decode_v2_b64_l32768", op="decode", form=2, batch=64, longest=32768, hq=64,
             hk=8, page=64, ragged=False, window=0, norm=False),
        # two short requests: latency
        dict(name="decode_v2_b2_l1000", op="decode", form=2, batch=2, longest=1000, hq=16, hk=2,
             page=16, ragged=True, window=0, norm=False),
        # ragged lengths behind a sliding window
        dict(name="decode_v2_ragged_window", op="decode", form=2, batch=29, longest=32768, hq=32,
             hk=8, page=32, ragged=True, window=4096, norm=False),
        # V1: 32 heads of their own cache, per-head norm in the epilogue
        dict(name="decode_v1_b16_l8191", op="decode", form=1, batch=16, longest=8191, hq=32,
             hk=32, page=128, ragged=False, window=0, norm=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("plan", "norm", "norm_bwd", "cache", "decode", "decode"))
    page = rng.choice((16, 32, 64, 128))
    if op == "plan":
        requests = _log(rng, 1, 1500)
        return dict(op=op, requests=requests, prompts=rng.randint(0, min(requests, 40)),
                    longest=_log(rng, 1, 32768), page=page, spare=rng.choice((0, 0, 77, 5000)),
                    tight=rng.random() < 0.5)
    if op in ("norm", "norm_bwd"):
        d = rng.choice((64, 128))
        hk = rng.choice((1, 2, 4, 8))
        hq = hk * rng.choice((2, 4, 6, 8))
        most = 16384 * 40 * 128 if op == "norm" else 16384 * 64 * 64
        return dict(op=op, tokens=_log(rng, 1, min(20000, most // ((hq + hk) * d))), hq=hq, hk=hk,
                    d=d, rot=rng.choice((d, d, d // 2, 0)),
                    pairs=rng.choice(("halves", "adjacent")),
                    dtype=rng.choice(("bf16", "bf16", "fp32")), fused=rng.random() < 0.5,
                    far=_log(rng, 64, 1000000))
    if op == "cache":
        return dict(op=op, tokens=_log(rng, 1, 16384), hk=rng.choice((1, 2, 4, 8)), page=page,
                    dtype=rng.choice(("bf16", "bf16", "fp32")), fused=rng.random() < 0.5,
                    dropped=rng.random() < 0.5)
    form = rng.choice((1, 2, 2))
    batch = _log(rng, 1, 64)
    hk = rng.choice((2, 4, 8)) if form == 2 else rng.choice((4, 8, 16))
    hq = hk * rng.choice((2, 4, 6, 8, 10)) if form == 2 else hk
    longest = _log(rng, 2, min(32768, 64 * 32768 * 4 // (batch * hk)))
    return dict(op=op, form=form, batch=batch, longest=longest, hq=hq, hk=hk, page=page,
                ragged=rng.random() < 0.6, window=rng.choice((0, 0, _log(rng, 1, 8192))),
                norm=form == 1 and rng.random() < 0.7)


# ---- the 4-bit format in elementary operations ----------------------------------
def _scale_bytes(amax):
    """Scale byte of each block from its largest magnitude (fp32), as uint8."""
    t = (amax.double() / 6.0).clamp(max=MAX_SCALE)
    step = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -14))) - 3.0)
    s = (torch.round(t / step) * step).to(torch.float16)      # exact: four significant bits
    b = (s.view(torch.int16).to(torch.int32) >> 7).to(torch.uint8)
    return torch.where(torch.isfinite(amax), b, torch.full_like(b, 255))


def _scale_values(b):
    return (b.to(torch.int32) << 7).to(torch.int16).view(torch.float16).float()


def _codes(x, s):
    """4-bit codes of x [..., 8, 16] for block scales s [..., 8, 1] (fp32)."""
    a = x.abs()
    c = torch.zeros_like(x, dtype=torch.uint8)
    for border, even_above in BORDERS:
        c += (a >= border * s) if even_above else (a > border * s)
    c = torch.where(s > 0, c, torch.zeros_like(c))
    c = torch.where((x < 0) & (c > 0), c + 8, c)
    return torch.where(torch.isfinite(s), c, torch.zeros_like(c))


def _level(c):
    lut = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=c.device)
    return lut[c.int()]


def _quantise(x):
    """(scale bytes [..., 8], codes [..., 8, 16]) of rows x [..., 128]."""
    x = x.float().reshape(*x.shape[:-1], 8, 16)
    amax = x.abs().amax(-1)
    amax = torch.where(torch.isnan(x).any(-1), torch.full_like(amax, math.nan), amax)
    b = _scale_bytes(amax)
    return b, _codes(x, _scale_values(b)[..., None])


def _held(x):
    """The values that the cache holds for rows x [..., 128], in fp32."""
    b, c = _quantise(x)
    return (_level(c) * _scale_values(b)[..., None]).reshape(x.shape)


def _pack_tiles(k, v):
    """Tiles [..., 2304] of rows k, v [..., 16, 128]."""
    lead = k.shape[:-2]
    out = []
    kb, kc = _quantise(k)
    vb, vc = _quantise(v)
    kc = kc.reshape(*lead, 16, 64, 2)
    vc = vc.reshape(*lead, 16, 64, 2)
    kc = kc[..., 0] | (kc[..., 1] << 4)
    vc = vc[..., 0] | (vc[..., 1] << 4)
    n = len(lead)
    out.append(kc.reshape(*lead, 1024))
    # V codes: [half of the tile][block of channels][token pair][token][8 bytes]
    vc = vc.reshape(*lead, 2, 4, 2, 8, 8).permute(*range(n), n, n + 3, n + 1, n + 2, n + 4)
    out.append(vc.reshape(*lead, 1024))
    # K scales: [token of the half][block pair][half][block]
    kb = kb.reshape(*lead, 2, 8, 4, 2).permute(*range(n), n + 1, n + 2, n, n + 3)
    out.append(kb.reshape(*lead, 128))
    # V scales: [block][token pair][half][token]
    vb = vb.reshape(*lead, 2, 4, 2, 8).permute(*range(n), n + 3, n + 1, n, n + 2)
    out.append(vb.reshape(*lead, 128))
    return torch.cat(out, -1)


def _unpack(tiles, what):
    """fp32 rows [..., 16, 128] of K ("k") or V ("v") from tiles [..., 2304]."""
    lead = tiles.shape[:-1]
    n = len(lead)
    if what == "k":
        c = tiles[..., :1024].reshape(*lead, 16, 64)
        b = tiles[..., 2048:2176].reshape(*lead, 8, 4, 2, 2)
        b = b.permute(*range(n), n + 2, n, n + 1, n + 3).reshape(*lead, 16, 8)
    else:
        c = tiles[..., 1024:2048].reshape(*lead, 2, 8, 4, 2, 8)
        c = c.permute(*range(n), n, n + 2, n + 3, n + 1, n + 4).reshape(*lead, 16, 64)
        b = tiles[..., 2176:2304].reshape(*lead, 8, 4, 2, 2)
        b = b.permute(*range(n), n + 2, n + 1, n + 3, n).reshape(*lead, 16, 8)
    lut = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=tiles.device)
    byte = torch.arange(256, device=tiles.device)
    two = torch.stack((lut[byte & 15], lut[byte >> 4]), -1)          # [256, 2]
    x = two[c.int()].reshape(*lead, 16, 8, 16)
    x *= _scale_values(b)[..., None]
    return x.reshape(*lead, 16, D)


# ---- states ----------------------------------------------------------------------
def _dtype(case):
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


def _slices(gen, tokens, widths, dtype, fused, dev):
    """Projection outputs: slices of one fused [tokens, sum] tensor, or tensors of their own.
    Channels differ in size, as projected activations do."""
    total = sum(widths)
    x = torch.randn(tokens, total, generator=gen, device=dev)
    x *= torch.exp(0.5 * torch.randn(total, generator=gen, device=dev))
    x = x.to(dtype)
    parts = list(x.split(widths, dim=1))
    return parts if fused else [p.contiguous() for p in parts]


def _random_cache(gen, pages, hk, page, dev):
    """A cache of normal rows, quantised."""
    cache = torch.empty(pages, hk, page * 144, dtype=torch.uint8, device=dev)
    flat = cache.view(-1, TILE_BYTES)
    chunk = 1 << 15
    for at in range(0, flat.shape[0], chunk):
        n = min(chunk, flat.shape[0] - at)
        k = torch.randn(n, 16, D, generator=gen, device=dev)
        v = torch.randn(n, 16, D, generator=gen, device=dev)
        flat[at:at + n] = _pack_tiles(k, v)
    return cache


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 7919 + 13)
    i32 = dict(dtype=torch.int32, device=dev)
    op = case["op"]
    s = {"case": dict(case), "seed": seed}
    if op == "plan":
        R, ps, longest = case["requests"], case["page"], case["longest"]
        new = torch.ones(R, **i32)
        lens = torch.randint(1, longest + 1, (R,), generator=gen, **i32)
        lens[torch.rand(R, generator=gen, device=dev) < 0.1] //= ps      # some short ones
        if case["prompts"]:
            at = torch.randperm(R, generator=gen, device=dev)[:case["prompts"]]
            new[at] = torch.randint((longest + 1) // 2, longest + 1, (case["prompts"],),
                                    generator=gen, **i32)
            lens[at] = 0
        new[torch.rand(R, generator=gen, device=dev) < 0.03] = 0         # paused requests
        new[:1].clamp_(min=1)
        old = (lens + ps - 1) // ps
        need = (lens + new + ps - 1) // ps - old
        total, held = int(need.sum()), int(old.sum())
        free = max(1, total * 9 // 10 if case["tight"] else total + 100)
        n_pages = held + free
        order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
        max_pages = (2 * longest + ps - 1) // ps
        blk = torch.arange(max_pages, device=dev)
        first = torch.cumsum(old, 0) - old
        table = order[(first[:, None] + blk).clamp(max=n_pages - 1)]
        table = torch.where(blk < old[:, None], table, torch.full_like(table, -1))
        stack = torch.full((n_pages,), -1, **i32)
        stack[:free] = order[held:]
        s.update(new=new, lens=lens, table=table.contiguous(), stack=stack,
                 count=torch.full((1,), free, **i32), n_slots=_slot_rows(case))
        return s
    if op in ("norm", "norm_bwd"):
        T, hq, hk, d = case["tokens"], case["hq"], case["hk"], case["d"]
        widths = [hq * d, hk * d, hk * d]
        q, k, _ = _slices(gen, T, widths, _dtype(case), case["fused"], dev)
        s.update(q=q.unflatten(1, (hq, d)), k=k.unflatten(1, (hk, d)))
        s["positions"] = torch.randint(0, case["far"], (T,), generator=gen, **i32)
        # the framework takes the frequencies a model keeps, in fp32
        i = torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64)
        s["inv_freq"] = (10000.0 ** (-i / max(1, case["rot"]))).float() if case["rot"] else None
        s["wq"] = 1 + 0.2 * torch.randn(d, generator=gen, device=dev)
        s["wk"] = 1 + 0.2 * torch.randn(d, generator=gen, device=dev)
        if op == "norm_bwd":
            s["gq"] = torch.randn(T, hq, d, generator=gen, device=dev)
            s["gk"] = torch.randn(T, hk, d, generator=gen, device=dev)
        return s
    if op == "cache":
        T, hk, ps = case["tokens"], case["hk"], case["page"]
        _, k, v = _slices(gen, T, [4 * hk * D, hk * D, hk * D], _dtype(case), case["fused"], dev)
        s.update(k=k.unflatten(1, (hk, D)), v=v.unflatten(1, (hk, D)))
        pages = (T + ps - 1) // ps + 3
        order = torch.randperm(pages, generator=gen, device=dev)
        tok = torch.arange(T, device=dev)
        slots = (order[tok // ps] * ps + tok % ps).to(torch.int32)
        if T <= 256:   # a decode step: every token lies in a page of another request
            pages = T + 3
            slots = (torch.randperm(pages, generator=gen, device=dev)[:T] * ps +
                     torch.randint(0, ps, (T,), generator=gen, device=dev)).to(torch.int32)
        if case["dropped"]:
            slots[torch.rand(T, generator=gen, device=dev) < 0.02] = -1
        s["slots"] = slots
        s["cache"] = torch.zeros(pages, hk, ps * 144, dtype=torch.uint8, device=dev)
        s["back_k"] = torch.zeros(T, hk, D, dtype=torch.bfloat16, device=dev)
        s["back_v"] = torch.zeros(T, hk, D, dtype=torch.bfloat16, device=dev)
        return s
    B, hq, hk, ps, L = case["batch"], case["hq"], case["hk"], case["page"], case["longest"]
    if case["ragged"]:
        lens = torch.randint(0, L + 1, (B,), generator=gen, **i32)
        lens[0] = L
    else:
        lens = torch.full((B,), L, **i32)
    per = (L + ps - 1) // ps
    pages = B * per + 1
    table = torch.randperm(pages, generator=gen, device=dev)[:B * per].to(torch.int32)
    table = table.view(B, per)
    used = torch.arange(per, device=dev) < ((lens + ps - 1) // ps)[:, None]
    s["table"] = torch.where(used, table, torch.full_like(table, -1)).contiguous()
    s["lens"] = lens
    s["cache"] = _random_cache(gen, pages, hk, ps, dev)
    s["q"] = torch.randn(B, hq, D, generator=gen, device=dev).to(torch.bfloat16)
    n_lam = hq // 2 if case["form"] == 2 else hq
    s["lam"] = 0.2 + 0.6 * torch.rand(n_lam, generator=gen, device=dev)
    s["gain"] = 1 + 0.1 * torch.randn(D, generator=gen, device=dev) if case["norm"] else None
    return s


def _slot_rows(case):
    """Rows of a step's token budget: one for each request, and the prompts' usual lengths."""
    return case["requests"] + case["prompts"] * case["longest"] * 4 // 5 + case["spare"]


LAMBDA_INIT = 0.7778701   # layer 12


# ---- one pass ----------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"plan": _own_plan, "norm": _own_norm, "norm_bwd": _own_norm_bwd,
                "cache": _own_cache, "decode": _own_decode}[op](s)
    return {"plan": _plan, "norm": _norm, "norm_bwd": _norm_bwd, "cache": _cache,
            "decode": _decode}[op](s)


def _own_plan(s):
    from differential_attention_sm_b200 import binding as da
    r = da.diffattn_page_plan(s["new"], s["lens"], s["table"], s["stack"], s["count"],
                              s["case"]["page"], s["n_slots"])
    r["block_table"] = s["table"]
    return r


def _own_norm(s):
    from differential_attention_sm_b200 import binding as da
    c = s["case"]
    q, k = da.diffattn_qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"],
                                    q_weight=s["wq"], k_weight=s["wk"], norm_eps=1e-6,
                                    interleaved=c["pairs"] == "adjacent")
    return {"q": q, "k": k}


def _own_norm_bwd(s):
    from differential_attention_sm_b200 import binding as da
    c = s["case"]
    if "workspace" not in s:   # a training program keeps one
        need = da.diffattn_qk_norm_rope_bwd_workspace_size(c["tokens"], c["hq"], c["hk"], c["d"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=s["q"].device)
    return da.diffattn_qk_norm_rope_bwd(s["q"], s["k"], s["gq"], s["gk"], s["positions"],
                                        s["inv_freq"], q_weight=s["wq"], k_weight=s["wk"],
                                        norm_eps=1e-6, interleaved=c["pairs"] == "adjacent",
                                        workspace=s["workspace"])


def _own_cache(s):
    from differential_attention_sm_b200 import binding as da
    da.diffattn_kv4_append(s["k"], s["v"], s["slots"], s["cache"])
    k, v = da.diffattn_kv4_read(s["cache"], s["slots"], out=(s["back_k"], s["back_v"]))
    return {"k": k, "v": v}


def _own_decode(s):
    from differential_attention_sm_b200 import binding as da
    c = s["case"]
    if "workspace" not in s:   # a server keeps one
        need = (da.diffattn_v2_decode_kv4_workspace_size(c["batch"], c["hq"], c["hk"])
                if c["form"] == 2
                else da.diffattn_v1_decode_kv4_workspace_size(c["batch"], c["hq"]))
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=s["q"].device)
    if c["form"] == 2:
        return da.diffattn_v2_decode_kv4(s["q"], s["cache"], s["table"], s["lens"], s["lam"],
                                         window=c["window"], workspace=s["workspace"])
    return da.diffattn_v1_decode_kv4(s["q"], s["cache"], s["table"], s["lens"], s["lam"],
                                     window=c["window"], apply_norm=c["norm"],
                                     norm_weight=s["gain"], norm_eps=1e-5,
                                     lambda_init=LAMBDA_INIT, workspace=s["workspace"])


def _plan(s):
    ps, new, lens, table = s["case"]["page"], s["new"].long(), s["lens"].long(), s["table"]
    R, max_pages = table.shape
    n = s["n_slots"]
    ends = torch.cumsum(new, 0)
    offsets = torch.cat((ends.new_zeros(1), ends))
    old = (lens + ps - 1) // ps
    need = (lens + new + ps - 1) // ps - old
    fits = (lens + new <= max_pages * ps) & ((new == 0) | (ends <= n))
    need = torch.where(fits, need, torch.zeros_like(need))
    upto = torch.cumsum(need, 0)
    count = s["count"].long()
    served = fits & ((need == 0) | (upto <= count))
    blk = torch.arange(max_pages, device=table.device)
    take = count - 1 - (upto - need)[:, None] - (blk - old[:, None])
    fresh = served[:, None] & (blk >= old[:, None]) & (blk < (old + need)[:, None])
    table = torch.where(fresh, s["stack"][take.clamp(0, s["stack"].numel() - 1)], table)
    i = torch.arange(n, device=table.device)
    r = torch.searchsorted(ends, i, right=True).clamp(max=R - 1)
    j = i - offsets[r]
    inside = i < ends[-1]
    pos = torch.where(inside, lens[r] + j, torch.zeros_like(j))
    ok = inside & served[r]
    slot = table[r, torch.where(ok, pos // ps, torch.zeros_like(pos))].long() * ps + pos % ps
    slot = torch.where(ok, slot, torch.full_like(slot, -1))
    used = torch.where(upto <= count, upto, torch.zeros_like(upto)).amax()
    i32 = torch.int32
    return {"slots": slot.to(i32), "positions": pos.to(i32), "offsets": offsets.to(i32),
            "served": served.to(i32),
            "cache_lens": torch.where(served, lens + new, lens).to(i32),
            "free_count": (count - used).to(i32), "block_table": table}


def _angles(s):
    """cos, sin [T, 1, rot / 2]: the angle is formed in 64 bits, far positions lose it in 32."""
    a = s["positions"].double()[:, None] * s["inv_freq"].double()
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _rotate(x, s, sign):
    if s["inv_freq"] is None:
        return x
    rot = s["case"]["rot"]
    cos, sin = _angles(s)
    sin = sign * sin
    head, tail = x[..., :rot], x[..., rot:]
    if s["case"]["pairs"] == "halves":
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((head, tail), -1)


def _norm(s):
    out = {}
    for x, w, name in ((s["q"], s["wq"], "q"), (s["k"], s["wk"], "k")):
        x32 = x.float()
        r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + 1e-6)
        out[name] = _rotate(x32 * r * w, s, 1.0).to(x.dtype)
    return out


def _norm_bwd(s):
    out = {}
    for x, w, dy, name in ((s["q"], s["wq"], s["gq"], "q"), (s["k"], s["wk"], s["gk"], "k")):
        x32 = x.float()
        r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + 1e-6)
        g = _rotate(dy, s, -1.0)
        n = x32 * r
        out["d%s_weight" % name] = (g * n).double().sum((0, 1)).float()
        wg = w * g
        out["d%s" % name] = r * (wg - n * (n * wg).mean(-1, keepdim=True))
    return out


def _cache(s):
    put = (s["slots"] >= 0)[:, None, None]
    zero = torch.zeros((), device=s["k"].device)
    return {"k": torch.where(put, _held(s["k"]), zero).to(torch.bfloat16),
            "v": torch.where(put, _held(s["v"]), zero).to(torch.bfloat16)}


def _rows_of(s, what):
    """fp32 rows [B, hk, L, 128] of every sequence's cache."""
    table = s["table"].clamp(min=0).long()
    tiles = s["cache"][table]                                       # [B, per, hk, bytes]
    B, per, hk, _ = tiles.shape
    tiles = tiles.view(B, per, hk, -1, TILE_BYTES).permute(0, 2, 1, 3, 4)
    x = _unpack(tiles, what)                                        # [B, hk, per, tiles, 16, D]
    return x.reshape(B, hk, -1, D)


def _decode(s):
    c = s["case"]
    B, hk = c["batch"], c["hk"]
    q = s["q"].float()
    if c["form"] == 2:
        q = q.view(B, hk, c["hq"] // hk, D)
        width = D
    else:   # a V1 head's branches: its first and last 64 features
        q = torch.stack((torch.cat((q[..., :64], torch.zeros_like(q[..., 64:])), -1),
                         torch.cat((torch.zeros_like(q[..., :64]), q[..., 64:]), -1)), 2)
        width = 64
    scores = torch.matmul(q, _rows_of(s, "k").transpose(-1, -2)) / math.sqrt(width)
    t = torch.arange(scores.shape[-1], device=q.device)
    lens = s["lens"].long()[:, None]
    seen = t < lens
    if c["window"]:
        seen = seen & (t >= lens - c["window"])
    seen = seen[:, None, None]
    scores = torch.where(seen, scores, torch.full_like(scores, -math.inf))
    top = scores.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(scores - top), torch.zeros_like(scores))
    del scores
    total = p.sum(-1, keepdim=True)
    # rows past a sequence's end may hold anything: they are taken out of the product
    rows = torch.where(seen.transpose(-1, -2), _rows_of(s, "v"), torch.zeros((), device=q.device))
    o = torch.matmul(p, rows)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.view(B, -1, 2, D)
    o = o[:, :, 0] - s["lam"][:, None] * o[:, :, 1]
    if c["norm"]:
        o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + 1e-5) * s["gain"] * (1 - LAMBDA_INIT)
    return o.to(torch.bfloat16)


# ---- what a pass cannot do without -----------------------------------------------------
def work(case):
    op = case["op"]
    if op == "plan":
        R, tokens = case["requests"], case["requests"] + case["prompts"] * case["longest"] * 0.75
        # lengths in and out, offsets, served, slots and positions, the new pages in and out
        return {"bytes": 20.0 * R + 8.0 * _slot_rows(case) + 8.0 * tokens / case["page"],
                "flops": 0.0}
    if op in ("norm", "norm_bwd"):
        T, rows, d = case["tokens"], case["hq"] + case["hk"], case["d"]
        size = 4 if case["dtype"] == "fp32" else 2
        n = float(T) * rows * d
        if op == "norm":
            return {"bytes": 2 * size * n + 4.0 * T, "flops": 8 * n}
        return {"bytes": (size + 8) * n + 4.0 * T, "flops": 16 * n}
    if op == "cache":
        rows = 2.0 * case["tokens"] * case["hk"]
        size = 4 if case["dtype"] == "fp32" else 2
        # rows in, held bytes out; held bytes in, bf16 rows out
        return {"bytes": rows * (D * size + 72 + 72 + 2 * D) + 8.0 * case["tokens"],
                "flops": 8 * rows * D}
    B, hk = case["batch"], case["hk"]
    mean = case["longest"] / 2 if case["ragged"] else case["longest"]
    if case["window"]:
        W, L = case["window"], case["longest"]
        if not case["ragged"]:
            mean = min(W, L)
        elif W < L:   # mean of min(len, W) over lengths spread evenly up to L
            mean = (W * W / 2 + W * (L - W)) / L
    heads = case["hq"] if case["form"] == 2 else 2 * case["hq"]
    qk = D if case["form"] == 2 else 64
    return {"bytes": 144.0 * B * hk * mean + 2.0 * B * case["hq"] * D * 2,
            "flops": 2.0 * B * heads * mean * (qk + D)}


# ---- the definition in 64 bits ------------------------------------------------------------
def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None       # whole numbers: compared as they are
    s = prepare(case, seed)
    if op == "norm":
        return {n: _exact_norm(s, s[n].double(), s["w" + n].double()) for n in ("q", "k")}
    if op == "norm_bwd":
        out = {}
        for n in ("q", "k"):
            x = s[n].double().requires_grad_(True)
            w = s["w" + n].double().requires_grad_(True)
            with torch.enable_grad():
                y = _exact_norm(s, x, w)
                dx, dw = torch.autograd.grad(y, (x, w), s["g" + n].double())
            out["d" + n], out["d%s_weight" % n] = dx, dw
        return out
    if op == "cache":
        out = {}
        for n in ("k", "v"):
            held = _exact_held(s[n].double())
            held[s["slots"] < 0] = 0
            out[n] = held
        return out
    return _exact_decode(s)


def _exact_norm(s, x, w):
    y = x / torch.sqrt(torch.mean(x ** 2, -1, keepdim=True) + 1e-6) * w
    rot = s["case"]["rot"]
    if not rot:
        return y
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                       torch.outer(s["positions"].double(), s["inv_freq"].double()))[:, None]
    if s["case"]["pairs"] == "halves":
        z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
        return torch.cat((z.real, z.imag, y[..., rot:]), -1)
    z = torch.view_as_complex(y[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn
    return torch.cat((torch.view_as_real(z).flatten(-2), y[..., rot:]), -1)


def _exact_held(x):
    """Nearest scale on the 8-bit grid, then the nearest level; ties to the even index."""
    dev = x.device
    grid = torch.arange(227, device=dev)                     # bytes 0 .. 0xE2
    e, m = grid // 8, grid % 8
    scales = torch.where(e == 0, m * 2.0 ** -17, (8.0 + m) * torch.exp2(e.double() - 18.0)).double()
    blocks = x.reshape(*x.shape[:-1], 8, 16)
    t = blocks.abs().amax(-1) / 6.0
    hi = torch.searchsorted(scales, t.contiguous()).clamp(max=226)
    lo = (hi - 1).clamp(min=0)
    up, down = scales[hi] - t, t - scales[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    pick = torch.where(t >= scales[226], torch.full_like(pick, 226), pick)
    sc = scales[pick][..., None]
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=dev)
    best = torch.zeros_like(blocks)
    gap = torch.full_like(blocks, math.inf)
    for i in (0, 2, 4, 6, 1, 3, 5, 7):                       # even indices first: they keep ties
        g = (blocks.abs() - levels[i] * sc).abs()
        best = torch.where(g < gap, levels[i] * sc, best)
        gap = torch.minimum(g, gap)
    return (best * torch.sign(blocks)).reshape(x.shape)


def _exact_decode(s):
    c = s["case"]
    dev = s["q"].device
    ps = c["page"]
    rows = []
    for b in range(c["batch"]):
        n = int(s["lens"][b])
        first = max(0, n - c["window"]) if c["window"] else 0
        if n == first:
            rows.append(torch.zeros(c["hq"] // 2 if c["form"] == 2 else c["hq"], D,
                                    dtype=torch.float64, device=dev))
            continue
        t = torch.arange(first, n, device=dev)
        K, V = _exact_rows(s, b, t)                          # [hk, n, D]
        q = s["q"][b].double()
        lam = s["lam"].double()
        if c["form"] == 2:
            group = c["hq"] // c["hk"]
            kv = torch.arange(c["hq"], device=dev) // group
            att = torch.softmax(torch.einsum("hd,hnd->hn", q, K[kv]) / math.sqrt(D), -1)
            o = torch.einsum("hn,hnd->hd", att, V[kv])
            outs = o[0::2] - lam[:, None] * o[1::2]
        else:
            a1 = torch.softmax(torch.einsum("hd,hnd->hn", q[:, :64], K[..., :64]) / 8.0, -1)
            a2 = torch.softmax(torch.einsum("hd,hnd->hn", q[:, 64:], K[..., 64:]) / 8.0, -1)
            outs = torch.einsum("hn,hnd->hd", a1 - lam[:, None] * a2, V)
            if c["norm"]:
                outs = outs * torch.rsqrt((outs ** 2).mean(-1, keepdim=True) + 1e-5)
                outs = outs * s["gain"].double() * (1 - LAMBDA_INIT)
        rows.append(outs)
    return torch.stack(rows)


def _exact_rows(s, b, t):
    """K and V rows [hk, n, 128] in 64 bits at tokens t of sequence b, byte by byte."""
    ps = s["case"]["page"]
    dev = t.device
    page = s["table"][b, t // ps].long()
    hk = s["cache"].shape[1]
    record = s["cache"].view(s["cache"].shape[0], hk, ps // TILE, TILE_BYTES)
    u = t % TILE
    tile = (t % ps) // TILE
    ch = torch.arange(D, device=dev)
    at_k = u[:, None] * 64 + ch // 2
    at_v = 1024 + 512 * (u[:, None] // 8) + 64 * (ch // 16) + 16 * ((u[:, None] % 8) // 2) \
        + 8 * (u[:, None] % 2) + (ch % 16) // 2
    blk = ch // 16
    at_ks = 2048 + 16 * (u[:, None] % 8) + 4 * (blk // 2) + 2 * (u[:, None] // 8) + blk % 2
    at_vs = 2176 + 16 * blk + 4 * ((u[:, None] % 8) // 2) + 2 * (u[:, None] // 8) + u[:, None] % 2
    out = []
    for codes, scales in ((at_k, at_ks), (at_v, at_vs)):
        rows = torch.empty(hk, t.numel(), D, dtype=torch.float64, device=dev)
        for h in range(hk):
            byte = record[page[:, None], h, tile[:, None], codes].long()
            nib = torch.where(ch % 2 == 0, byte & 15, byte >> 4)
            m = nib & 7
            mag = torch.where(m < 2, m * 0.5, (1 + 0.5 * (m % 2)) * torch.exp2((m // 2 - 1).double()))
            sb = record[page[:, None], h, tile[:, None], scales].long()
            sc = torch.where(sb < 8, sb * 2.0 ** -17, (8 + sb % 8) * torch.exp2((sb // 8).double() - 18))
            rows[h] = torch.where(nib >= 8, -mag, mag).double() * sc
        out.append(rows)
    return out
