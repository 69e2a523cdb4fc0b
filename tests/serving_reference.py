"""Plain 64-bit definitions (numpy, CPU) of the operators around decode, for
their tests: the 4-bit cache format byte by byte, the page plan request by
request, QK norm with rotation and its gradients, and decode over rows.

Error bounds of the decode (`decode_bound`) are derived here too.
"""
import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ---- the 4-bit cache ----------------------------------------------------------
def scale_values():
    """Value of every scale byte 0 .. 255 (fp16 with bits byte << 7)."""
    return (np.arange(256, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)


def quantise(rows):
    """(scale bytes [..., 8], codes [..., 128]) of rows [..., 128], float64."""
    rows = np.asarray(rows, np.float64)
    x = rows.reshape(-1, 16)
    grid = scale_values()[:0xE3]
    sb = np.empty(len(x), np.uint8)
    codes = np.zeros(x.shape, np.uint8)
    for i, blk in enumerate(x):
        if not np.isfinite(blk).all():
            sb[i] = 0xFF
            continue
        # above the largest scale and level the distances of huge values would all round alike
        d = np.abs(grid - min(np.abs(blk).max() / 6.0, grid[-1]))
        near = np.flatnonzero(d == d.min())
        s = near[0] if near[0] % 2 == 0 else near[-1]
        sb[i] = s
        if s == 0:
            continue
        for j, v in enumerate(blk):
            e = np.abs(LEVELS * grid[s] - min(abs(v), 6.0 * grid[s]))
            near = np.flatnonzero(e == e.min())
            c = near[0] if near[0] % 2 == 0 else near[-1]
            codes[i, j] = c + (8 if v < 0 and c else 0)
    return sb.reshape(rows.shape[:-1] + (8,)), codes.reshape(rows.shape)


def held(rows):
    """Values that the cache holds for rows [..., 128]."""
    sb, c = quantise(rows)
    v = LEVELS[c & 7] * np.where(c & 8, -1.0, 1.0)
    return v * np.repeat(scale_values()[sb], 16, axis=-1)


def byte_of(kind, t, c):
    """Byte of the tile with the code of token t, channel c; and its scale's."""
    b = c // 16
    if kind == "k":
        return t * 64 + c // 2, 2048 + 16 * (t % 8) + 4 * (b // 2) + 2 * (t // 8) + b % 2
    return (1024 + 512 * (t // 8) + 64 * b + 16 * ((t % 8) // 2) + 8 * (t % 2) + (c % 16) // 2,
            2176 + 16 * b + 4 * ((t % 8) // 2) + 2 * (t // 8) + t % 2)


def cache_rows(cache, table, lens, kind):
    """Rows [B][heads, len, 128] of every sequence, from the cache's bytes."""
    pages, heads, nbytes = cache.shape
    ps = nbytes // 144
    sv = scale_values()
    t = np.arange(16)[:, None]
    c = np.arange(128)[None]
    at, at_s = byte_of(kind, t, c)
    out = []
    for b, n in enumerate(lens):
        n = int(n)
        rows = np.zeros((heads, n, 128))
        for p0 in range(0, n, 16):
            tile = cache[table[b, p0 // ps], :, (p0 % ps) // 16 * 2304:][:, :2304]
            code = np.where(c % 2 == 0, tile[:, at] & 15, tile[:, at] >> 4)
            v = LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0)
            with np.errstate(invalid="ignore"):
                v = v * sv[tile[:, at_s]]
            m = min(16, n - p0)
            rows[:, p0:p0 + m] = v[:, :m]
        out.append(rows)
    return out


# ---- page plan ------------------------------------------------------------------
def page_plan(new, lens, table, stack, count, ps, n_slots):
    new = [max(0, int(n)) for n in new]
    lens = [max(0, int(n)) for n in lens]
    table = table.copy()
    R, max_pages = table.shape
    count = min(max(int(count), 0), len(stack))
    slots = np.full(n_slots, -1, np.int64)
    positions = np.zeros(n_slots, np.int64)
    offsets, served, out_lens = [0], [], []
    asked = 0
    left = count
    for r in range(R):
        at = offsets[-1]
        end = at + new[r]
        offsets.append(end)
        fits = lens[r] + new[r] <= max_pages * ps and (new[r] == 0 or end <= n_slots)
        old = -(-lens[r] // ps)
        need = -(-(lens[r] + new[r]) // ps) - old if fits else 0
        ok = fits and (need == 0 or asked + need <= count)
        if ok:
            for j in range(need):
                table[r, old + j] = stack[count - 1 - asked - j]
            left = min(left, count - asked - need) if need else left
        asked += need
        served.append(int(ok))
        out_lens.append(lens[r] + new[r] if ok else lens[r])
        for j in range(new[r]):
            if at + j < n_slots:
                pos = lens[r] + j
                positions[at + j] = pos
                if ok:
                    slots[at + j] = table[r, pos // ps] * ps + pos % ps
    return dict(slots=slots, positions=positions, offsets=np.array(offsets),
                served=np.array(served), cache_lens=np.array(out_lens),
                free_count=np.array([left]), block_table=table)


# ---- QK norm and rotation ----------------------------------------------------------
def pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, pos, inv_freq, interleaved, sign=1.0):
    """x [T, H, d] turned by sign * pos * inv_freq."""
    y = x.copy()
    if inv_freq is None or len(inv_freq) == 0:
        return y
    a, b = pairs(2 * len(inv_freq), interleaved)
    ang = (pos[:, None].astype(np.longdouble) * inv_freq.astype(np.longdouble))
    c = np.cos(ang).astype(np.float64)[:, None]
    s = sign * np.sin(ang).astype(np.float64)[:, None]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def norm_rope(x, w, eps, pos, inv_freq, interleaved):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return rotate(x * r * w, pos, inv_freq, interleaved)


def norm_rope_bwd(x, w, eps, pos, inv_freq, interleaved, dy):
    """(dx, dw)"""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = rotate(dy, pos, inv_freq, interleaved, -1.0)
    n = x * r
    wg = w * g
    return r * (wg - n * (n * wg).mean(-1, keepdims=True)), (g * n).sum((0, 1))


def pair_size(x, inv_freq, interleaved):
    """|x|, and for rotated features the sum of both members' magnitudes: what
    the rounding of a product with a cosine or sine is relative to."""
    m = np.abs(x)
    if inv_freq is not None and len(inv_freq):
        a, b = pairs(2 * len(inv_freq), interleaved)
        m[..., a] = m[..., b] = m[..., a] + m[..., b]
    return m


# ---- decode -------------------------------------------------------------------------
def _branch(q, K, V, scale):
    """Output, its bound and the weights of one softmax; q [128], K, V [n, 128]."""
    s = K @ q * scale
    top = s.max()
    e = np.exp(s - top)
    l = e.sum()
    a = e / l
    n = len(s)
    # Scores: products are exact, the sum of 128 is in fp32 (16 adds a matrix
    # instruction, 8 of them, a step 2^-23 if it truncates); q's smallest
    # features lose 2^-25 of the largest; the scale and the exponential add
    # 2^-21 of the score's size at most.
    size = (np.abs(K) @ np.abs(q)) * abs(scale)
    ds = (size * (32 * 2.0 ** -23 + 2.0 ** -21) +
          2.0 ** -25 * np.abs(q).max() * np.abs(K).sum(1) * abs(scale)).max()
    # Weights: 2^-11 of themselves in fp16, and 2^-25 where they are subnormal,
    # against a sum of 2^5 at least; sums of values in fp32, one rounding a
    # matrix instruction and a few at the joins.
    rel = 2.0 ** -11 + 2 * ds + 2.0 ** -20 + 2.0 ** -23 * (n / 16 + 80)
    av = np.abs(V)
    return a @ V, rel * (a @ av) + n * 2.0 ** -30 * av.max(0)


def decode(q, K, V, lam, form, window=0, norm=None):
    """Output [heads, 128] of one sequence and its bound before the rounding to
    bf16.  q [Hq, 128]; K, V [Hkv, n, 128]; norm = (eps, gain, post_scale)."""
    n = K.shape[1]
    lo = max(0, n - window) if window else 0
    K, V = K[:, lo:], V[:, lo:]
    heads = q.shape[0] // 2 if form == 2 else q.shape[0]
    out, bound = np.zeros((heads, 128)), np.zeros((heads, 128))
    if n == 0:
        return out, bound
    for p in range(heads):
        if form == 2:
            h = 2 * p // (q.shape[0] // K.shape[0])
            o1, b1 = _branch(q[2 * p], K[h], V[h], 128 ** -0.5)
            o2, b2 = _branch(q[2 * p + 1], K[h], V[h], 128 ** -0.5)
        else:
            z = np.zeros(64)
            o1, b1 = _branch(np.concatenate((q[p, :64], z)), K[p], V[p], 0.125)
            o2, b2 = _branch(np.concatenate((z, q[p, 64:])), K[p], V[p], 0.125)
        o = o1 - lam[p] * o2
        e = b1 + abs(lam[p]) * b2 + 2.0 ** -22 * (np.abs(o1) + np.abs(lam[p] * o2))
        if norm is not None:
            eps, gain, post = norm
            r = np.sqrt((o * o).mean() + eps)
            y = o / r * gain * post
            e = e / r * np.abs(gain * post) + np.abs(y) * (np.sqrt((e * e).mean()) / r + 2.0 ** -20)
            o = y
        out[p], bound[p] = o, e
    return out, bound
