"""The operators around the attention kernels, in float64 on the CPU.

Plain NumPy, written from the formulas: norms of query and key heads with the
rotation of positions and their gradient, the 4-bit format and its layout in
a paged cache, the bookkeeping of pages, and attention over such a cache.
Shares no code with the CUDA path.
"""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ------------------------------------------------------ norm and rotation
def rope_table(rows, rot, base=10000.0):
    """fp32 [rows, rot]: cosines, then sines, of position * base^(-2i/rot)."""
    ang = np.arange(rows)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def _rotation(table, positions, d, interleaved):
    """Rotation matrices [..., d, d] of the positions."""
    rot = table.shape[1]
    pos = np.clip(positions, 0, table.shape[0] - 1)
    t = table[pos].astype(np.float64)
    m = np.zeros(pos.shape + (d, d))
    m[..., range(d), range(d)] = 1.0
    for i in range(rot // 2):
        u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = t[..., i], t[..., rot // 2 + i]
        m[..., u, u], m[..., u, v] = c, -s
        m[..., v, u], m[..., v, v] = s, c
    return m


def norm_rope(qkv, H, Hkv, table, positions, qw, kw, eps, interleaved):
    """qkv [B,N,H+2Hkv,d] -> q [B,H,N,d], k, v [B,Hkv,N,d]."""
    x = np.asarray(qkv, np.float64)
    d = x.shape[3]
    m = _rotation(table, positions, d, interleaved)
    out = []
    for part, w in ((x[:, :, :H], qw), (x[:, :, H:H + Hkv], kw)):
        if w is not None:
            part = part / np.sqrt((part ** 2).mean(-1, keepdims=True) + eps)
            part = part * np.asarray(w, np.float64)
        out.append(np.einsum("bnij,bnhj->bhni", m, part))
    return out[0], out[1], x[:, :, H + Hkv:].transpose(0, 2, 1, 3)


def norm_rope_bwd(qkv, H, Hkv, table, positions, qw, kw, eps, interleaved,
                  dq, dk, dv):
    """Gradients (dqkv, dqw, dkw) of norm_rope."""
    x = np.asarray(qkv, np.float64)
    d = x.shape[3]
    m = _rotation(table, positions, d, interleaved)
    parts, dws = [], []
    for part, w, dz in ((x[:, :, :H], qw, dq), (x[:, :, H:H + Hkv], kw, dk)):
        dy = np.einsum("bnij,bhni->bnhj", m, np.asarray(dz, np.float64))
        if w is None:
            parts.append(dy)
            dws.append(None)
            continue
        r = 1.0 / np.sqrt((part ** 2).mean(-1, keepdims=True) + eps)
        dws.append((dy * part * r).sum((0, 1, 2)))
        gw = dy * np.asarray(w, np.float64)
        # d r / d x_i = -r^3 x_i / d
        parts.append(gw * r - part * r ** 3 * (gw * part).sum(
            -1, keepdims=True) / d)
    parts.append(np.asarray(dv, np.float64).transpose(0, 2, 1, 3))
    return np.concatenate(parts, 2), dws[0], dws[1]


# ------------------------------------------------------------ 4-bit format
def _e4m3_grid():
    """The 127 non-negative finite E4M3 values by code."""
    v = []
    for c in range(127):
        e, f = c >> 3, c & 7
        v.append(f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10))
    return np.array(v)


E4M3 = _e4m3_grid()


def nearest_code(x, grid):
    """Index of the nearest value of an ascending grid, ties to the even
    index, saturating.  (Both formats' codes are even where their last bit
    is zero.)"""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    a, b = x - grid[lo], grid[hi] - x
    pick_hi = (b < a) | ((a == b) & (hi % 2 == 0))
    return np.where(pick_hi, hi, lo)


def quantise(x, g):
    """Codes [..., d] (sign in bit 3) and scale codes [..., d/16]."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[:-1] + (-1, 16))
    amax = np.abs(b).max(-1)
    nan = np.isnan(amax)
    s = np.where(nan, 127, nearest_code(
        np.where(nan, 0, np.minimum(amax / 6 / g, 1e9)), E4M3))
    scale = np.where(nan, 0, E4M3[np.minimum(s, 126)])[..., None] * g
    none = scale == 0
    q = np.where(none, 0.0, b / np.where(none, 1.0, scale))
    c = nearest_code(np.minimum(np.abs(q), 1e9), E2M1)
    c = np.where(np.isnan(q), 0, c + 8 * np.signbit(q))
    return c.reshape(x.shape).astype(np.uint8), s.astype(np.uint8)


def dequantise(codes, scales, g):
    c = codes.astype(int)
    v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    mag = scales & 127                    # (a scale written here has no sign)
    s = np.where(mag == 127, np.nan, E4M3[np.minimum(mag, 126)])
    s = s * np.where(scales & 128, -1.0, 1.0) * g
    return (v.reshape(v.shape[:-1] + (-1, 16)) * s[..., None]).reshape(v.shape)


def _places(d, tok):
    """Byte offsets in a group, by dim pair (codes) and block (scales)."""
    pair, blk = np.arange(d // 2), np.arange(d // 16)
    per = d // 16
    k = tok * (d // 2) + pair
    ks = 8 * d + tok * per + blk
    v = 9 * d + ((((tok // 8) * 8 + pair // per) * 4 + tok % 8 // 2) * 2
                 + tok % 2) * per + pair % per
    vs = 17 * d + (((tok // 8) * per + blk) * 4 + tok % 8 // 2) * 2 + tok % 2
    return k, ks, v, vs


def cache_write(cache, slot, head, k, v, gk, gv):
    """One token of one head into cache uint8 [pages,Hkv,page/16,18d]."""
    per, d = cache.shape[2], cache.shape[3] // 18
    grp = cache[slot // (16 * per), head, slot % (16 * per) // 16]
    ka, ksa, va, vsa = _places(d, slot % 16)
    for x, g, at, sat in ((k, gk, ka, ksa), (v, gv, va, vsa)):
        c, s = quantise(x, g)
        grp[at] = c[0::2] | (c[1::2] << 4)
        grp[sat] = s


def cache_values(cache, gk, gv):
    """All keys and values, float64 [pages, Hkv, page_size, d] each."""
    pages, Hkv, per, width = cache.shape
    d = width // 18
    k = np.empty((pages, Hkv, per, 16, d))
    v = np.empty_like(k)
    for tok in range(16):
        ka, ksa, va, vsa = _places(d, tok)
        for out, g, at, sat in ((k, gk, ka, ksa), (v, gv, va, vsa)):
            b = cache[..., at]
            c = np.stack([b & 15, b >> 4], -1).reshape(pages, Hkv, per, d)
            out[..., tok, :] = dequantise(c, cache[..., sat], g)
    return (k.reshape(pages, Hkv, 16 * per, d),
            v.reshape(pages, Hkv, 16 * per, d))


# ------------------------------------------------------------- bookkeeping
def plan(new, lens, table, free, page, T):
    """One step, request by request, on Python lists (changed in place);
    `free` is the stack's used part.  Returns slots, positions, granted."""
    R, M = len(lens), len(table[0]) if table else 0
    pages = lambda n: -(-n // page)  # noqa: E731
    for r in reversed(range(R)):
        if new[r] < 0:
            after = max(0, lens[r] + new[r])
            for i in reversed(range(pages(after), pages(lens[r]))):
                free.append(table[r][i])
            lens[r] = after
    slots = [[-1] * T for _ in range(R)]
    pos = [[0] * T for _ in range(R)]
    granted = [0] * R
    start, wanted = len(free), 0
    for r in range(R):
        n = new[r]
        if n <= 0 or n > T or lens[r] + n > M * page:
            continue
        need = pages(lens[r] + n) - pages(lens[r])
        wanted += need
        if need and wanted > start:
            continue
        for i in range(need):
            table[r][pages(lens[r]) + i] = free.pop()
        for t in range(n):
            p = lens[r] + t
            slots[r][t] = table[r][p // page] * page + p % page
            pos[r][t] = p
        lens[r] += n
        granted[r] = n
    return slots, pos, granted


# --------------------------------------------------------------- attention
def cache_attention(q, cache, table, lens, q_lens, scale, window, gk, gv):
    """o [B,H,T,d], lse [B,H,T]; NaN in rows past a request's new tokens."""
    q = np.asarray(q, np.float64)
    B, H, T, d = q.shape
    pages, Hkv, per, _ = cache.shape
    page = 16 * per
    all_k, all_v = cache_values(cache, gk, gv)
    o = np.full(q.shape, np.nan)
    lse = np.full((B, H, T), np.nan)
    for b in range(B):
        L = min(max(int(lens[b]), 0), len(table[b]) * page)
        n = T if q_lens is None else min(max(int(q_lens[b]), 0), T)
        j = np.arange(L)
        pg = np.asarray(table[b], int)[j // page] if L else j
        ok = (pg >= 0) & (pg < pages)
        at, pg = j[ok], pg[ok]
        for h in range(H):
            K = all_k[pg, h // (H // Hkv), at % page]
            V = all_v[pg, h // (H // Hkv), at % page]
            for t in range(n):
                i = L - n + t
                see = at <= i
                if window >= 0:
                    see &= at >= i - window
                if not see.any():
                    o[b, h, t], lse[b, h, t] = 0.0, -np.inf
                    continue
                s = K[see] @ q[b, h, t] * scale
                m = s.max()
                p = np.exp(s - m)
                o[b, h, t] = p @ V[see] / p.sum()
                lse[b, h, t] = m + np.log(p.sum())
    return o, lse
