"""The paged cache held in 8 bits, in float64 on the CPU.

Plain NumPy, written from the definition: a value is an E4M3 code times a
power of two that 16 tokens of a head share.  Shares no code with the CUDA
path.
"""
import numpy as np

from .serve import E4M3, nearest_code

MOST = 60                                  # exponents lie within -60 .. 60


def exponent(amax):
    """The smallest e with amax <= 448 2^e."""
    e = -MOST
    while e < MOST and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def encode(x, e):
    """E4M3 bytes of x / 2^e: nearest, ties to even, saturating."""
    x = np.asarray(x, np.float64)
    nan = np.isnan(x)
    mag = np.where(nan, 0, np.minimum(np.abs(x), 1e300)) * 2.0 ** -e
    c = np.where(nan, 127, nearest_code(mag, E4M3))
    return (c + 128 * (np.signbit(x) & ~nan)).astype(np.uint8)


def decode(codes, e):
    mag = (codes & 127).astype(int)
    v = np.where(mag == 127, np.nan, E4M3[np.minimum(mag, 126)])
    return np.where(codes & 128, -v, v) * 2.0 ** np.asarray(e, np.float64)


def places(d, tok):
    """Byte offsets in a group of a token's key and value codes."""
    dim = np.arange(d)
    k = np.ravel_multi_index(
        (tok // 8 + 0 * dim, dim // 64, tok % 8 + 0 * dim, dim % 32 // 8,
         dim % 64 // 32, dim % 8), (2, d // 64, 8, 4, 2, 8))
    v = np.ravel_multi_index(
        (dim // 64, tok // 8 + 0 * dim, dim % 64 // 8, tok % 8 // 2 + 0 * dim,
         dim % 8, tok % 2 + 0 * dim), (d // 64, 2, 8, 4, 8, 2))
    return k, 16 * d + v


def append(cache, slots, k, v):
    """One call on cache uint8 [pages,Hkv,page/16,32d+16] (in place), k, v
    [B,Hkv,N,d], slots [B,N].  Returns the values held, NaN where skipped."""
    pages, Hkv, per, width = cache.shape
    d = (width - 16) // 32
    groups = {}
    for (b, n), s in np.ndenumerate(slots):
        if 0 <= s < pages * per * 16:
            groups.setdefault(int(s) // 16, {})[int(s) % 16] = (b, n)
    held = [np.full(np.shape(x), np.nan) for x in (k, v)]
    for gid, toks in groups.items():
        for h in range(Hkv):
            grp = cache[gid // per, h, gid % per]
            for which, x in enumerate((k, v)):
                at = [places(d, t)[which] for t in range(16)]
                rows = {t: np.asarray(x[b, h, n], np.float64) for t, (b, n) in toks.items()}
                amax = max((np.abs(r[np.isfinite(r)]).max(initial=0.0) for r in rows.values()))
                e = exponent(amax)
                old = int(np.clip(grp[32 * d + which].astype(np.int8), -MOST, MOST))
                if 0 not in toks:
                    e = max(e, old)
                    if e > old:
                        for t in range(16):
                            if t not in toks:
                                grp[at[t]] = encode(decode(grp[at[t]], old), e)
                for t, r in rows.items():
                    grp[at[t]] = encode(r, e)
                    held[which][toks[t][0], h, toks[t][1]] = decode(grp[at[t]], e)
                grp[32 * d + which] = np.int8(e).astype(np.uint8)
    return held


def values(cache):
    """All keys and values, float64 [pages, Hkv, page_size, d] each."""
    pages, Hkv, per, width = cache.shape
    d = (width - 16) // 32
    out = []
    for which in (0, 1):
        e = np.clip(cache[..., 32 * d + which].astype(np.int8), -MOST, MOST)
        x = np.stack([decode(cache[..., places(d, t)[which]], e[..., None])
                      for t in range(16)], -2)
        out.append(x.reshape(pages, Hkv, 16 * per, d))
    return out


def read(cache, table, lens, starts, N):
    """k, v [B,Hkv,N,d], NaN in rows that are not written, and which are."""
    pages, Hkv, per, width = cache.shape
    page, B = 16 * per, len(table)
    all_k, all_v = values(cache)
    k = np.full((B, Hkv, N, (width - 16) // 32), np.nan)
    v = np.full(k.shape, np.nan)
    done = np.zeros((B, N), bool)
    for b in range(B):
        cap = len(table[b]) * page
        L = min(max(int(lens[b]), 0), cap)
        lo = min(max(int(starts[b]), 0), cap) if starts is not None else 0
        for n in range(min(N, max(0, L - lo))):
            pg = int(table[b][(lo + n) // page])
            if 0 <= pg < pages:
                k[b, :, n], v[b, :, n] = all_k[pg, :, (lo + n) % page], all_v[pg, :, (lo + n) % page]
                done[b, n] = True
    return k, v, done


def attention(q, cache, table, lens, q_lens, scale, window):
    """o [B,H,T,d], lse [B,H,T], NaN in rows past a request's new tokens; the
    third: sum of weight times magnitude of the values, per element of o."""
    q = np.asarray(q, np.float64)
    B, H, T, d = q.shape
    pages, Hkv, per, _ = cache.shape
    page = 16 * per
    all_k, all_v = values(cache)
    o, mag = np.full(q.shape, np.nan), np.zeros(q.shape)
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
                mag[b, h, t] = p @ np.abs(V[see]) / p.sum()
                lse[b, h, t] = m + np.log(p.sum())
    return o, lse, mag


def products(q, cache, table, lens, q_lens, scale, window):
    """The same with what bounds its rounding, a matrix product per request and
    head: o, lse and mag as attention()'s, top [B,H,T]: the largest
    weight times its value's power of two, and few [B,H,T]: how many keys that
    the row sees have less than 2^-22 of that."""
    q = np.asarray(q, np.float64)
    B, H, T, d = q.shape
    pages, Hkv, per, _ = cache.shape
    page = 16 * per
    all_k, all_v = values(cache)
    unit = 2.0 ** np.clip(cache[..., 32 * d + 1].astype(np.int8), -MOST, MOST).astype(np.float64)
    unit = unit.repeat(16, -1)             # [pages, Hkv, page_size]
    o, mag = np.full(q.shape, np.nan), np.zeros(q.shape)
    lse, top, few = np.full((B, H, T), np.nan), np.zeros((B, H, T)), np.zeros((B, H, T))
    for b in range(B):
        L = min(max(int(lens[b]), 0), len(table[b]) * page)
        n = T if q_lens is None else min(max(int(q_lens[b]), 0), T)
        j = np.arange(L)
        pg = np.asarray(table[b], int)[j // page] if L else j
        ok = (pg >= 0) & (pg < pages)
        at, pg = j[ok], pg[ok]
        i = L - n + np.arange(n)[:, None]
        see = at <= i
        if window >= 0:
            see &= at >= i - window
        some = see.any(1)
        for h in range(H):
            hk = h // (H // Hkv)
            K, V, u = (x[pg, hk, at % page] for x in (all_k, all_v, unit))
            V = np.where(see.any(0)[:, None], V, 0)
            s = np.where(see, q[b, h, :n] @ np.where(see.any(0)[:, None], K, 0).T * scale, -np.inf)
            m = np.where(some, s.max(1, initial=-np.inf), 0)[:, None]
            p = np.exp(s - m)
            l = p.sum(1)
            p /= np.where(some, l, 1)[:, None]
            o[b, h, :n], mag[b, h, :n] = p @ V, p @ np.abs(V)
            with np.errstate(divide="ignore"):
                lse[b, h, :n] = m[:, 0] + np.log(l)
            top[b, h, :n] = (p * u).max(1, initial=0)
            few[b, h, :n] = (see & (p * u < top[b, h, :n, None] * 2.0 ** -22)).sum(1)
    return o, lse, mag, top, few
