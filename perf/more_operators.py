"""The 8-bit cache and the rotation with several axes, as cases.

  rope, rope_bwd  norms of the query and key heads with a rotation whose pairs
                  turn by the token's place on one of several axes (time,
                  height, width), from a projection's output to the
                  attention's layout, and the gradient of that
  append          new keys and values into a paged cache held in 8 bits, with
                  a scale for each block of 16 tokens and head
  read            tokens of that cache back into the attention's layout
  attn            attention of new tokens over that cache

``run`` computes a case in elementary torch operations, or, where ``own`` is
set, by the library's calls.  ``exact`` computes it once more in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # One decode step of 32 requests of a model with three axes: latency.
        {"name": "rope_decode_32x1", "op": "rope", "B": 32, "N": 1, "H": 32, "Hkv": 8, "d": 128, "rot": 128, "axes": 3, "alternate": False, "norm": True, "interleaved": False},
        # Prompts of images and text, the headline shape's query heads, odd length.
        {"name": "rope_images_3x5001", "op": "rope", "B": 3, "N": 5001, "H": 64, "Hkv": 8, "d": 128, "rot": 128, "axes": 3, "alternate": False, "norm": True, "interleaved": False},
        # Backward of a medium training step.
        {"name": "rope_bwd_4x1024", "op": "rope_bwd", "B": 4, "N": 1024, "H": 32, "Hkv": 32, "d": 128, "rot": 128, "axes": 3, "alternate": False, "norm": True, "interleaved": False},
        # Backward of long ragged rows, small heads, axes taken in turn by neighbouring pairs.
        {"name": "rope_bwd_7x3001_d64", "op": "rope_bwd", "B": 7, "N": 3001, "H": 24, "Hkv": 8, "d": 64, "rot": 64, "axes": 3, "alternate": True, "norm": True, "interleaved": False},
        # One new token for each of 128 requests, most of them into a block that holds some.
        {"name": "append_decode_128", "op": "append", "B": 128, "N": 1, "Hkv": 8, "d": 128, "page": 64},
        # Prompts written to the cache.
        {"name": "append_prompt_8x4000", "op": "append", "B": 8, "N": 4000, "Hkv": 8, "d": 128, "page": 64},
        # A short prefix taken back from the cache: latency.
        {"name": "read_one_1x700_d64", "op": "read", "B": 1, "N": 700, "Hkv": 8, "d": 64, "page": 16, "len_min": 700, "len_max": 700},
        # Prefixes of a batch taken back, to run a bf16 pass over them.
        {"name": "read_batch_12x6000", "op": "read", "B": 12, "N": 6000, "Hkv": 8, "d": 128, "page": 64, "len_min": 3000, "len_max": 6500},
        # One request with a short history: latency.
        {"name": "attn_one_1x900_d64", "op": "attn", "B": 1, "T": 1, "H": 16, "Hkv": 16, "d": 64, "page": 16, "len_min": 900, "len_max": 900, "window": -1},
        # A full decode batch with ragged histories.
        {"name": "attn_batch_64x8192", "op": "attn", "B": 64, "T": 1, "H": 64, "Hkv": 8, "d": 128, "page": 64, "len_min": 100, "len_max": 8192, "window": -1},
        # Few requests with long histories.
        {"name": "attn_long_3x131072", "op": "attn", "B": 3, "T": 1, "H": 32, "Hkv": 8, "d": 128, "page": 128, "len_min": 100000, "len_max": 131072, "window": -1},
        # Chunks of two prompts over what the cache holds of them already.
        {"name": "attn_chunk_2x512", "op": "attn", "B": 2, "T": 512, "H": 64, "Hkv": 8, "d": 128, "page": 64, "len_min": 5000, "len_max": 16384, "window": -1},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _heads(rng, most):
    Hkv = rng.choice([1, 2, 4, 8, 16])
    return min(most, Hkv * rng.choice([1, 2, 3, 4, 7, 8])) // Hkv * Hkv, Hkv


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "read", "attn", "attn"])
    d = rng.choice([64, 128, 128])
    if op in ("rope", "rope_bwd"):
        H, Hkv = _heads(rng, 64)
        tokens = _spread(rng, 1, 12288 if op == "rope" else 8192)
        B = _spread(rng, 1, min(64, tokens))
        return {"op": op, "B": B, "N": max(1, tokens // B), "H": H, "Hkv": Hkv, "d": d, "rot": rng.choice([d, d, d // 2]),
                "axes": rng.choice([2, 3, 3, 4]), "alternate": rng.random() < 0.4, "norm": rng.random() < 0.8,
                "interleaved": rng.random() < 0.4}
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        tokens = _spread(rng, 1, 32000)
        B = _spread(rng, 1, min(256, tokens))
        return {"op": op, "B": B, "N": max(1, tokens // B), "Hkv": rng.choice([1, 2, 4, 8]), "d": d, "page": page}
    if op == "read":
        tokens = _spread(rng, 1, 50000)
        B = _spread(rng, 1, min(64, tokens))
        N = max(1, tokens // B)
        return {"op": op, "B": B, "N": N, "Hkv": rng.choice([1, 2, 4, 8]), "d": d, "page": page, "len_min": N // 2, "len_max": N + N // 8}
    H, Hkv = _heads(rng, 64)
    T = rng.choice([1, 1, 1, rng.randint(2, 9), _spread(rng, 10, 512)])
    budget = min(3 * 100000 * 8 // Hkv, int(8e10 / (4 * H * d * T)))
    hi = _spread(rng, 1, min(131072, budget))
    B = _spread(rng, 1, max(1, min(128, budget // hi, 32768 // T)))
    return {"op": op, "B": B, "T": T, "H": H, "Hkv": Hkv, "d": d, "page": page, "len_min": max(0, hi // rng.choice([1, 2, 50])),
            "len_max": hi, "window": rng.choice([-1, -1, -1, hi // 3])}


def _lengths(n, lo, hi):
    """n whole numbers from hi down to lo, evenly spread."""
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _axis_of_pairs(case):
    """Axis of each rotated pair: sections, the first one of a quarter of the
    pairs where there are three axes and more, or the axes in turn."""
    half, n = case["rot"] // 2, case["axes"]
    if case["alternate"]:
        return [i % n for i in range(half)]
    first = half // 4 if n > 2 else half // n
    rest = half - first
    return [0] * first + [1 + i * (n - 1) // rest for i in range(rest)]


# ----------------------------------------------------- the 8-bit format, plain
# 16 tokens of one key/value head are one group of 32 d + 16 bytes:
#   K codes [2][d/64][8][4][2][8]  (token / 8, dim / 64, token % 8,
#                                   dim % 32 / 8, dim % 64 / 32, dim % 8)
#   V codes [d/64][2][8][4][8][2]  (dim / 64, token / 8, dim % 64 / 8,
#                                   token % 8 / 2, dim % 8, token % 2)
#   K's exponent, V's exponent (signed bytes), 14 bytes that nothing uses
# A code is E4M3 of value / 2^exponent.
EXP = 60  # exponents lie within -EXP .. EXP


def _exponent(amax):
    """Smallest e with amax <= 448 2^e (448 is 0.875 2^9)."""
    m, x = torch.frexp(amax)
    e = torch.where(m > 0.875, x - 8, x - 9)
    return torch.where(amax > 0, e, -EXP).clamp(-EXP, EXP)


def _pow2(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _code(x, e):
    """E4M3 bytes of fp32 x / 2^e."""
    return (x * _pow2(-e)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _value(c, e):
    return c.contiguous().view(torch.float8_e4m3fn).float() * _pow2(e)


def _k_bytes(c):
    """Bytes [..., 16 d] of key codes [..., 16, d]."""
    n, d = c.dim() - 2, c.shape[-1]
    c = c.reshape(*c.shape[:n], 2, 8, d // 64, 2, 4, 8)
    return c.permute(*range(n), n, n + 2, n + 1, n + 4, n + 3, n + 5).flatten(n)


def _v_bytes(c):
    n, d = c.dim() - 2, c.shape[-1]
    c = c.reshape(*c.shape[:n], 2, 4, 2, d // 64, 8, 8)
    return c.permute(*range(n), n + 3, n, n + 4, n + 1, n + 5, n + 2).flatten(n)


def _k_codes(b, d):
    """Key codes [..., 16, d] of bytes [..., 16 d]."""
    n = b.dim() - 1
    b = b.reshape(*b.shape[:n], 2, d // 64, 8, 4, 2, 8)
    return b.permute(*range(n), n, n + 2, n + 1, n + 4, n + 3, n + 5).reshape(*b.shape[:n], 16, d)


def _v_codes(b, d):
    n = b.dim() - 1
    b = b.reshape(*b.shape[:n], d // 64, 2, 8, 4, 8, 2)
    return b.permute(*range(n), n + 1, n + 3, n + 5, n, n + 2, n + 4).reshape(*b.shape[:n], 16, d)


def _groups(k, v):
    """Group bytes [..., 32 d + 16] of fp32 keys and values [..., 16, d]."""
    ke, ve = _exponent(k.abs().amax((-1, -2))), _exponent(v.abs().amax((-1, -2)))
    head = torch.zeros(*ke.shape, 16, dtype=torch.uint8, device=k.device)
    head[..., 0], head[..., 1] = ke.to(torch.int8).view(torch.uint8), ve.to(torch.int8).view(torch.uint8)
    return torch.cat([_k_bytes(_code(k, ke[..., None, None])), _v_bytes(_code(v, ve[..., None, None])), head], -1)


def _ungroup(grp):
    """fp32 keys and values [..., 16, d] of group bytes."""
    d = (grp.shape[-1] - 16) // 32
    e = grp[..., 32 * d:32 * d + 2].contiguous().view(torch.int8).int()
    return (_value(_k_codes(grp[..., :16 * d], d), e[..., 0, None, None]),
            _value(_v_codes(grp[..., 16 * d:32 * d], d), e[..., 1, None, None]))


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))

    def normal(*shape, dtype=torch.bfloat16, mult=1.0):
        return (torch.randn(shape, generator=gen, device=DEV) * mult).to(dtype)

    def tokens(*shape, dtype=torch.bfloat16, mult=1.0):
        """Rows whose sizes differ, with a few large dims."""
        x = torch.randn(shape, generator=gen, device=DEV) * mult
        x *= torch.exp2(0.7 * torch.randn((*shape[:-1], 1), generator=gen, device=DEV))
        x[..., ::37] *= 3.0
        return x.to(dtype)

    def shuffled(n):
        return torch.randperm(n, generator=gen, device=DEV).to(torch.int32)

    s = {"op": case["op"]}
    if case["op"] in ("rope", "rope_bwd"):
        B, N, H, Hkv, d, rot, A = (case[x] for x in ("B", "N", "H", "Hkv", "d", "rot", "axes"))
        s.update(H=H, Hkv=Hkv, eps=1e-6, interleaved=case["interleaved"], axes=bytes(_axis_of_pairs(case)))
        s["axis"] = torch.tensor(list(s["axes"]), device=DEV)
        s["qkv"] = normal(B, N, H + 2 * Hkv, d)
        P = 32768
        freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
        ang = torch.arange(P, dtype=torch.float64, device=DEV)[:, None] * freq
        s["rope"] = torch.cat([ang.cos(), ang.sin()], -1).float()
        # Text, whose tokens have the same place on every axis, then an image
        # of its own width in each entry, row by row.
        start = torch.randint(0, P - N - 1, (B, 1), generator=gen, device=DEV)
        width = torch.randint(7, 64, (B, 1), generator=gen, device=DEV)
        n = torch.arange(N, device=DEV)[None]
        text = N // 3
        i = (n - text).clamp(min=0)
        place = [start + torch.where(n < text, n, text + x) for x in (0 * i, i // width, i % width, i // 2)]
        s["positions"] = torch.stack(place[:A]).to(torch.int32).contiguous()
        s["q_weight"] = 1 + normal(d, dtype=torch.float32, mult=0.1) if case["norm"] else None
        s["k_weight"] = 1 + normal(d, dtype=torch.float32, mult=0.1) if case["norm"] else None
        if case["op"] == "rope_bwd":
            s["dq"], s["dk"], s["dv"] = normal(B, H, N, d), normal(B, Hkv, N, d), normal(B, Hkv, N, d)
    elif case["op"] == "append":
        B, N, Hkv, d, page = (case[x] for x in ("B", "N", "Hkv", "d", "page"))
        s["k"], s["v"] = tokens(B, Hkv, N, d, mult=1.5), tokens(B, Hkv, N, d, mult=0.7)
        per = -(-N // page) + 1
        pages = B * per + 3
        ids = shuffled(pages)
        new = torch.tensor(_lengths(B, (N + 1) // 2, N), dtype=torch.int32, device=DEV)[shuffled(B).long()]
        start = torch.randint(0, page, (B, 1), generator=gen, device=DEV)
        t = torch.arange(N, device=DEV)[None]
        pos = start + t
        slot = ids[torch.arange(B, device=DEV)[:, None] * per + pos // page] * page + pos % page
        s["slots"] = torch.where(t < new[:, None], slot, -1).to(torch.int32)
        # A cache that has been in use: the blocks hold earlier tokens.
        s["cache"] = _groups(tokens(pages, Hkv, page // 16, 16, d, dtype=torch.float32),
                             tokens(pages, Hkv, page // 16, 16, d, dtype=torch.float32, mult=0.5))
        s["k_out"], s["v_out"] = torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
    else:
        B, Hkv, d, page = (case[x] for x in ("B", "Hkv", "d", "page"))
        lens = _lengths(B, case["len_min"], case["len_max"])
        at = shuffled(B).long()
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)[at]
        blocks = -(-case["len_max"] // page)
        have = (s["seq_lens"] + page - 1) // page
        pages = sum(-(-n // page) for n in lens) + 5
        ids = shuffled(pages)
        i = torch.arange(max(1, blocks), device=DEV)[None]
        off = (have.cumsum(0) - have)[:, None]
        s["block_table"] = torch.where(i < have[:, None], ids[(off + i).clamp(max=pages - 1)], -1).to(torch.int32)
        s["cache"] = torch.cat([_groups(tokens(n, Hkv, page // 16, 16, d, dtype=torch.float32, mult=1.2),
                                        tokens(n, Hkv, page // 16, 16, d, dtype=torch.float32, mult=0.7))
                                for n in [1024] * (pages // 1024) + [pages % 1024] if n])
        if case["op"] == "read":
            N = case["N"]
            s["N"] = N
            # From some way into the longer requests on.
            s["starts"] = ((s["seq_lens"] - N).clamp(min=0) // 2).to(torch.int32)
            s["k_out"] = torch.zeros((B, Hkv, N, d), dtype=torch.bfloat16, device=DEV)
            s["v_out"] = torch.zeros_like(s["k_out"])
        else:
            T, H = case["T"], case["H"]
            s["q_lens"] = None if T == 1 else torch.tensor(_lengths(B, (T + 1) // 2, T), dtype=torch.int32, device=DEV)[at.flip(0)]
            s["q"] = normal(B, H, T, d, mult=1.5)
            s.update(scale=1.0 / math.sqrt(d), window=case["window"])
            # Buffers that a program keeps; rows past a request's new tokens stay.
            s["out"] = torch.zeros_like(s["q"])
            s["lse"] = torch.zeros((B, H, T), dtype=torch.float32, device=DEV)
    return s


# ------------------------------------------------------------ the library's calls
def _run_own(s):
    import tiled_attention_bwd_gb300 as fa
    if s["op"] == "rope":
        q, k, v = fa.fa_qk_norm_rope_axes(s["qkv"], s["H"], s["Hkv"], s["rope"], s["positions"], s["axes"], s["q_weight"],
                                          s["k_weight"], eps=s["eps"], interleaved=s["interleaved"])
        return {"q": q, "k": k, "v": v}
    if s["op"] == "rope_bwd":
        dqkv, dqw, dkw = fa.fa_qk_norm_rope_axes_bwd(s["qkv"], s["H"], s["Hkv"], s["rope"], s["dq"], s["dk"], s["dv"], s["positions"],
                                                     s["axes"], s["q_weight"], s["k_weight"], eps=s["eps"],
                                                     interleaved=s["interleaved"])
        return {"dqkv": dqkv, "dqw": dqw, "dkw": dkw}
    if s["op"] == "append":
        fa.fa_cache8_append(s["k"], s["v"], s["cache"], s["slots"], k_out=s["k_out"], v_out=s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"], "cache": s["cache"]}
    if s["op"] == "read":
        k, v = fa.fa_cache8_read(s["cache"], s["block_table"], s["seq_lens"], s["N"], starts=s["starts"], k_out=s["k_out"],
                                 v_out=s["v_out"])
        return {"k": k, "v": v}
    o, lse = fa.fa_cache8_attn(s["q"], s["cache"], s["block_table"], s["seq_lens"], s["scale"], q_lens=s["q_lens"],
                               window=s["window"], out=s["out"], lse=s["lse"])
    return {"o": o, "lse": lse}


# -------------------------------------------------------------- the plain forms
def _turned(x, c, n, interleaved, back=False):
    """x [B,N,h,d] with its first 2 * c.shape[-1] dims rotated."""
    r = 2 * c.shape[-1]
    c, n = c[:, :, None], (-n if back else n)[:, :, None]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    y = (a * c - b * n, b * c + a * n)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat([y, x[..., r:]], -1)


def _angles(s):
    """Cosines and sines [B,N,rot/2] of every pair's own axis."""
    half = s["rope"].shape[1] // 2
    at = s["positions"].long()[s["axis"]].permute(1, 2, 0)  # [B,N,half]
    i = torch.arange(half, device=at.device)
    return s["rope"][at, i], s["rope"][at, half + i]


def _plain_rope(s):
    H, Hkv = s["H"], s["Hkv"]
    x = s["qkv"].float()
    c, n = _angles(s)
    q, k, v = x[:, :, :H], x[:, :, H:H + Hkv], x[:, :, H + Hkv:]
    if s["q_weight"] is not None:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + s["eps"]) * s["q_weight"]
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + s["eps"]) * s["k_weight"]
    q, k = _turned(q, c, n, s["interleaved"]), _turned(k, c, n, s["interleaved"])
    return {"q": q.transpose(1, 2).to(torch.bfloat16).contiguous(), "k": k.transpose(1, 2).to(torch.bfloat16).contiguous(),
            "v": v.transpose(1, 2).to(torch.bfloat16).contiguous()}


def _plain_rope_bwd(s):
    H, Hkv = s["H"], s["Hkv"]
    x = s["qkv"].float()
    c, n = _angles(s)

    def one(x, dz, w):
        dy = _turned(dz.float().transpose(1, 2), c, n, s["interleaved"], back=True)
        if w is None:
            return dy, None
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
        xh = x * r
        g = dy * w
        return r * (g - xh * (g * xh).mean(-1, keepdim=True)), (dy * xh).sum((0, 1, 2))

    dq, dqw = one(x[:, :, :H], s["dq"], s["q_weight"])
    dk, dkw = one(x[:, :, H:H + Hkv], s["dk"], s["k_weight"])
    d = torch.cat([dq, dk, s["dv"].float().transpose(1, 2)], 2).to(torch.bfloat16)
    return {"dqkv": d, "dqw": dqw, "dkw": dkw}


def _plain_append(s):
    cache, slots = s["cache"], s["slots"]
    pages, Hkv, per, d = cache.shape[0], cache.shape[1], cache.shape[2], (cache.shape[3] - 16) // 32
    ok = slots >= 0
    at = slots[ok].long()
    used, idx = torch.unique(at // 16, return_inverse=True)   # groups that get tokens
    place = at % 16
    fresh = torch.zeros(used.numel(), dtype=torch.bool, device=at.device)
    fresh[idx[place == 0]] = True
    grp = cache.transpose(1, 2).reshape(pages * per, Hkv, -1)[used]  # [n,Hkv,32d+16]
    old = grp[..., 32 * d:32 * d + 2].contiguous().view(torch.int8).int()
    written = torch.zeros(used.numel(), 16, dtype=torch.bool, device=at.device)
    written[idx, place] = True
    res = []
    for which, (x, codes, to_bytes, out) in enumerate(((s["k"], _k_codes, _k_bytes, s["k_out"]), (s["v"], _v_codes, _v_bytes, s["v_out"]))):
        x = x.transpose(1, 2)[ok].float()                     # [tokens,Hkv,d]
        amax = torch.where(x.isfinite(), x.abs(), torch.zeros_like(x)).amax(-1)
        need = torch.full((used.numel(), Hkv), -EXP, dtype=torch.int32, device=at.device)
        need = need.scatter_reduce(0, idx[:, None].expand(-1, Hkv), _exponent(amax), "amax")
        e = torch.where(fresh[:, None], need, torch.maximum(old[..., which], need))
        c = codes(grp[..., which * 16 * d:(which + 1) * 16 * d], d)
        grown = _code(_value(c, old[..., which, None, None] - e[..., None, None]), torch.zeros_like(e)[..., None, None])
        keep = fresh[:, None, None, None] | (old[..., which] == e)[..., None, None]
        c = torch.where(keep, c, grown)
        mine = e[idx][..., None]
        fine = _code(x, mine)
        c[idx, :, place] = fine
        grp[..., which * 16 * d:(which + 1) * 16 * d] = to_bytes(c)
        grp[..., 32 * d + which] = e.to(torch.int8).view(torch.uint8)
        rows = out.transpose(1, 2)
        rows[ok] = _value(fine, mine).to(torch.bfloat16)
        res.append(out)
    cache.transpose(1, 2)[used // per, used % per] = grp
    return {"k": res[0], "v": res[1], "cache": cache}


def _plain_cache(s):
    """fp32 keys and values [B,Hkv,L,d] of the block tables' pages."""
    grp = s["cache"][s["block_table"].clamp(min=0).long()].transpose(1, 2)  # [B,Hkv,M,page/16,32d+16]
    k, v = _ungroup(grp)
    return k.flatten(2, 4), v.flatten(2, 4)


def _plain_read(s):
    k, v = _plain_cache(s)
    B, Hkv, L, d = k.shape
    at = s["starts"][:, None] + torch.arange(s["N"], device=k.device)
    have = (at < s["seq_lens"][:, None])[:, None, :, None]
    at = at.clamp(max=L - 1).long()[:, None, :, None].expand(-1, Hkv, -1, d)
    for x, out in ((k, s["k_out"]), (v, s["v_out"])):
        out.copy_(torch.where(have, x.gather(2, at).to(torch.bfloat16), out))
    return {"k": s["k_out"], "v": s["v_out"]}


def _plain_attn(s):
    q = s["q"]
    B, H, T, d = q.shape
    k, v = _plain_cache(s)
    Hkv, L = k.shape[1], k.shape[2]
    ql = torch.full((B,), T, device=q.device) if s["q_lens"] is None else s["q_lens"]
    t = torch.arange(T, device=q.device)
    i = (s["seq_lens"] - ql)[:, None] + t                   # the row's position
    j = torch.arange(L, device=q.device)
    see = (j <= i[..., None]) & (j < s["seq_lens"][:, None, None])
    if s["window"] >= 0:
        see = see & (j >= i[..., None] - s["window"])
    x = (q.float().view(B, Hkv, -1, d) @ k.transpose(-1, -2)).view(B, Hkv, -1, T, L) * s["scale"]
    x = x.masked_fill(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, -1, L) @ v).view(B, Hkv, -1, T, d) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + torch.log(l)).view(B, H, T)
    row = (t < ql[:, None])[:, None]
    s["out"].copy_(torch.where(row[..., None], o.view(B, H, T, d).to(torch.bfloat16), s["out"]))
    s["lse"].copy_(torch.where(row, lse, s["lse"]))
    return {"o": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _plain_rope, "rope_bwd": _plain_rope_bwd, "append": _plain_append, "read": _plain_read,
            "attn": _plain_attn}[state["op"]](state)


# ------------------------------------------------------------------ what it costs
def work(case):
    op = case["op"]
    if op in ("rope", "rope_bwd"):
        rows, H, Hkv, d = case["B"] * case["N"], case["H"], case["Hkv"], case["d"]
        all_ = rows * (H + 2 * Hkv) * d
        side = rows * 4 * case["axes"] + min(rows, 32768) * case["rot"] * 4
        if op == "rope":
            return {"bytes": 4 * all_ + side, "flops": 8 * rows * (H + Hkv) * d}
        x = 2 * rows * (H + Hkv) * d if case["norm"] else 0
        return {"bytes": 4 * all_ + x + side, "flops": 16 * rows * (H + Hkv) * d}
    d, Hkv = case["d"], case["Hkv"]
    if op == "append":
        rows = sum(_lengths(case["B"], (case["N"] + 1) // 2, case["N"])) * Hkv
        return {"bytes": rows * (4 * d + 4 * d + 2 * d) + rows // 16 * 2 + case["B"] * case["N"] * 4, "flops": 4 * rows * d}
    lens = _lengths(case["B"], case["len_min"], case["len_max"])
    if op == "read":
        N = case["N"]
        rows = sum(min(N, n - max(0, n - N) // 2) for n in lens) * Hkv
        return {"bytes": rows * (2 * d + 4 * d) + rows // 16 * 2, "flops": 2 * rows * d}
    B, T, H = case["B"], case["T"], case["H"]
    rows = [1] * B if T == 1 else [(T + (T + 1) // 2) / 2] * B   # on average
    w = case["window"]
    seen = [min(n, w + T) if w >= 0 else n for n in lens]
    pairs = sum(r * max(0, (min(n, w) if w >= 0 else n) - (r - 1) / 2) for r, n in zip(rows, lens))
    return {"bytes": int(sum(seen) * Hkv * (2 * d + 0.125) + sum(rows) * H * (4 * d + 4)), "flops": int(4 * H * d * pairs)}


# ------------------------------------------------------------------- in 64 bits
def _e4m3(code):
    """fp64 values of E4M3 bytes, from their fields."""
    c = code.to(torch.int64)
    e, f = (c >> 3) & 15, (c & 7).to(torch.float64)
    mag = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2((e - 10).to(torch.float64)))
    mag = torch.where((c & 127) == 127, torch.full_like(mag, math.nan), mag)
    return torch.where(c >= 128, -mag, mag)


def _bytes_of(d, tok, dim):
    """Where the codes of a token's dims lie in a group: K's and V's."""
    k = ((((tok // 8) * (d // 64) + dim // 64) * 8 + tok % 8) * 4 + dim % 32 // 8) * 16 + dim % 64 // 32 * 8 + dim % 8
    v = ((((dim // 64) * 2 + tok // 8) * 8 + dim % 64 // 8) * 4 + tok % 8 // 2) * 16 + dim % 8 * 2 + tok % 2
    return k, 16 * d + v


def _exact_tokens(s, b, lo, hi):
    """fp64 keys and values [Hkv, hi - lo, d] of request b's tokens."""
    cache = s["cache"]
    page, d = 16 * cache.shape[2], (cache.shape[3] - 16) // 32
    pos = torch.arange(lo, hi, device=DEV)
    raw = cache[s["block_table"][b, pos // page].long(), :, pos % page // 16]  # [n,Hkv,32d+16]
    dim = torch.arange(d, device=DEV)[None]
    at = _bytes_of(d, (pos % 16)[:, None], dim)
    res = []
    for which in (0, 1):
        c = _e4m3(raw.gather(2, at[which][:, None].expand(-1, raw.shape[1], -1)))
        e = raw[..., 32 * d + which].to(torch.int64)
        res.append((c * torch.exp2(torch.where(e > 127, e - 256, e).to(torch.float64))[..., None]).transpose(0, 1))
    return res


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] in ("rope", "rope_bwd"):
        H, Hkv, d, rot = (case[x] for x in ("H", "Hkv", "d", "rot"))
        half = rot // 2
        # The rotation as complex factors on the rotated pairs, pair by pair.
        tab = s["rope"].to(f64)
        cols = []
        for i, axis in enumerate(_axis_of_pairs(case)):
            row = tab[s["positions"][axis].long()]
            cols.append(torch.complex(row[..., i], row[..., half + i]))
        turn = torch.stack(cols, -1).unsqueeze(2)
        first = torch.arange(half, device=DEV) * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)

        def rotate(y, factor):
            z = torch.complex(y[..., first], y[..., second]) * factor
            y = y.clone()
            y[..., first], y[..., second] = z.real, z.imag
            return y

        x = s["qkv"].to(f64)
        parts = {"q": (x[:, :, :H], s["q_weight"]), "k": (x[:, :, H:H + Hkv], s["k_weight"])}
        res, into = {}, []
        for name, (y, w) in parts.items():
            std = (y.pow(2).sum(-1, keepdim=True) / d + s["eps"]).sqrt()
            if case["op"] == "rope":
                z = y if w is None else y / std * w.to(f64)
                res[name] = rotate(z, turn).transpose(1, 2)
            else:
                dy = rotate(s["d" + name].to(f64).transpose(1, 2), turn.conj())
                if w is None:
                    res["d%sw" % name] = None
                    into.append(dy)
                else:
                    res["d%sw" % name] = torch.einsum("bnhd,bnhd->d", dy, y / std)
                    dyw = dy * w.to(f64)
                    # d(y/std): through the numerator, and through std.
                    into.append(dyw / std - y * (dyw * y).sum(-1, keepdim=True) / (d * std.pow(3)))
        if case["op"] == "rope":
            return {"q": res["q"], "k": res["k"], "v": x[:, :, H + Hkv:].transpose(1, 2)}
        return {"dqkv": torch.cat(into + [s["dv"].to(f64).transpose(1, 2)], 2), "dqw": res["dqw"], "dkw": res["dkw"]}
    if case["op"] == "append":
        res = {"cache": None}
        per, d = s["cache"].shape[2], case["d"]
        ok = s["slots"] >= 0
        slot = s["slots"].clamp(min=0).long()
        g = slot // 16
        head = s["cache"][g // per, :, g % per, 32 * d:32 * d + 2].to(torch.int64)  # [B,N,Hkv,2]
        head = torch.where(head > 127, head - 256, head)
        n = int(g.max()) + 1
        begun = torch.zeros(n, dtype=torch.bool, device=DEV)
        begun[g[ok & (slot % 16 == 0)]] = True
        for which, name in enumerate("kv"):
            x = s[name].to(f64).transpose(1, 2)             # [B,N,Hkv,d]
            top = x.abs().amax(-1)
            e = torch.ceil(torch.log2(top / 448)).clamp(-EXP, EXP)
            most = torch.full((n, x.shape[2]), float(-EXP), dtype=f64, device=DEV)
            most.index_reduce_(0, g[ok], e[ok], "amax")
            e = most[g]
            e = torch.where(begun[g][..., None], e, torch.maximum(e, head[..., which].to(f64)))
            unit = torch.exp2(e)[..., None]
            a = (x.abs() / unit).clamp(max=448.0)
            # E4M3 by its step: 3 bits below the leading one, 2^-9 at least.
            step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
            val = torch.round(a / step) * step * unit * torch.sign(x)
            res[name] = torch.where(ok[..., None, None], val, torch.zeros_like(val)).transpose(1, 2)
        return res
    if case["op"] == "read":
        res = {x: torch.zeros(s["k_out"].shape, dtype=f64, device=DEV) for x in "kv"}
        for b, (n, lo) in enumerate(zip(s["seq_lens"].tolist(), s["starts"].tolist())):
            hi = min(n, lo + case["N"])
            res["k"][b, :, :hi - lo], res["v"][b, :, :hi - lo] = _exact_tokens(s, b, lo, hi)
        return res
    B, T, H, Hkv, d, w = (case[x] for x in ("B", "T", "H", "Hkv", "d", "window"))
    o = torch.zeros((B, H, T, d), dtype=f64, device=DEV)
    lse = torch.zeros((B, H, T), dtype=f64, device=DEV)
    for b, L in enumerate(s["seq_lens"].tolist()):
        new = T if s["q_lens"] is None else int(s["q_lens"][b])
        lo = max(0, L - new - w) if w >= 0 else 0
        keys, vals = _exact_tokens(s, b, lo, L)
        i = torch.arange(L - new, L, device=DEV)[:, None]
        j = torch.arange(lo, L, device=DEV)
        hide = j > i
        if w >= 0:
            hide = hide | (j < i - w)
        for h in range(H):
            a = s["q"][b, h, :new].to(f64) @ keys[h // (H // Hkv)].T * s["scale"]
            a = a.masked_fill(hide, -math.inf)
            lse[b, h, :new] = torch.logsumexp(a, -1)
            # A row before the cache's first token sees nothing: zeros.
            p = torch.exp(a - torch.where(lse[b, h, :new] > -math.inf, lse[b, h, :new], 0.0)[:, None])
            o[b, h, :new] = p @ vals[h // (H // Hkv)]
    return {"o": o, "lse": lse}
