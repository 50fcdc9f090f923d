"""The serving and training operators around the attention kernels, as cases.

  rope, rope_bwd  norms of the query and key heads with the rotation of their
                  positions, from a projection's output to the attention's
                  layout, and the gradient of that
  plan            block tables and slot maps of a paged cache
  append          new keys and values into a cache held in 4 bits
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
        # One decode step of 32 requests: latency of a small call.
        {"name": "rope_decode_32x1", "op": "rope", "B": 32, "N": 1, "H": 32, "Hkv": 8, "d": 128, "rot": 128, "norm": True, "interleaved": False},
        # Training, the headline attention shape with grouped heads.
        {"name": "rope_train_4x4096", "op": "rope", "B": 4, "N": 4096, "H": 64, "Hkv": 8, "d": 128, "rot": 128, "norm": True, "interleaved": False},
        # Backward of a medium training step.
        {"name": "rope_bwd_4x1024", "op": "rope_bwd", "B": 4, "N": 1024, "H": 32, "Hkv": 32, "d": 128, "rot": 128, "norm": True, "interleaved": False},
        # Backward of long ragged rows, small heads, half of each head rotated.
        {"name": "rope_bwd_7x3001_d64", "op": "rope_bwd", "B": 7, "N": 3001, "H": 24, "Hkv": 8, "d": 64, "rot": 32, "norm": True, "interleaved": True},
        # One more token for each of 256 running requests, then taken back
        # (a rejected draft token).
        {"name": "plan_decode_256", "op": "plan", "R": 256, "T": 1, "page": 64, "len_min": 1, "len_max": 8192},
        # Prompts of up to 4096 tokens admitted together, then dropped.
        {"name": "plan_prompts_48x4096", "op": "plan", "R": 48, "T": 4096, "page": 16, "len_min": 0, "len_max": 0},
        # One new token for each of 128 requests.
        {"name": "append_decode_128", "op": "append", "B": 128, "N": 1, "Hkv": 8, "d": 128, "page": 64},
        # Prompts written to the cache.
        {"name": "append_prompt_8x4000", "op": "append", "B": 8, "N": 4000, "Hkv": 8, "d": 128, "page": 64},
        # One request with a short history: latency.
        {"name": "attn_one_1x900_d64", "op": "attn", "B": 1, "T": 1, "H": 16, "Hkv": 16, "d": 64, "page": 16, "len_min": 900, "len_max": 900, "window": -1},
        # A full decode batch with ragged histories.
        {"name": "attn_batch_64x8192", "op": "attn", "B": 64, "T": 1, "H": 64, "Hkv": 8, "d": 128, "page": 64, "len_min": 100, "len_max": 8192, "window": -1},
        # Few requests with long histories.
        {"name": "attn_long_3x131072", "op": "attn", "B": 3, "T": 1, "H": 32, "Hkv": 8, "d": 128, "page": 128, "len_min": 100000, "len_max": 131072, "window": -1},
        # Draft tokens checked together, one shared key/value head, a band.
        {"name": "attn_draft_16x5_mqa", "op": "attn", "B": 16, "T": 5, "H": 8, "Hkv": 1, "d": 128, "page": 32, "len_min": 3, "len_max": 30000, "window": 20000},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _heads(rng, most):
    Hkv = rng.choice([1, 2, 4, 8, 16])
    return min(most, Hkv * rng.choice([1, 2, 3, 4, 7, 8])) // Hkv * Hkv, Hkv


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "plan", "append", "attn", "attn"])
    d = rng.choice([64, 128, 128])
    if op in ("rope", "rope_bwd"):
        H, Hkv = _heads(rng, 64)
        tokens = _spread(rng, 1, 12288 if op == "rope" else 8192)
        B = _spread(rng, 1, min(64, tokens))
        return {"op": op, "B": B, "N": max(1, tokens // B), "H": H, "Hkv": Hkv, "d": d,
                "rot": rng.choice([d, d, d // 2]), "norm": rng.random() < 0.8, "interleaved": rng.random() < 0.4}
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        T = rng.choice([1, _spread(rng, 2, 4096)])
        R = _spread(rng, 1, 1024) if T == 1 else _spread(rng, 1, max(1, 196608 // T))
        hi = _spread(rng, 1, 16384)
        return {"op": op, "R": R, "T": T, "page": page, "len_min": min(hi, rng.choice([0, 1, 17])), "len_max": hi}
    if op == "append":
        tokens = _spread(rng, 1, 32000)
        B = _spread(rng, 1, min(256, tokens))
        return {"op": op, "B": B, "N": max(1, tokens // B), "Hkv": rng.choice([1, 2, 4, 8]), "d": d, "page": page}
    H, Hkv = _heads(rng, 64)
    T = rng.choice([1, 1, 1, rng.randint(2, 9)])
    budget = 3 * 100000 * 8 // Hkv
    hi = _spread(rng, 1, min(131072, budget))
    B = _spread(rng, 1, max(1, min(128, budget // hi)))
    return {"op": op, "B": B, "T": T, "H": H, "Hkv": Hkv, "d": d, "page": page, "len_min": max(0, hi // rng.choice([1, 2, 50])),
            "len_max": hi, "window": rng.choice([-1, -1, -1, hi // 3])}


def _lengths(n, lo, hi):
    """n whole numbers from hi down to lo, evenly spread."""
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


# ----------------------------------------------------- the 4-bit format, plain
# 16 tokens of one key/value head are one group of 18 d bytes:
#   K codes [16][d/2]          two dims a byte, the even one low
#   K scales [16][d/16]        E4M3
#   V codes [2][8][4][2][d/16] (token/8, dims in eighths, token%8/2, token%2)
#   V scales [2][d/16][4][2]   (token/8, block of 16 dims, token%8/2, token%2)
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _codes(x, g):
    """E2M1 codes [..., d] and E4M3 scale bytes [..., d/16] of fp32 x."""
    b = x.unflatten(-1, (-1, 16))
    s = (b.abs().amax(-1) / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = s.float().unsqueeze(-1) * g
    y = torch.where(f > 0, b / f, torch.zeros_like(b))
    a = y.abs()
    # Ties go to the even code.
    c = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
         + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte())
    c = c + 8 * (torch.signbit(y)).byte()
    return c.flatten(-2), s.view(torch.uint8)


def _values(codes, scales, g, table):
    """fp32 values of codes [..., d] and scale bytes [..., d/16]."""
    v = table[codes.int()].unflatten(-1, (-1, 16))
    return (v * (scales.contiguous().view(torch.float8_e4m3fn).float() * g).unsqueeze(-1)).flatten(-2)


def _pairs(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _unpairs(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _groups(k, v, gk, gv):
    """Group bytes [..., 18 d] of fp32 keys and values [..., 16, d]."""
    d = k.shape[-1]
    lead = k.shape[:-2]
    kc, ks = _codes(k, gk)
    vc, vs = _codes(v, gv)
    vc = _pairs(vc).reshape(*lead, 2, 4, 2, 8, d // 16)
    vs = vs.reshape(*lead, 2, 4, 2, d // 16)
    n = len(lead)
    vc = vc.permute(*range(n), n, n + 3, n + 1, n + 2, n + 4)
    vs = vs.permute(*range(n), n, n + 3, n + 1, n + 2)
    return torch.cat([_pairs(kc).flatten(-2), ks.flatten(-2), vc.flatten(n), vs.flatten(n)], -1)


def _ungroup(grp, gk, gv, table):
    """fp32 keys and values [..., 16, d] of group bytes [..., 18 d]."""
    d = grp.shape[-1] // 18
    lead = grp.shape[:-1]
    n = len(lead)
    kc = grp[..., :8 * d].reshape(*lead, 16, d // 2)
    ks = grp[..., 8 * d:9 * d].reshape(*lead, 16, d // 16)
    vc = grp[..., 9 * d:17 * d].reshape(*lead, 2, 8, 4, 2, d // 16)
    vs = grp[..., 17 * d:].reshape(*lead, 2, d // 16, 4, 2)
    vc = vc.permute(*range(n), n, n + 2, n + 3, n + 1, n + 4).reshape(*lead, 16, d // 2)
    vs = vs.permute(*range(n), n, n + 2, n + 3, n + 1).reshape(*lead, 16, d // 16)
    return _values(_unpairs(kc), ks, gk, table), _values(_unpairs(vc), vs, gv, table)


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))

    def normal(*shape, dtype=torch.bfloat16, mult=1.0):
        return (torch.randn(shape, generator=gen, device=DEV) * mult).to(dtype)

    def shuffled(n):
        return torch.randperm(n, generator=gen, device=DEV).to(torch.int32)

    s = {"op": case["op"], "e2m1": torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float32, device=DEV)}
    if case["op"] in ("rope", "rope_bwd"):
        B, N, H, Hkv, d, rot = (case[x] for x in ("B", "N", "H", "Hkv", "d", "rot"))
        s.update(H=H, Hkv=Hkv, eps=1e-6, interleaved=case["interleaved"])
        s["qkv"] = normal(B, N, H + 2 * Hkv, d)
        # A table of cosines and sines for as far as the model reaches.
        P = 32768
        freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
        ang = torch.arange(P, dtype=torch.float64, device=DEV)[:, None] * freq
        s["rope"] = torch.cat([ang.cos(), ang.sin()], -1).float()
        start = torch.randint(0, P - N + 1, (B, 1), generator=gen, device=DEV)
        s["positions"] = (start + torch.arange(N, device=DEV)).to(torch.int32)
        s["q_weight"] = 1 + normal(d, dtype=torch.float32, mult=0.1) if case["norm"] else None
        s["k_weight"] = 1 + normal(d, dtype=torch.float32, mult=0.1) if case["norm"] else None
        if case["op"] == "rope_bwd":
            s["dq"], s["dk"], s["dv"] = normal(B, H, N, d), normal(B, Hkv, N, d), normal(B, Hkv, N, d)
    elif case["op"] == "plan":
        R, T, page = case["R"], case["T"], case["page"]
        lens = _lengths(R, case["len_min"], case["len_max"])
        new = _lengths(R, (T + 1) // 2, T)
        blocks = -(-(case["len_max"] + T) // page)
        used = sum(-(-n // page) for n in lens)
        pages = used + sum(-(-(n + m) // page) for n, m in zip(lens, new)) + 8
        at = shuffled(R).long()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)[at]
        s["new"] = torch.tensor(new, dtype=torch.int32, device=DEV)[at.flip(0)]
        s["back"] = -s["new"]
        ids = shuffled(pages)
        have = (s["lens"] + page - 1) // page
        i = torch.arange(blocks, device=DEV)[None]
        off = (have.cumsum(0) - have)[:, None]
        s["block_table"] = torch.where(i < have[:, None], ids[(off + i).clamp(max=pages - 1)], -1).to(torch.int32)
        s["free_list"] = torch.cat([ids[used:], torch.full((used,), -1, dtype=torch.int32, device=DEV)])
        s["free_count"] = torch.tensor([pages - used], dtype=torch.int32, device=DEV)
        s.update(page=page, T=T)
    elif case["op"] == "append":
        B, N, Hkv, d, page = (case[x] for x in ("B", "N", "Hkv", "d", "page"))
        s["k"], s["v"] = normal(B, Hkv, N, d, mult=1.5), normal(B, Hkv, N, d, mult=0.7)
        per = -(-N // page) + 1
        ids = shuffled(B * per + 3)
        new = torch.tensor(_lengths(B, (N + 1) // 2, N), dtype=torch.int32, device=DEV)[shuffled(B).long()]
        start = torch.randint(0, page, (B, 1), generator=gen, device=DEV)
        t = torch.arange(N, device=DEV)[None]
        pos = start + t
        slot = ids[torch.arange(B, device=DEV)[:, None] * per + pos // page] * page + pos % page
        s["slots"] = torch.where(t < new[:, None], slot, -1).to(torch.int32)
        s["cache"] = torch.zeros((B * per + 3, Hkv, page // 16, 18 * d), dtype=torch.uint8, device=DEV)
        s["k_out"], s["v_out"] = torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
        s.update(k_scale=1.0, v_scale=0.5)
    else:
        B, T, H, Hkv, d, page = (case[x] for x in ("B", "T", "H", "Hkv", "d", "page"))
        lens = _lengths(B, case["len_min"], case["len_max"])
        at = shuffled(B).long()
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)[at]
        s["q_lens"] = None if T == 1 else torch.tensor(_lengths(B, (T + 1) // 2, T), dtype=torch.int32, device=DEV)[at.flip(0)]
        blocks = -(-case["len_max"] // page)
        have = (s["seq_lens"] + page - 1) // page
        pages = sum(-(-n // page) for n in lens) + 5
        ids = shuffled(pages)
        i = torch.arange(max(1, blocks), device=DEV)[None]
        off = (have.cumsum(0) - have)[:, None]
        s["block_table"] = torch.where(i < have[:, None], ids[(off + i).clamp(max=pages - 1)], -1).to(torch.int32)
        s.update(k_scale=1.0, v_scale=0.5)
        s["cache"] = _groups(normal(pages, Hkv, page // 16, 16, d, dtype=torch.float32, mult=1.5),
                             normal(pages, Hkv, page // 16, 16, d, dtype=torch.float32, mult=0.7), 1.0, 0.5)
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
        q, k, v = fa.fa_qk_norm_rope(s["qkv"], s["H"], s["Hkv"], s["rope"], s["positions"], s["q_weight"], s["k_weight"],
                                     eps=s["eps"], interleaved=s["interleaved"])
        return {"q": q, "k": k, "v": v}
    if s["op"] == "rope_bwd":
        dqkv, dqw, dkw = fa.fa_qk_norm_rope_bwd(s["qkv"], s["H"], s["Hkv"], s["rope"], s["dq"], s["dk"], s["dv"], s["positions"],
                                                s["q_weight"], s["k_weight"], eps=s["eps"], interleaved=s["interleaved"])
        return {"dqkv": dqkv, "dqw": dqw, "dkw": dkw}
    if s["op"] == "plan":
        state = (s["lens"], s["block_table"], s["free_list"], s["free_count"])
        slots, positions, granted = fa.fa_cache4_plan(s["new"], *state, s["page"], s["T"])
        fa.fa_cache4_plan(s["back"], *state, s["page"], s["T"])
        return {"slots": slots, "positions": positions, "granted": granted, "lens": s["lens"], "table": s["block_table"],
                "free": s["free_list"], "count": s["free_count"]}
    if s["op"] == "append":
        fa.fa_cache4_append(s["k"], s["v"], s["cache"], s["slots"], s["k_scale"], s["v_scale"], k_out=s["k_out"], v_out=s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"], "cache": s["cache"]}
    o, lse = fa.fa_cache4_attn(s["q"], s["cache"], s["block_table"], s["seq_lens"], s["scale"], q_lens=s["q_lens"],
                               window=s["window"], k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"], lse=s["lse"])
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


def _plain_rope(s):
    H, Hkv = s["H"], s["Hkv"]
    x = s["qkv"].float()
    t = s["rope"][s["positions"].long()]
    c, n = t.chunk(2, -1)
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
    c, n = s["rope"][s["positions"].long()].chunk(2, -1)

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


def _plain_plan(s, new):
    """One call: requests that shrink give their pages back, the others take
    theirs in order.  Returns slots, positions and the tokens granted."""
    lens, table, page, T = s["lens"], s["block_table"], s["page"], s["T"]
    R, M = table.shape
    P = s["free_list"].numel()
    dev = lens.device
    have = (lens + page - 1) // page
    after = torch.where(new < 0, (lens + new).clamp(min=0), lens)
    keep = (after + page - 1) // page
    back = have - keep
    i = torch.arange(M, device=dev)[None]
    # The last request's last page is pushed first.
    behind = (back.flip(0).cumsum(0).flip(0) - back)[:, None]
    at = s["free_count"] + behind + (have[:, None] - 1 - i)
    given = (i >= keep[:, None]) & (i < have[:, None])
    stack = torch.cat([s["free_list"], s["free_list"].new_zeros(1)])
    stack = stack.scatter(0, torch.where(given, at, P).long().flatten(), table.flatten())[:P]
    count = s["free_count"] + back.sum()
    total = after.long() + new.clamp(min=0)
    fits = (new > 0) & (new <= T) & (total <= M * page)
    need = torch.where(fits, (total + page - 1) // page - keep, 0)
    upto = need.cumsum(0)
    granted = torch.where(fits & ((need == 0) | (upto <= count)), new, 0)
    need = torch.where(granted > 0, need, 0)
    j = i - keep[:, None]
    taken = (j >= 0) & (j < need[:, None])
    src = (count - 1 - (upto - need)[:, None] - j).clamp(0, P - 1)
    table.copy_(torch.where(taken, stack[src.long()], table))
    s["free_list"].copy_(stack)
    s["free_count"].copy_(count - need.sum())
    lens.copy_((after + granted).to(torch.int32))
    t = torch.arange(T, device=dev)[None]
    ok = t < granted[:, None]
    pos = (after[:, None] + t).clamp(max=M * page - 1)
    slot = table.gather(1, (pos // page).long()) * page + pos % page
    return torch.where(ok, slot, -1).to(torch.int32), torch.where(ok, pos, 0).to(torch.int32), granted.to(torch.int32)


def _plain_append(s):
    cache, slots = s["cache"], s["slots"]
    pages, Hkv, per, d = cache.shape[0], cache.shape[1], cache.shape[2], cache.shape[3] // 18
    page = 16 * per
    k, v = s["k"].float().transpose(1, 2), s["v"].float().transpose(1, 2)  # [B,N,Hkv,d]
    kc, ks = _codes(k, s["k_scale"])
    vc, vs = _codes(v, s["v_scale"])
    ok = slots >= 0
    used = ok[:, None, :, None]
    s["k_out"].copy_(torch.where(used, _values(kc, ks, s["k_scale"], s["e2m1"]).to(torch.bfloat16).transpose(1, 2), s["k_out"]))
    s["v_out"].copy_(torch.where(used, _values(vc, vs, s["v_scale"], s["e2m1"]).to(torch.bfloat16).transpose(1, 2), s["v_out"]))
    at = slots[ok].long()
    grp = cache.view(pages, Hkv, per, 18 * d)
    p, r = at // page, at % page
    u, t = r // 16, r % 16
    h = torch.arange(Hkv, device=at.device)
    base = ((p[:, None] * Hkv + h) * per + u[:, None]) * (18 * d)  # [n,Hkv]
    flat = grp.view(-1)

    def put(where, what):
        flat[(base[..., None] + where[:, None]).flatten()] = what[ok].flatten()

    b = torch.arange(d // 2, device=at.device)
    q = torch.arange(d // 16, device=at.device)
    put(t[:, None] * (d // 2) + b, _pairs(kc))
    put(8 * d + t[:, None] * (d // 16) + q, ks)
    e, f, half = t % 8 // 2, t % 2, t // 8
    v_at = ((half[:, None] * 8 + b // (d // 16)) * 4 + e[:, None]) * 2 + f[:, None]
    put(9 * d + v_at * (d // 16) + b % (d // 16), _pairs(vc))
    put(17 * d + ((half[:, None] * (d // 16) + q) * 4 + e[:, None]) * 2 + f[:, None], vs)
    return {"k": s["k_out"], "v": s["v_out"], "cache": cache}


def _plain_attn(s):
    q, cache, table = s["q"], s["cache"], s["block_table"]
    B, H, T, d = q.shape
    Hkv, page = cache.shape[1], 16 * cache.shape[2]
    grp = cache[table.clamp(min=0).long()].transpose(1, 2)  # [B,Hkv,M,page/16,18d]
    k, v = _ungroup(grp, s["k_scale"], s["v_scale"], s["e2m1"])
    k, v = k.flatten(2, 4), v.flatten(2, 4)                 # [B,Hkv,L,d]
    L = k.shape[2]
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
    if state["op"] == "rope":
        return _plain_rope(state)
    if state["op"] == "rope_bwd":
        return _plain_rope_bwd(state)
    if state["op"] == "plan":
        slots, positions, granted = _plain_plan(state, state["new"])
        _plain_plan(state, state["back"])
        return {"slots": slots, "positions": positions, "granted": granted, "lens": state["lens"], "table": state["block_table"],
                "free": state["free_list"], "count": state["free_count"]}
    return _plain_append(state) if state["op"] == "append" else _plain_attn(state)


# ------------------------------------------------------------------ what it costs
def work(case):
    op = case["op"]
    if op in ("rope", "rope_bwd"):
        rows, H, Hkv, d = case["B"] * case["N"], case["H"], case["Hkv"], case["d"]
        all_ = rows * (H + 2 * Hkv) * d
        side = rows * 4 + min(rows, 32768) * case["rot"] * 4
        if op == "rope":
            return {"bytes": 4 * all_ + side, "flops": 8 * rows * (H + Hkv) * d}
        x = 2 * rows * (H + Hkv) * d if case["norm"] else 0
        return {"bytes": 4 * all_ + x + side, "flops": 16 * rows * (H + Hkv) * d}
    if op == "plan":
        # Both calls: lengths and counts, the pages that change hands, and
        # the slots and positions of the new tokens.
        R, T, page = case["R"], case["T"], case["page"]
        lens, new = _lengths(R, case["len_min"], case["len_max"]), _lengths(R, (T + 1) // 2, T)
        moved = sum(new) // page + (R if new[0] % page else 0)
        return {"bytes": 2 * (R * 16 + moved * 8 + R * T * 8), "flops": 0}
    if op == "append":
        rows = sum(_lengths(case["B"], (case["N"] + 1) // 2, case["N"])) * case["Hkv"]
        d = case["d"]
        return {"bytes": rows * (4 * d + 4 * d + 18 * d // 16) + case["B"] * case["N"] * 4, "flops": 8 * rows * d}
    B, T, H, Hkv, d = (case[x] for x in ("B", "T", "H", "Hkv", "d"))
    seen = [min(n, case["window"] + T) if case["window"] >= 0 else n for n in _lengths(B, case["len_min"], case["len_max"])]
    rows = B * T if T == 1 else sum(_lengths(B, (T + 1) // 2, T))
    return {"bytes": sum(seen) * Hkv * 18 * d // 16 + rows * H * (4 * d + 4), "flops": 4 * sum(seen) * H * d * rows / B}


# ------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "plan":
        return None  # whole numbers only
    if case["op"] in ("rope", "rope_bwd"):
        B, N, H, Hkv, d, rot = (case[x] for x in ("B", "N", "H", "Hkv", "d", "rot"))
        half = rot // 2
        # The rotation as complex factors on the rotated pairs.
        tab = s["rope"].to(f64)[s["positions"].long()]
        turn = torch.complex(tab[..., :half], tab[..., half:]).unsqueeze(2)
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
        for name, g in (("k", s["k_scale"]), ("v", s["v_scale"])):
            x = s[name].to(f64).unflatten(-1, (-1, 16))
            sc = (x.abs().amax(-1, keepdim=True) / 6 / g).clamp(max=448.0)
            # E4M3 by its step: 3 bits below the leading one, 2^-9 at least.
            step = torch.exp2(torch.floor(torch.log2(sc.clamp(min=2.0 ** -6))) - 3)
            sc = torch.round(sc / step) * step * g
            a = torch.where(sc > 0, x.abs() / sc, torch.zeros_like(x)).clamp(max=6.0)
            st = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
            val = torch.round(a / st) * st * sc * torch.sign(x)
            ok = (s["slots"] >= 0)[:, None, :, None]
            res[name] = torch.where(ok, val.flatten(-2), torch.zeros_like(s[name], dtype=f64))
        return res
    B, T, H, Hkv, d, page = (case[x] for x in ("B", "T", "H", "Hkv", "d", "page"))
    o = torch.zeros((B, H, T, d), dtype=f64, device=DEV)
    lse = torch.zeros((B, H, T), dtype=f64, device=DEV)
    mag = torch.tensor(E2M1 + [-x for x in E2M1], dtype=f64, device=DEV)
    n = torch.arange(16, device=DEV)
    half, e, f = n // 8, n % 8 // 2, n % 2
    dim = torch.arange(d, device=DEV)
    k_at = n[:, None] * (d // 2) + dim // 2
    ks_at = 8 * d + n[:, None] * (d // 16) + dim // 16
    oct_, byte = dim // (d // 8), dim % (d // 8) // 2
    v_at = 9 * d + ((((half[:, None] * 8 + oct_) * 4 + e[:, None]) * 2) + f[:, None]) * (d // 16) + byte
    vs_at = 17 * d + ((half[:, None] * (d // 16) + dim // 16) * 4 + e[:, None]) * 2 + f[:, None]
    odd = dim % 2 * 4
    lens = s["seq_lens"].tolist()
    for b in range(B):
        L = lens[b]
        new = T if s["q_lens"] is None else int(s["q_lens"][b])
        pg = s["block_table"][b, :-(-L // page)].long()
        raw = s["cache"][pg]                                # [M,Hkv,page/16,18d]
        for hk in range(Hkv):
            u = raw[:, hk].reshape(-1, 18 * d)
            nib = lambda at: mag[((u[:, at].int() >> odd) & 15)]  # noqa: E731
            sc = lambda at: u[:, at].contiguous().view(torch.float8_e4m3fn).to(f64)  # noqa: E731
            kk = (nib(k_at) * sc(ks_at)).reshape(-1, d)[:L] * s["k_scale"]
            vv = (nib(v_at) * sc(vs_at)).reshape(-1, d)[:L] * s["v_scale"]
            for t in range(new):
                i = L - new + t
                lo = max(0, i - s["window"]) if s["window"] >= 0 else 0
                hq = slice(hk * (H // Hkv), (hk + 1) * (H // Hkv))
                if i < 0:
                    lse[b, hq, t] = -math.inf
                    continue
                a = s["q"][b, hq, t].to(f64) @ kk[lo:i + 1].T * s["scale"]
                lse[b, hq, t] = torch.logsumexp(a, -1)
                o[b, hq, t] = torch.softmax(a, -1) @ vv[lo:i + 1]
    return {"o": o, "lse": lse}
