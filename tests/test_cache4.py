"""The paged 4-bit cache: format, bookkeeping and refusals on the CPU; plan,
append and attention on the GPU against the float64 oracle.

Codes, scales, slots, tables and counts have to be equal.  The attention's
tolerances: K, V and Q enter the products exactly.  A score is a sum of d
products in fp32, within es = (d + 8) 2^-24 scale sum |q||k| of its value, so
a weight is within 2 es + 2^-20 (exponential, sums) of its own; P is rounded
to f16 (half a step: 2^-11 of the weight, or less than 2^-32 of the row's
largest where it vanishes); O is rounded to bf16 (2^-8).  The LSE is within
es + 2^-20 (1 + |lse|).
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import serve
from tiled_attention_bwd_gb300 import build as fa_build
from tiled_attention_bwd_gb300 import fa

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5


def f64(t):
    return t.detach().to("cpu").double().numpy()


# ------------------------------------------------------------------- on CPU
def test_format_rounds_to_nearest_even():
    g = serve.E2M1
    x = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 9.0, 0.2, 0.26])
    want = np.array([0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 6.0, 0.0, 0.5])
    assert np.array_equal(g[serve.nearest_code(x, g)], want)
    assert serve.E4M3[126] == 448 and serve.E4M3[1] == 2.0 ** -9
    assert serve.nearest_code(1000.0, serve.E4M3) == 126


def test_every_value_is_a_bf16_and_an_f16():
    v = np.outer(serve.E2M1, serve.E4M3).ravel().astype(np.float32)
    t = torch.from_numpy(v)
    assert torch.equal(t.bfloat16().float(), t)
    assert torch.equal(t.half().float(), t)


def test_quantisation_error_is_at_most_a_sixth_of_the_largest():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((50, 64))
    c, s = serve.quantise(x, 1.0)
    y = serve.dequantise(c, s, 1.0)
    amax = np.abs(x).reshape(50, 4, 16).max(-1).repeat(16, -1).reshape(50, 64)
    # Half the widest step (1 of 6) of a scale off by 2^-4 at most.
    assert (np.abs(x - y) <= amax / 6 * (1 + 2.0 ** -4) + 1e-12).all()


@pytest.mark.parametrize("d", [64, 128])
def test_layout_places_every_byte_once(d):
    seen = np.zeros(18 * d, int)
    for tok in range(16):
        for at in serve._places(d, tok):
            seen[at] += 1
    assert (seen == 1).all()


def test_plan_oracle_takes_back_what_it_grants():
    rng = np.random.default_rng(1)
    R, M, page, P = 7, 6, 16, 30
    lens, table, free = [0] * R, [[-1] * M for _ in range(R)], list(range(P))
    for _ in range(20):
        new = [int(x) for x in rng.integers(0, 40, R)]
        before = (list(lens), list(free))
        _, _, granted = serve.plan(new, lens, table, free, page, 40)
        serve.plan([-g for g in granted], lens, table, free, page, 40)
        assert (lens, free) == before
        serve.plan([int(x) for x in rng.integers(-30, 30, R)], lens, table,
                   free, page, 40)
        held = [table[r][i] for r in range(R) for i in range(-(-lens[r] // page))]
        assert sorted(held + free) == list(range(P))


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fa.load_library()


def p(x):
    return ctypes.c_void_p(x) if x else None


def _plan(lib, new=256, lens=512, table=768, free=1024, count=1280, slots=1536,
          pos=1792, granted=2048, R=1, M=1, P=1, page=16, T=1):
    return lib.fa_cache4_plan(p(new), p(lens), p(table), p(free), p(count),
                              p(slots), p(pos), p(granted), R, M, P, page, T,
                              None)


@pytest.mark.parametrize("want,bad", [
    (INVALID, dict(R=-1)), (INVALID, dict(T=-1)), (INVALID, dict(M=-1)),
    (INVALID, dict(page=0)), (UNSUPPORTED, dict(page=8)),
    (UNSUPPORTED, dict(page=48)), (UNSUPPORTED, dict(page=512)),
    (UNSUPPORTED, dict(P=1 << 28)), (UNSUPPORTED, dict(M=1 << 28)),
    (UNSUPPORTED, dict(R=1 << 20, T=1 << 12)),
    (UNSUPPORTED, dict(R=1 << 20, M=1 << 12)), (INVALID, dict(new=0)),
    (INVALID, dict(lens=0)), (INVALID, dict(table=0)), (INVALID, dict(free=0)),
    (INVALID, dict(count=0)), (INVALID, dict(slots=0)),
    (INVALID, dict(pos=0)), (INVALID, dict(granted=0)),
    (INVALID, dict(lens=514)), (INVALID, dict(slots=1537)),
    (INVALID, dict(granted=256)), (INVALID, dict(slots=1792)),
    (INVALID, dict(new=508, R=2)), (INVALID, dict(T=65)),
])
def test_plan_refusals(lib, want, bad):
    assert _plan(lib, **bad) == want


def _append(lib, k=16, v=16, cache=16, slots=16, gk=1.0, gv=1.0, ko=0, vo=0,
            B=1, Hkv=1, N=1, d=128, pages=1, page=16):
    return lib.fa_cache4_append(p(k), p(v), p(cache), p(slots), gk, gv, p(ko),
                                p(vo), B, Hkv, N, d, pages, page, None)


@pytest.mark.parametrize("want,bad", [
    (UNSUPPORTED, dict(d=96)), (INVALID, dict(d=-64)),
    (UNSUPPORTED, dict(page=24)), (INVALID, dict(pages=-1)),
    (UNSUPPORTED, dict(pages=1 << 28)), (INVALID, dict(gk=3.0)),
    (INVALID, dict(gk=0.0)), (INVALID, dict(gv=-1.0)),
    (INVALID, dict(gv=float("inf"))), (INVALID, dict(gk=float("nan"))),
    (INVALID, dict(gk=2.0 ** 61)), (INVALID, dict(gv=2.0 ** -61)),
    (INVALID, dict(ko=16)), (INVALID, dict(vo=16)), (INVALID, dict(k=0)),
    (INVALID, dict(v=8)), (INVALID, dict(cache=0)), (INVALID, dict(slots=2)),
    (INVALID, dict(ko=1032, vo=2048)), (INVALID, dict(B=-1)),
    (INVALID, dict(k=256, v=512, ko=512, vo=1024)),
    (INVALID, dict(k=256, v=512, ko=1024, vo=1264)),
    (INVALID, dict(k=256, v=512, ko=256, vo=528)),
    (UNSUPPORTED, dict(B=1 << 20, N=1 << 12)),
])
def test_append_refusals(lib, want, bad):
    assert _append(lib, **bad) == want


def _attn(lib, q=16, cache=16, table=16, lens=16, ql=16, o=16, lse=16, ws=256,
          wsb=1 << 40, B=1, H=2, Hkv=1, T=1, d=128, M=1, pages=1, page=16,
          window=-1, scale=0.1, gk=1.0, gv=1.0):
    return lib.fa_cache4_attn(p(q), p(cache), p(table), p(lens), p(ql), p(o),
                              p(lse), p(ws), wsb, B, H, Hkv, T, d, M, pages,
                              page, window, scale, gk, gv, None)


@pytest.mark.parametrize("want,bad", [
    (UNSUPPORTED, dict(d=80)), (UNSUPPORTED, dict(page=1)),
    (INVALID, dict(Hkv=0)), (INVALID, dict(H=3, Hkv=2)),
    (INVALID, dict(H=1, Hkv=2)), (INVALID, dict(T=-1)),
    (INVALID, dict(scale=0.0)), (INVALID, dict(scale=float("nan"))),
    (INVALID, dict(gk=1.5)), (INVALID, dict(gv=0.3)), (INVALID, dict(q=0)),
    (INVALID, dict(scale=1e30, gk=2.0 ** 60)),
    (INVALID, dict(q=8)), (INVALID, dict(cache=0)), (INVALID, dict(table=0)),
    (INVALID, dict(lens=0)), (INVALID, dict(ql=2)), (INVALID, dict(o=0)),
    (INVALID, dict(o=8)), (INVALID, dict(lse=0)), (INVALID, dict(lse=2)),
    (WORKSPACE, dict(ws=0)), (WORKSPACE, dict(ws=16)),
    (WORKSPACE, dict(wsb=100)), (UNSUPPORTED, dict(M=1 << 28)),
    (UNSUPPORTED, dict(pages=1 << 28)),
    (UNSUPPORTED, dict(B=1 << 20, H=1 << 12)),
    (UNSUPPORTED, dict(B=1 << 15, T=1 << 16)),
    (UNSUPPORTED, dict(B=1 << 20, M=1 << 10, page=256)),
    (UNSUPPORTED, dict(T=1 << 30, H=1, M=1 << 23, page=256)),
    (UNSUPPORTED, dict(B=1 << 10, T=1 << 18, M=1 << 20, page=256)),
])
def test_attention_refusals(lib, want, bad):
    assert _attn(lib, **bad) == want


def test_empty_calls_and_sizes(lib):
    assert _plan(lib, R=0, new=0, lens=0) == OK
    assert _append(lib, N=0, k=0, v=0) == OK
    assert _append(lib, pages=0, cache=0) == OK
    assert _attn(lib, B=0, q=0) == OK
    assert _attn(lib, T=0, q=0, ws=0) == OK
    assert lib.fa_cache4_page_bytes(8, 64, 128) == 8 * 64 * 144
    assert lib.fa_cache4_page_bytes(2, 16, 64) == 2 * 16 * 72
    assert lib.fa_cache4_page_bytes(2, 24, 64) == 0
    assert lib.fa_cache4_page_bytes(0, 16, 64) == 0
    assert lib.fa_cache4_attn_workspace_size(1, 4, 3, 1, 128) == 0


def test_binding_refusals():
    z = torch.zeros
    with pytest.raises(ValueError):        # not on a GPU
        fa.fa_cache4_append(z(1), z(1), z((1, 1, 1, 18 * 64), dtype=torch.uint8), z(1))
    with pytest.raises(ValueError):
        fa.fa_cache4_plan(z(1, dtype=torch.int32), z(1), z(1), z(1), z(1), 16, 1)


# ------------------------------------------------------------ plan on the GPU
def i32(x, dev="cuda:0"):
    return torch.tensor(x, dtype=torch.int32, device=dev)


@pytest.mark.gpu
@pytest.mark.parametrize("R,M,page,P,T,seed", [
    (1, 1, 16, 1, 1, 0), (5, 4, 16, 12, 1, 1), (33, 9, 32, 200, 70, 2),
    (256, 6, 64, 700, 1, 3), (1500, 3, 16, 2100, 2, 4), (40, 33, 128, 900, 1000, 5),
    (2500, 2, 256, 2600, 300, 6),
])
def test_plan_matches_oracle(R, M, page, P, T, seed):
    rng = np.random.default_rng(seed)
    lens, table = [0] * R, [[-1] * M for _ in range(R)]
    free = [int(x) for x in rng.permutation(P)]
    g_lens, g_table = i32(lens), i32(table)
    g_free, g_count = i32(free), i32([P])
    for step in range(12):
        new = rng.integers(-T, T + 1, R)
        new[rng.random(R) < 0.2] = 0
        if step % 4 == 3:                  # the end of some, too much for some
            new[rng.random(R) < 0.5] = -2 ** 31
            new[rng.random(R) < 0.1] = T + 1
            new[rng.random(R) < 0.1] = 2 ** 31 - 1
        new = [int(x) for x in new]
        want = serve.plan(new, lens, table, free, page, T)
        got = fa.fa_cache4_plan(i32(new), g_lens, g_table, g_free, g_count, page, T)
        for w, g in zip(want, got):
            assert torch.equal(i32(w), g), step
        assert g_lens.tolist() == lens
        assert g_table.tolist() == table
        assert g_count.item() == len(free)
        assert g_free[:len(free)].tolist() == free


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 40, 2 ** 28, 2 ** 31 - 1])
@pytest.mark.parametrize("T", [3, 9])
def test_plan_gives_no_slots_on_pages_outside_the_cache(bad, T):
    """A bad id in the table (request 0) and in the stack (request 1)."""
    page, n = 16, T - 1
    table, lens = i32([[bad, -1], [3, -1]]), i32([10, 14])
    free, count = i32([7, bad] + [0] * 38), i32([2])
    slots, pos, granted = fa.fa_cache4_plan(i32([n, n]), lens, table, free,
                                            count, page, T)
    assert granted.tolist() == [n, n] and lens.tolist() == [10 + n, 14 + n]
    ids = [[bad, bad if n > 6 else -1], [3, 7 if n > 6 else bad if n > 2 else -1]]
    assert table.tolist() == ids
    for r, at in ((0, 10), (1, 14)):
        for t in range(T):
            p = at + t
            held = ids[r][p // page]
            ok = t < n and 0 <= held < 40
            assert slots[r, t].item() == (held * page + p % page if ok else -1)
            assert pos[r, t].item() == (p if t < n else 0)


@pytest.mark.gpu
def test_plan_brings_values_into_range():
    """Lengths, counts and page ids that no call writes are clamped."""
    lens, table = i32([-7, 1 << 30, 5]), i32([[0, 1], [9, -4], [2, 3]])
    free, count = i32([4, 5, 6]), i32([100])
    slots, pos, granted = fa.fa_cache4_plan(i32([1, -2 ** 31, 20]), lens, table,
                                            free, count, 16, 20)
    torch.cuda.synchronize()
    assert lens.tolist() == [1, 0, 25]
    assert granted.tolist() == [1, 0, 20]
    assert 0 <= count.item() <= 3


# ---------------------------------------------------------- append on the GPU
def special_rows(n, d, seed):
    """Rows that meet the format's corners."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, d), generator=g) * torch.exp2(
        torch.randint(-14, 12, (n, d // 16), generator=g).float()).repeat_interleave(16, 1)
    # Exact ties between codes: a largest value of 6 s and multiples of s / 4.
    tie = torch.randint(-24, 25, (n, d), generator=g) / 4.0
    tie[:, ::16] = 6.0
    tie *= torch.randint(8, 16, (n, 1), generator=g) / 8.0
    x = torch.where(torch.arange(n)[:, None] % 3 == 1, tie, x)
    x[0] = 0.0
    if n > 4:
        x[1, 3] = float("inf")
        x[1, 20] = -float("inf")
        x[2, 5] = float("nan")
        x[3] = -0.0
        x[4] = torch.randn(d, generator=g) * 1e-30
        x[4, 17] = 3e38
    return x.bfloat16()


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hkv,N,d,page,gk,gv", [
    (1, 1, 1, 128, 16, 1.0, 1.0), (2, 3, 1, 64, 32, 1.0, 0.5),
    (3, 2, 37, 128, 64, 2.0 ** -8, 4.0), (1, 4, 130, 64, 256, 1.0, 2.0 ** 20),
    (5, 1, 20, 64, 16, 2.0 ** -60, 2.0 ** 60),
])
def test_append_matches_oracle(B, Hkv, N, d, page, gk, gv):
    dev = torch.device("cuda:0")
    pages = B * N // page + B + 3
    rng = np.random.default_rng(N)
    slots = rng.permutation(pages * page)[:B * N].reshape(B, N).astype(np.int32)
    slots[rng.random((B, N)) < 0.15] = -1
    if N > 5:
        slots[0, 1] = pages * page         # behind the cache: skipped
        slots[0, 2] = 2 ** 31 - 1
        slots[0, 4] = -2 ** 31
    k = special_rows(B * Hkv * N, d, 1).view(B, Hkv, N, d)
    v = special_rows(B * Hkv * N, d, 2).flip(0).view(B, Hkv, N, d)
    cache = rng.integers(0, 256, (pages, Hkv, page // 16, 18 * d)).astype(np.uint8)
    g_cache = torch.from_numpy(cache.copy()).to(dev)
    out = [torch.full((B, Hkv, N, d), 7.0, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    plain = g_cache.clone()
    fa.fa_cache4_append(k.to(dev), v.to(dev), plain, i32(slots), gk, gv)
    fa.fa_cache4_append(k.to(dev), v.to(dev), g_cache, i32(slots), gk, gv, *out)
    assert torch.equal(plain, g_cache)
    want = [np.full((B, Hkv, N, d), 7.0) for _ in range(2)]
    for b in range(B):
        for n in range(N):
            if not 0 <= slots[b, n] < pages * page:
                continue
            for h in range(Hkv):
                serve.cache_write(cache, slots[b, n], h, f64(k[b, h, n]),
                                  f64(v[b, h, n]), gk, gv)
                for w, x, g in ((want[0], k, gk), (want[1], v, gv)):
                    w[b, h, n] = serve.dequantise(*serve.quantise(f64(x[b, h, n]), g), g)
    assert np.array_equal(g_cache.cpu().numpy(), cache)
    for g, w in zip(out, want):
        assert np.array_equal(f64(g), w, equal_nan=True)
    # Rows that are 16-byte aligned only.
    odd = [torch.zeros(B * Hkv * N * d + 8, dtype=torch.bfloat16, device=dev)[8:].view_as(k)
           for _ in range(4)]
    odd[0].copy_(k), odd[1].copy_(v)
    odd[2].fill_(7.0), odd[3].fill_(7.0)
    assert odd[0].data_ptr() % 32 == 16
    again = torch.from_numpy(cache.copy()).to(dev)
    fa.fa_cache4_append(odd[0], odd[1], again, i32(slots), gk, gv, odd[2], odd[3])
    assert torch.equal(again, g_cache)
    for x, g in zip(odd[2:], out):
        assert np.array_equal(f64(x), f64(g), equal_nan=True)
    # In place: the values may replace the keys and values themselves.
    k2, v2 = k.to(dev), v.to(dev)
    fa.fa_cache4_append(k2, v2, plain, i32(slots), gk, gv, k2, v2)
    used = torch.from_numpy((slots >= 0) & (slots < pages * page))[:, None, :, None].to(dev)
    for a, b, x in ((k2, out[0], k), (v2, out[1], v)):
        assert np.array_equal(f64(torch.where(used, a, 0)), f64(torch.where(used, b, 0)),
                              equal_nan=True)
        assert np.array_equal(f64(torch.where(used, 0, a)), f64(torch.where(used, 0, x.to(dev))),
                              equal_nan=True)


# ------------------------------------------------------- attention on the GPU
def random_cache(rng, pages, Hkv, page, d, lo=0x28, hi=0x40):
    c = rng.integers(0, 256, (pages, Hkv, page // 16, 18 * d)).astype(np.uint8)
    for at in (slice(8 * d, 9 * d), slice(17 * d, 18 * d)):
        c[..., at] = rng.integers(lo, hi, c[..., at].shape)
    return c


def attn_case(B, H, Hkv, T, d, page, lens, q_lens, window, seed=0, extra=2,
              scales=(0x28, 0x40)):
    rng = np.random.default_rng(seed + 17)
    blocks = max(1, max(-(-n // page) for n in lens)) + extra
    used = sum(-(-n // page) for n in lens)
    pages = used + 3
    ids = rng.permutation(pages)
    table = np.full((B, blocks), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        m = -(-n // page)
        table[b, :m] = ids[at:at + m]
        at += m
    cache = random_cache(rng, pages, Hkv, page, d, *scales)
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((B, H, T, d), generator=g) * 1.5).bfloat16()
    return dict(q=q, cache=cache, table=table, lens=np.array(lens, np.int32),
                q_lens=None if q_lens is None else np.array(q_lens, np.int32),
                window=window, scale=d ** -0.5, gk=0.5, gv=2.0)


def gpu_attn(c, out=None, lse=None, workspace=None):
    dev = torch.device("cuda:0")
    return fa.fa_cache4_attn(
        c["q"].to(dev), torch.from_numpy(c["cache"]).to(dev), i32(c["table"]),
        i32(c["lens"]), c["scale"], None if c["q_lens"] is None else i32(c["q_lens"]),
        c["window"], c["gk"], c["gv"], out, lse, workspace)


def check_attn(c, o, lse, rows_left=7.0):
    q = f64(c["q"])
    B, H, T, d = q.shape
    Hkv = c["cache"].shape[1]
    ro, rl = serve.cache_attention(q, c["cache"], c["table"], c["lens"],
                                   c["q_lens"], c["scale"], c["window"],
                                   c["gk"], c["gv"])
    o, lse = f64(o), f64(lse)
    left = np.isnan(rl)                    # past the request's new tokens
    assert (o[left] == rows_left).all() and (lse[left] == rows_left).all()
    none = np.isneginf(rl)
    assert (o[none] == 0).all() and np.isneginf(lse[none]).all()
    live = ~left & ~none
    k, v = serve.cache_values(c["cache"], c["gk"], c["gv"])
    k, v = np.nan_to_num(np.abs(k)), np.nan_to_num(np.abs(v))
    kmax = k.max((0, 2)).repeat(H // Hkv, 0)[None, :, None]  # [1,H,1,d]
    vmax = v.max((0, 2)).repeat(H // Hkv, 0)[None, :, None]
    es = (d + 8) * 2.0 ** -24 * c["scale"] * (np.abs(q) * kmax).sum(-1)
    assert np.isfinite(o[live]).all() and np.isfinite(lse[live]).all()
    room = es + 2.0 ** -20 * (1 + np.abs(np.where(live, rl, 0)))
    assert (np.abs(lse[live] - rl[live]) <= room[live]).all()
    w = 2.0 ** -11 + 2 * es + 2.0 ** -20 + int(max(c["lens"])) * 2.0 ** -32
    room = 2.0 ** -8 * np.abs(np.where(live[..., None], ro, 0)) + w[..., None] * vmax
    err = np.abs(o - ro)
    assert (err[live] <= room[live]).all(), (err - room)[live].max()


ATTN = [  # B, H, Hkv, T, d, page, lens, q_lens, window
    (1, 1, 1, 1, 128, 16, [1], None, -1),
    (1, 1, 1, 1, 64, 16, [0], None, -1),
    (2, 8, 1, 1, 128, 64, [17, 700], None, -1),
    (3, 12, 4, 1, 64, 32, [0, 64, 65], None, -1),
    (4, 7, 7, 1, 128, 128, [255, 256, 257, 1], None, -1),
    (1, 16, 16, 1, 64, 256, [900], None, 100),
    (2, 16, 1, 1, 128, 16, [333, 15], None, 0),          # 16 rows
    (3, 6, 2, 4, 128, 16, [4, 3, 100], None, -1),        # 12 rows, rows before the start
    (4, 8, 2, 5, 64, 32, [40, 9, 0, 77], [5, 1, 2, 0], 20),
    (2, 10, 2, 5, 128, 64, [300, 70], [3, 5], -1),       # 25 rows: more row blocks
    (2, 4, 1, 33, 64, 16, [33, 129], [33, 20], 40),
    (1, 8, 8, 70, 128, 32, [70], None, -1),              # a prompt through the cache
    (2, 8, 1, 3, 64, 64, [500, 129], [3, 1], -1),        # 24 rows
    (2, 8, 1, 4, 64, 64, [500, 128], None, 33),          # 32 rows
    (1, 12, 2, 4, 128, 32, [700], None, -1),             # 24 rows
    (2, 16, 2, 4, 128, 64, [300, 77], [4, 2], -1),       # 32 rows
    (2, 8, 1, 8, 128, 16, [411, 66], [8, 3], 50),        # 64 rows
    (2, 7, 1, 7, 128, 16, [90, 640], [2, 7], -1),        # 49 rows
    (1, 16, 2, 5, 64, 32, [301], None, -1),              # 40 rows
    (150, 2, 1, 1, 64, 16, [(7 * i) % 90 for i in range(150)], None, -1),
    (700, 1, 1, 2, 64, 16, [(5 * i) % 40 for i in range(700)], [i % 3 for i in range(700)], 9),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", ATTN)
def test_attention_matches_oracle(case):
    c = attn_case(*case)
    out = torch.full(c["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda:0")
    lse = torch.full(c["q"].shape[:3], 7.0, device="cuda:0")
    gpu_attn(c, out, lse)
    assert fa.fa_check_device_status("cuda:0") == OK
    check_attn(c, out, lse)


@pytest.mark.gpu
def test_attention_splits_a_long_history():
    c = attn_case(1, 4, 2, 1, 128, 64, [9001], None, -1, seed=3)
    check_attn(c, *gpu_attn(c))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 3])
def test_unseen_places_may_hold_anything(T):
    """Behind the last token, before the window, and on pages outside the
    cache: NaN scales there change nothing."""
    c = attn_case(2, 4, 2, T, 128, 16, [250, 37], None, 60, seed=4)
    want = gpu_attn(c)
    d, page = 128, 16
    for b, n in enumerate(c["lens"]):
        for j in list(range(0, max(0, n - T - 60))) + list(range(n, -(-n // page) * page)):
            grp = c["cache"][c["table"][b, j // page]][:, j % page // 16]
            _, ksa, _, vsa = serve._places(d, j % 16)
            grp[:, ksa], grp[:, vsa] = 0x7f, 0xff
    unused = sorted(set(range(c["cache"].shape[0])) - set(c["table"].ravel().tolist()))
    c["cache"][unused] = 0xff
    for a, b in zip(want, gpu_attn(c)):
        assert torch.equal(a, b)
    # Pages wholly before the window may be given back.
    c["table"][0, :10] = -1
    c["table"][0, -1] = 1 << 30
    for a, b in zip(want, gpu_attn(c)):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("d,H,T,window,lens", [
    (128, 4, 4, -1, [100, 36]),     # 8 rows
    (128, 8, 5, 7, [40, 300]),      # 16 rows
    (128, 16, 8, 7, [40, 300]),     # 32 rows
    (64, 4, 4, 9, [100, 31]),
    (64, 16, 5, -1, [33, 129]),     # 40 rows
])
def test_a_nan_reaches_the_rows_that_see_it(d, H, T, window, lens):
    """A NaN scale of a key or of a value, at tokens that the first rows, the
    last rows, or (with a window) both do not see."""
    page = 16
    for of_key in (False, True):
        for back in (0, 1, T - 1, T, T + 6):
            c = attn_case(2, H, H // 4, T, d, page, lens, None, window, seed=back)
            clean, cache = gpu_attn(c), c["cache"]
            c["cache"] = cache.copy()
            for b, n in enumerate(lens):
                j = n - 1 - back
                grp = c["cache"][c["table"][b, j // page], 0, j % page // 16]
                _, ksa, _, vsa = serve._places(d, j % 16)
                grp[(ksa if of_key else vsa)[back % (d // 16)]] = 0xff if back & 1 else 0x7f
            ro, rl = serve.cache_attention(
                f64(c["q"]), c["cache"], c["table"], c["lens"], None, c["scale"],
                window, c["gk"], c["gv"])
            o, lse = gpu_attn(c)
            assert np.array_equal(np.isnan(f64(o)), np.isnan(ro))
            assert np.array_equal(np.isnan(f64(lse)), np.isnan(rl))
            # What is left is as without the NaN: with a value's to the bit,
            # with a key's within the tolerance, as rows that share a tile
            # grow their maxima together.
            o, lse = (torch.where(torch.isnan(x), y, x) for x, y in zip((o, lse), clean))
            if not of_key:
                assert torch.equal(o, clean[0]) and torch.equal(lse, clean[1])
            c["cache"] = cache
            check_attn(c, o, lse)


@pytest.mark.gpu
def test_pages_outside_the_cache_hide_their_tokens():
    c = attn_case(2, 4, 1, 1, 64, 16, [130, 60], None, -1, seed=5)
    c["table"][0, 2], c["table"][0, 5] = -3, 10 ** 9
    c["table"][1, :4] = [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1]   # nothing left
    check_attn(c, *gpu_attn(c))


@pytest.mark.gpu
def test_a_window_of_everything_hides_nothing():
    c = attn_case(2, 4, 2, 3, 64, 16, [100, 2], None, -1, seed=12)
    want = gpu_attn(c)
    for c["window"] in (2 ** 31 - 1, 1000, 100, 99):
        for a, b in zip(want, gpu_attn(c)):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_lengths_out_of_range_are_clamped():
    c = attn_case(3, 2, 1, 2, 64, 16, [32, 32, 32], None, -1, seed=6, extra=0)
    c["lens"] = np.array([-5, 2 ** 31 - 1, 32], np.int32)
    c["q_lens"] = np.array([1, 2 ** 31 - 1, -7], np.int32)
    out = torch.full(c["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda:0")
    lse = torch.full(c["q"].shape[:3], 7.0, device="cuda:0")
    gpu_attn(c, out, lse)
    c["lens"] = np.array([0, 32, 32], np.int32)
    c["q_lens"] = np.array([1, 2, 0], np.int32)
    check_attn(c, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("mult", [1e-30, 1e-4, 30.0, 1e4])
def test_attention_over_the_range_of_queries(mult):
    """Rows of very different size, sharp and flat softmaxes."""
    c = attn_case(1, 4, 1, 2, 128, 32, [400], None, -1, seed=7)
    c["q"] = (c["q"].float() * mult).bfloat16()
    c["q"][0, 1] = 0
    c["q"][0, 2, :, 1:] *= 2.0 ** -20      # one dim far above the others
    check_attn(c, *gpu_attn(c))


@pytest.mark.gpu
def test_many_small_weights_do_not_vanish():
    """One key 2^17 times as likely as each of 30000 others with one and the
    same value: the others' weights, 2^-17, still count."""
    n, d, page = 30000, 64, 256
    c = attn_case(1, 1, 1, 1, d, page, [n], None, -1, seed=8, extra=0)
    c["cache"][:] = 0
    c["cache"][..., 8 * d:9 * d] = 0x38    # scales of one
    c["cache"][..., 17 * d:] = 0x38
    c["cache"][..., 9 * d:17 * d] = 0x22   # values of one
    _, _, va, _ = serve._places(d, 5)
    ka = serve._places(d, 5)[0]
    first = c["cache"][c["table"][0, 0], 0, 0]
    first[ka] = 0x22
    first[va] = 0xaa                       # minus one
    c["q"][:] = 1.0
    c["scale"] = 17 * np.log(2) / (d * c["gk"])
    check_attn(c, *gpu_attn(c))


@pytest.mark.gpu
def test_attention_is_repeatable_and_shares_a_workspace_in_order():
    c = attn_case(5, 8, 2, 1, 128, 32, [1000, 3, 0, 555, 2000], None, -1, seed=9)
    ws = torch.full((fa.fa_cache4_attn_workspace_size(5, 8, 2, 1, 128),), 0xff,
                    dtype=torch.uint8, device="cuda:0")
    first = gpu_attn(c, workspace=ws)
    other = attn_case(5, 8, 2, 1, 128, 32, [9, 90, 900, 9, 9], None, -1, seed=10)
    gpu_attn(other, workspace=ws)
    for a, b in zip(first, gpu_attn(c, workspace=ws)):
        assert torch.equal(a, b)
    check_attn(c, *first)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Pages beyond 4 GiB of a cache: the same as a small cache's."""
    Hkv, d, page = 8, 128, 256
    small = attn_case(2, 8, Hkv, 1, d, page, [600, 257], None, -1, seed=11)
    want = gpu_attn(small)
    per = fa.fa_cache4_page_bytes(Hkv, page, d)
    n = small["cache"].shape[0]
    pages = (5 << 30) // per
    big = torch.empty((pages, Hkv, page // 16, 18 * d), dtype=torch.uint8, device="cuda:0")
    big[pages - n:] = torch.from_numpy(small["cache"]).cuda()
    table = torch.where(i32(small["table"]) >= 0, i32(small["table"]) + (pages - n), -1)
    args = (small["q"].cuda(), big, table.contiguous(), i32(small["lens"]), small["scale"])
    got = fa.fa_cache4_attn(*args, k_scale=small["gk"], v_scale=small["gv"])
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    # And written there: the last slots of the cache.
    k = torch.randn((1, Hkv, 3, d), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    slots = i32([[pages * page - 1, pages * page - 18, (pages - 1) * page]])
    fa.fa_cache4_append(k, k, big, slots)
    tiny = torch.zeros((1, Hkv, page // 16, 18 * d), dtype=torch.uint8, device="cuda:0")
    tiny[0] = torch.from_numpy(small["cache"][n - 1]).cuda()
    fa.fa_cache4_append(k, k, tiny, slots - (pages - 1) * page)
    assert torch.equal(big[-1], tiny[0])


@pytest.mark.gpu
def test_two_streams_at_once():
    cs = [attn_case(3, 8, 2, 1, 128, 64, [1500, 700, 90], None, -1, seed=s) for s in (1, 2)]
    want = [gpu_attn(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[], []]
    for _ in range(5):
        for s, c, g in zip(streams, cs, got):
            with torch.cuda.stream(s):
                g.append(gpu_attn(c))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for pair in g:
            assert torch.equal(w[0], pair[0]) and torch.equal(w[1], pair[1])


# ----------------------------------------------------------- a run of them all
class Serving:
    """Requests over one layer: plan, norm and rotation, append, attention."""

    def __init__(self, R, H, Hkv, d, page, pages, max_blocks, T, seed=0):
        dev = torch.device("cuda:0")
        self.R, self.H, self.Hkv, self.d, self.page, self.T = R, H, Hkv, d, page, T
        self.lens, self.table = i32([0] * R), i32([[-1] * max_blocks] * R)
        self.free, self.count = i32(list(range(pages))), i32([pages])
        self.cache = torch.full((pages, Hkv, page // 16, 18 * d), 0xff,
                                dtype=torch.uint8, device=dev)
        self.rope = torch.from_numpy(serve.rope_table(max_blocks * page, d)).to(dev)
        g = torch.Generator().manual_seed(seed)
        self.qw = (1 + 0.1 * torch.randn(d, generator=g)).to(dev)
        self.kw = (1 + 0.1 * torch.randn(d, generator=g)).to(dev)
        self.scale = d ** -0.5
        self.new = i32([0] * R)
        self.qkv = torch.zeros((R, T, H + 2 * Hkv, d), dtype=torch.bfloat16, device=dev)
        self.out = torch.zeros((R, H, T, d), dtype=torch.bfloat16, device=dev)
        self.lse = torch.zeros((R, H, T), device=dev)

    def step(self):
        slots, pos, granted = fa.fa_cache4_plan(
            self.new, self.lens, self.table, self.free, self.count, self.page, self.T)
        q, k, v = fa.fa_qk_norm_rope(self.qkv, self.H, self.Hkv, self.rope, pos,
                                     self.qw, self.kw)
        fa.fa_cache4_append(k, v, self.cache, slots, 1.0, 0.5, k, v)
        fa.fa_cache4_attn(q, self.cache, self.table, self.lens, self.scale,
                          granted, -1, 1.0, 0.5, self.out, self.lse)
        return slots, granted, q, k, v


@pytest.mark.gpu
def test_a_run_of_requests():
    """Prompts, decode steps, an end and a new request.  Every step's output
    equals the attention of all of the request's tokens so far, kept as the
    values that the append returned."""
    R, H, Hkv, d, T = 3, 4, 2, 64, 50
    s = Serving(R, H, Hkv, d, 16, 24, 8, T)
    rng = np.random.default_rng(2)
    hist = [[], [], []]
    steps = [[50, 20, 0], [1, 1, 33], [1, 1, 1], [-200, 3, 1], [40, -2, 1], [5, 5, 5]]
    for i, new in enumerate(steps):
        s.new.copy_(i32(new))
        s.qkv.copy_(torch.from_numpy(rng.standard_normal(s.qkv.shape)).bfloat16())
        s.out.fill_(7.0), s.lse.fill_(7.0)
        slots, granted, q, k, v = s.step()
        assert fa.fa_check_device_status("cuda:0") == OK
        granted = granted.tolist()
        assert granted == [max(0, n) for n in new]
        for r in range(R):
            if new[r] < 0:
                del hist[r][max(0, len(hist[r]) + new[r]):]
            for t in range(granted[r]):
                hist[r].append((f64(k[r, :, t]), f64(v[r, :, t])))
            assert s.lens[r].item() == len(hist[r])
            L = len(hist[r])
            for h in range(H):
                for t in range(T):
                    if t >= granted[r]:
                        assert (s.out[r, h, t] == 7).all() and s.lse[r, h, t] == 7
                        continue
                    n = L - granted[r] + t + 1
                    K = np.array([x[0][h // 2] for x in hist[r][:n]])
                    V = np.array([x[1][h // 2] for x in hist[r][:n]])
                    x = K @ f64(q[r, h, t]) * s.scale
                    w = np.exp(x - x.max())
                    o = w @ V / w.sum()
                    # f16 weights, fp32 scores, bf16 output.
                    room = 2.0 ** -8 * np.abs(o) + 2.0 ** -10 * np.abs(V).max(0)
                    assert (np.abs(f64(s.out[r, h, t]) - o) <= room).all()
                    assert abs(s.lse[r, h, t].item() - (x.max() + np.log(w.sum()))) <= 1e-4


@pytest.mark.gpu
def test_prompt_through_the_cache_equals_the_attention_forward():
    """fa_fwd_varlen on the values that the append returned, against
    fa_cache4_attn over the cache: the same operation, twice."""
    s = Serving(2, 4, 2, 128, 32, 20, 8, 200)
    s.new.copy_(i32([200, 131]))
    s.qkv.copy_(torch.randn(s.qkv.shape, generator=torch.Generator().manual_seed(1)))
    _, granted, q, k, v = s.step()
    o, lse = fa.fa_fwd_varlen(q, k, v, granted, True, s.scale)
    for r, n in enumerate([200, 131]):
        # Either side is within its own rounding of P (bf16: 2^-8 of the
        # weights there) and O.
        a, b = f64(s.out[r, :, :n]), f64(o[r, :, :n])
        vmax = np.abs(f64(v[r, :, :n])).max((1, 2)).repeat(2, 0)[:, None, None]
        assert (np.abs(a - b) <= 2.0 ** -7 * np.abs(b) + (2.0 ** -8 + 2.0 ** -10) * vmax).all()
        assert np.abs(f64(s.lse[r, :, :n]) - f64(lse[r, :, :n])).max() <= 1e-4


@pytest.mark.gpu
def test_captured_decode_steps():
    """One captured step, replayed while the requests grow (lengths, tables
    and slots change on the device only), equals eager steps."""
    a, b = Serving(4, 8, 2, 128, 16, 40, 10, 1), Serving(4, 8, 2, 128, 16, 40, 10, 1)
    for s in (a, b):
        s.new.copy_(i32([1, 1, 0, 1]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.step()
    side.synchronize()
    b.step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side, capture_error_mode="thread_local"):
        a.step()
    for i in range(40):
        x = torch.randn(a.qkv.shape, generator=torch.Generator().manual_seed(i)).bfloat16()
        new = i32([1, 1, i % 2, -1 if i % 5 == 4 else 1])
        for s in (a, b):
            s.qkv.copy_(x)
            s.new.copy_(new)
        g.replay()
        b.step()
        torch.cuda.synchronize()
        for n in ("out", "lse", "lens", "table", "free", "count"):
            assert torch.equal(getattr(a, n), getattr(b, n)), (i, n)
    assert a.lens.tolist()[0] == 41
