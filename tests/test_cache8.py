"""The paged 8-bit cache: format and refusals on the CPU; append, read and
attention on the GPU against the float64 oracle.

Codes, exponents and values read back have to be equal.  The attention's
tolerances: K, V and Q enter the products exactly.  A score is a sum of d
products in fp32, within es = (d + 8) 2^-24 scale sum |q||k| of its value, so
a weight is within 2 es + 2^-20 (exponential, sums) of its own; P, times its
group's power of two, is rounded to f16 (half a step: 2^-11 of the product, or
less than 2^-32 of the largest that the row has where it vanishes); O is
rounded to bf16 (2^-8).  The LSE is within es + 2^-20 (1 + |lse|).
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import cache8, serve
from tiled_attention_bwd_gb300 import build as fa_build
from tiled_attention_bwd_gb300 import fa

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5
DEV = "cuda:0"


def f64(t):
    return t.detach().to("cpu").double().numpy()


def i32(x, dev=DEV):
    return torch.tensor(np.ascontiguousarray(x), dtype=torch.int32, device=dev)


# ------------------------------------------------------------------- on CPU
def test_codes_round_to_nearest_even():
    # Half way between 1 and 1.125 (even: 1), and 1.125 and 1.25 (even: 1.25).
    x = [1.0625, 1.1875, 448.0, 1e9, -np.inf, 2.0 ** -10, 3 * 2.0 ** -11, 0.0]
    want = [1.0, 1.25, 448.0, 448.0, -448.0, 0.0, 2.0 ** -9, 0.0]
    assert np.array_equal(cache8.decode(cache8.encode(x, 0), 0), want)
    assert np.isnan(cache8.decode(cache8.encode(np.nan, 3), 3))


def test_the_exponent_is_the_smallest_that_holds_the_largest():
    for e in (-60, -9, 0, 13):
        top = 448.0 * 2.0 ** e
        assert cache8.exponent(top) == e
        assert cache8.exponent(np.nextafter(top, 1e300)) == e + 1
    assert cache8.exponent(0.0) == -60 and cache8.exponent(1e38) == 60


def test_every_value_is_a_bf16():
    for e in (-60, 0, 60):
        v = torch.from_numpy((serve.E4M3 * 2.0 ** e).astype(np.float32))
        assert torch.equal(v.bfloat16().float(), v)


def test_growth_keeps_codes_above_the_small_ones():
    c = np.arange(127, dtype=np.uint8)
    for up in (1, 4, 9):
        new = cache8.encode(cache8.decode(c, 0), up)
        kept = serve.E4M3 >= 2.0 ** (up - 6)
        assert np.array_equal(cache8.decode(new, up)[kept], serve.E4M3[kept])


@pytest.mark.parametrize("d", [64, 128])
def test_layout_places_every_byte_once(d):
    seen = np.zeros(32 * d + 16, int)
    for tok in range(16):
        for at in cache8.places(d, tok):
            seen[at] += 1
    assert (seen[:32 * d] == 1).all() and (seen[32 * d:] == 0).all()


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fa.load_library()


def p(x):
    return ctypes.c_void_p(x) if x else None


def _append(lib, k=16, v=16, cache=1 << 20, slots=16, ko=0, vo=0, B=1, Hkv=1,
            N=1, d=128, pages=1, page=16):
    return lib.fa_cache8_append(p(k), p(v), p(cache), p(slots), p(ko), p(vo), B,
                                Hkv, N, d, pages, page, None)


@pytest.mark.parametrize("want,bad", [
    (UNSUPPORTED, dict(d=96)), (INVALID, dict(d=0)),
    (UNSUPPORTED, dict(page=24)), (INVALID, dict(pages=-1)),
    (UNSUPPORTED, dict(pages=1 << 28)), (INVALID, dict(ko=16)),
    (INVALID, dict(vo=16)), (INVALID, dict(k=0)), (INVALID, dict(v=8)),
    (INVALID, dict(cache=0)), (INVALID, dict(cache=8)),
    (INVALID, dict(slots=2)), (INVALID, dict(ko=1032, vo=2048)),
    (INVALID, dict(B=-1)), (INVALID, dict(N=-1)), (INVALID, dict(Hkv=-1)),
    (INVALID, dict(k=256, v=512, ko=512, vo=1024)),
    (INVALID, dict(k=256, v=512, ko=1024, vo=1264)),
    (INVALID, dict(k=256, v=512, ko=256, vo=528)),
    (INVALID, dict(k=(1 << 20) + 4096)),
    (INVALID, dict(slots=(1 << 20) + 4108)),
    (INVALID, dict(ko=1 << 20, vo=1 << 16)),
    (UNSUPPORTED, dict(B=1 << 20, N=1 << 12)),
    (UNSUPPORTED, dict(N=2 ** 31 - 32)),
])
def test_append_refusals(lib, want, bad):
    assert _append(lib, **bad) == want


def _read(lib, cache=1 << 20, table=16, lens=16, starts=0, ko=4096, vo=8192, B=1,
          Hkv=1, N=1, d=128, M=1, pages=1, page=16):
    return lib.fa_cache8_read(p(cache), p(table), p(lens), p(starts), p(ko),
                              p(vo), B, Hkv, N, d, M, pages, page, None)


@pytest.mark.parametrize("want,bad", [
    (UNSUPPORTED, dict(d=80)), (UNSUPPORTED, dict(page=512)),
    (INVALID, dict(page=0)), (INVALID, dict(N=-1)), (INVALID, dict(M=-1)),
    (INVALID, dict(cache=0)), (INVALID, dict(table=0)),
    (INVALID, dict(lens=0)), (INVALID, dict(ko=0)), (INVALID, dict(vo=0)),
    (INVALID, dict(ko=8)), (INVALID, dict(starts=2)), (INVALID, dict(lens=18)),
    (INVALID, dict(vo=4096)), (INVALID, dict(ko=1 << 20)),
    (INVALID, dict(table=4100)), (INVALID, dict(lens=8196)),
    (INVALID, dict(starts=4096)), (UNSUPPORTED, dict(M=1 << 28)),
    (UNSUPPORTED, dict(B=1 << 16, Hkv=1 << 16)),
    (UNSUPPORTED, dict(B=1 << 20, N=1 << 16)),
    (UNSUPPORTED, dict(N=2 ** 31 - 1)),
])
def test_read_refusals(lib, want, bad):
    assert _read(lib, **bad) == want


def _attn(lib, q=16, cache=1 << 20, table=16, lens=16, ql=16, o=4096, lse=16384,
          ws=1 << 30, wsb=1 << 40, B=1, H=2, Hkv=1, T=1, d=128, M=1, pages=1,
          page=16, window=-1, scale=0.1):
    return lib.fa_cache8_attn(p(q), p(cache), p(table), p(lens), p(ql), p(o),
                              p(lse), p(ws), wsb, B, H, Hkv, T, d, M, pages,
                              page, window, scale, None)


@pytest.mark.parametrize("want,bad", [
    (UNSUPPORTED, dict(d=80)), (UNSUPPORTED, dict(page=1)),
    (INVALID, dict(Hkv=0)), (INVALID, dict(H=3, Hkv=2)),
    (INVALID, dict(T=-1)), (INVALID, dict(scale=0.0)),
    (INVALID, dict(scale=float("nan"))), (INVALID, dict(scale=3e38)),
    (INVALID, dict(q=0)), (INVALID, dict(q=8)), (INVALID, dict(cache=0)),
    (INVALID, dict(table=0)), (INVALID, dict(lens=0)), (INVALID, dict(ql=2)),
    (INVALID, dict(o=0)), (INVALID, dict(o=4104)), (INVALID, dict(lse=0)),
    (INVALID, dict(o=(1 << 20) + 4096)), (INVALID, dict(lse=4600)),
    (WORKSPACE, dict(ws=0)), (WORKSPACE, dict(ws=16)),
    (WORKSPACE, dict(wsb=100)), (INVALID, dict(ws=1 << 20)),
    (UNSUPPORTED, dict(M=1 << 28)), (UNSUPPORTED, dict(pages=1 << 28)),
    (UNSUPPORTED, dict(M=(1 << 27) - 8, page=16)),
    (UNSUPPORTED, dict(B=1 << 20, H=1 << 12)),
    (UNSUPPORTED, dict(B=1 << 20, M=1 << 10, page=256)),
])
def test_attention_refusals(lib, want, bad):
    assert _attn(lib, **bad) == want


def test_empty_calls_and_sizes(lib):
    assert _append(lib, N=0, k=0, v=0) == OK
    assert _append(lib, pages=0, cache=0) == OK
    assert _read(lib, B=0, ko=0) == OK and _read(lib, N=0, vo=0) == OK
    assert _read(lib, M=0, table=0) == OK
    assert _attn(lib, B=0, q=0) == OK and _attn(lib, T=0, q=0, ws=0) == OK
    assert lib.fa_cache8_page_bytes(8, 64, 128) == 8 * 4 * 4112
    assert lib.fa_cache8_page_bytes(2, 16, 64) == 2 * 2064
    assert lib.fa_cache8_page_bytes(2, 24, 64) == 0
    assert lib.fa_cache8_page_bytes(0, 16, 64) == 0
    assert lib.fa_cache8_attn_workspace_size(1, 4, 3, 1, 128) == 0


def test_binding_refusals():
    z = torch.zeros
    with pytest.raises(ValueError):        # not on a GPU
        fa.fa_cache8_append(z(1), z(1), z((1, 1, 1, 2064), dtype=torch.uint8), z(1))
    with pytest.raises(ValueError):
        fa.fa_cache8_read(z((1, 1, 1, 2064), dtype=torch.uint8), z(1), z(1), 4)


# ---------------------------------------------------------- append on the GPU
def rows(n, d, seed, special=True):
    """Rows of different sizes, some at the format's corners."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, d), generator=g) * torch.exp2(
        torch.randint(-10, 8, (n, 1), generator=g).float())
    # Ties between codes once the largest is 448 2^e.
    tie = torch.randint(-255, 256, (n, d), generator=g) / 128.0
    tie[:, 0] = 448.0 / 256
    x = torch.where(torch.arange(n)[:, None] % 3 == 1, tie, x)
    if special and n > 5:
        x[0] = 0.0
        x[1, 3], x[1, 20] = float("inf"), -float("inf")
        x[2, 5], x[2, 40] = float("nan"), 1e-30
        x[3] = -0.0
        x[4, 17] = 3e38
        x[5] = torch.randn(d, generator=g) * 1e-38
    return x.bfloat16()


def same(got, want):
    return np.array_equal(f64(got), want, equal_nan=True)


def same_cache(got, want, d):
    """Equal bytes; a NaN's sign is not kept."""
    a, b = got.cpu().numpy(), want
    nan = ((a & 127) == 127) & ((b & 127) == 127)
    nan[..., 32 * d:] = False
    return np.array_equal(np.where(nan, 0, a), np.where(nan, 0, b))


def used_cache(rng, pages, Hkv, page, d, lo=-4, hi=4, nan=False):
    c = rng.integers(0, 256, (pages, Hkv, page // 16, 32 * d + 16)).astype(np.uint8)
    if not nan:
        codes = c[..., :32 * d]
        codes[(codes & 127) == 127] -= 1
    c[..., 32 * d:32 * d + 2] = rng.integers(lo, hi + 1, c[..., :2].shape).astype(np.int8).view(np.uint8)
    return c


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hkv,N,d,page,lo,hi", [
    (1, 1, 1, 128, 16, -4, 4), (2, 3, 1, 64, 32, -60, 60),
    (3, 2, 37, 128, 64, -12, 3), (1, 4, 130, 64, 256, -20, 0),
    (5, 1, 20, 64, 16, -128, 127), (7, 2, 16, 128, 128, -2, 30),
])
def test_append_matches_oracle(B, Hkv, N, d, page, lo, hi):
    """Runs of tokens from any place of a page on, in order."""
    rng = np.random.default_rng(N)
    per = -(-N // page) + 1
    pages = B * per + 2
    ids = rng.permutation(pages)
    slots = np.full((B, N), -1, np.int64)
    for b in range(B):
        start, n = rng.integers(0, page), rng.integers(max(1, N // 2), N + 1)
        pos = start + np.arange(n)
        slots[b, :n] = ids[b * per + pos // page] * page + pos % page
    if N > 5:
        slots[0, 1] = pages * page         # behind the cache: skipped
        slots[0, 2] = 2 ** 31 - 1
        slots[0, 4] = -2 ** 31
    check_append(rng, slots, B, Hkv, N, d, pages, page, lo, hi)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_append_in_any_order_within_sixteen(d):
    """A group's tokens backwards, shuffled, with others between them."""
    rng = np.random.default_rng(5)
    page, pages, B, N = 32, 12, 3, 64
    slots = np.full((B, N), -1, np.int64)
    slots[0, :16] = 32 + np.arange(16)[::-1]
    slots[0, 16:32] = 64 + rng.permutation(16)
    slots[1, 5:21] = np.stack([96 + np.arange(8), 128 + 3 + np.arange(8)], 1).ravel()
    slots[1, 40:56:5] = [163, 161, 174, 160]
    slots[2] = 192 + np.stack([np.arange(16), 16 + np.arange(16), 32 + np.arange(16),
                               48 + np.arange(16)]).ravel()
    check_append(rng, slots, B, 2, N, d, pages, page, -6, 6)


def check_append(rng, slots, B, Hkv, N, d, pages, page, lo, hi):
    slots = slots.astype(np.int32)
    k = rows(B * Hkv * N, d, 1).view(B, Hkv, N, d)
    v = rows(B * Hkv * N, d, 2).flip(0).view(B, Hkv, N, d)
    cache = used_cache(rng, pages, Hkv, page, d, lo, hi, nan=True)
    first = cache.copy()
    held = cache8.append(cache, slots, f64(k), f64(v))
    skipped = (slots < 0) | (slots >= pages * page)
    keep = np.broadcast_to(skipped[:, None, :, None], held[0].shape)
    want = [np.where(keep, 7.0, x) for x in held]
    g_k, g_v, g_slots = k.to(DEV), v.to(DEV), i32(slots)
    plain, full = (torch.from_numpy(first.copy()).to(DEV) for _ in range(2))
    out = [torch.full((B, Hkv, N, d), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    fa.fa_cache8_append(g_k, g_v, plain, g_slots)
    fa.fa_cache8_append(g_k, g_v, full, g_slots, *out)
    assert torch.equal(plain, full)
    assert same_cache(full, cache, d)
    assert same(out[0], want[0]) and same(out[1], want[1])
    # Again: nothing changes, the groups' exponents hold these tokens.
    fa.fa_cache8_append(g_k, g_v, full, g_slots, *out)
    assert torch.equal(plain, full)
    # Rows that are 16-byte aligned only, and in place.
    odd = [torch.zeros(B * Hkv * N * d + 8, dtype=torch.bfloat16, device=DEV)[8:].view_as(k)
           for _ in range(2)]
    odd[0].copy_(k), odd[1].copy_(v)
    again = torch.from_numpy(first.copy()).to(DEV)
    fa.fa_cache8_append(odd[0], odd[1], again, g_slots, *odd)
    assert torch.equal(again, full)
    for x, w, raw in zip(odd, want, (k, v)):
        assert same(x, np.where(keep, f64(raw), w))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_append_token_by_token(d):
    """Decode steps whose sizes grow, fall and grow again; a token taken back
    and written anew; a page that another request begins."""
    rng = np.random.default_rng(11)
    page, pages, Hkv, B = 16, 6, 2, 3
    cache = np.zeros((pages, Hkv, 1, 32 * d + 16), np.uint8)
    g_cache = torch.from_numpy(cache.copy()).to(DEV)
    pos = np.array([0, 3, 14])
    for step in range(24):
        size = 2.0 ** rng.integers(-9, 6)
        k, v = ((torch.randn((B, Hkv, 1, d), generator=torch.Generator().manual_seed(2 * step + i))
                 * size).bfloat16() for i in (0, 1))
        slots = ((pos // page * B + np.arange(B)) % pages * page + pos % page)[:, None].astype(np.int32)
        cache8.append(cache, slots, f64(k), f64(v))
        fa.fa_cache8_append(k.to(DEV), v.to(DEV), g_cache, i32(slots))
        assert same_cache(g_cache, cache, d), step
        pos += 1
        if step % 7 == 6:
            pos -= 2


# ------------------------------------------------------------ read on the GPU
def tables(rng, lens, page, extra, spare):
    blocks = max(1, max(-(-n // page) for n in lens)) + extra
    pages = sum(-(-n // page) for n in lens) + spare
    ids, at = rng.permutation(pages), 0
    table = np.full((len(lens), blocks), -1, np.int32)
    for b, n in enumerate(lens):
        m = -(-n // page)
        table[b, :m] = ids[at:at + m]
        at += m
    return table, pages


@pytest.mark.gpu
@pytest.mark.parametrize("Hkv,N,d,page,lens,starts", [
    (1, 1, 128, 16, [1], None), (2, 40, 64, 32, [40, 17, 0], None),
    (3, 33, 128, 64, [70, 200, 33], [5, 167, 1]),
    (1, 300, 64, 256, [299, 700], [16, 401]),
    (2, 20, 128, 16, [20, 50, 9, 64], [0, 45, 9, 1 << 30]),
    (1, 15, 64, 128, [100, 128], [-5, 2 ** 31 - 1]),
])
def test_read_matches_oracle(Hkv, N, d, page, lens, starts):
    rng = np.random.default_rng(N)
    table, pages = tables(rng, lens, page, 2, 3)
    cache = used_cache(rng, pages, Hkv, page, d, -60, 60, nan=True)
    if len(lens) > 2:
        table[1, 0] = pages                # a page that is not there
    k, v, done = cache8.read(cache, table, lens, starts, N)
    out = [torch.full(k.shape, 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    fa.fa_cache8_read(torch.from_numpy(cache).to(DEV), i32(table), i32(lens), N,
                      None if starts is None else i32(starts), *out)
    for got, w in zip(out, (k, v)):
        assert same(got, np.where(done[:, None, :, None], w, 7.0))


@pytest.mark.gpu
def test_read_returns_what_append_held():
    B, Hkv, N, d, page = 3, 2, 50, 128, 32
    rng = np.random.default_rng(2)
    table, pages = tables(rng, [N] * B, page, 0, 1)
    pos = np.arange(N)
    slots = (table[:, pos // page] * page + pos % page).astype(np.int32)
    k, v = (rows(B * Hkv * N, d, s, special=False).view(B, Hkv, N, d).to(DEV) for s in (1, 2))
    cache = torch.zeros((pages, Hkv, page // 16, 32 * d + 16), dtype=torch.uint8, device=DEV)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    fa.fa_cache8_append(k, v, cache, i32(slots), ko, vo)
    k2, v2 = fa.fa_cache8_read(cache, i32(table), i32([N] * B), N)
    assert torch.equal(k2, ko) and torch.equal(v2, vo)
    # A value is within half a step of its own, or of the smallest step.
    for x, y in ((k, ko), (v, vo)):
        amax = x.double().abs().view(B, Hkv, N, d).amax((2, 3), keepdim=True)
        assert ((x.double() - y.double()).abs()
                <= torch.maximum(x.double().abs() * 2.0 ** -4, amax * 2.0 ** -17)).all()


# ------------------------------------------------------- attention on the GPU
def attn_case(B, H, Hkv, T, d, page, lens, q_lens, window, seed=0, extra=2, exps=(-3, 2)):
    rng = np.random.default_rng(seed + 17)
    table, pages = tables(rng, lens, page, extra, 3)
    cache = used_cache(rng, pages, Hkv, page, d, *exps)
    # Codes of a few units, so that a softmax has more than one term.
    codes = cache[..., :32 * d]
    codes[...] = (codes & 0x80) | (0x20 + codes % 0x18)
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((B, H, T, d), generator=g) * 1.5).bfloat16()
    return dict(q=q, cache=cache, table=table, lens=np.array(lens, np.int32),
                q_lens=None if q_lens is None else np.array(q_lens, np.int32),
                window=window, scale=d ** -0.5)


def gpu_attn(c, out=None, lse=None, workspace=None):
    if out is None:
        out = torch.full(c["q"].shape, 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full(c["q"].shape[:3], 7.0, device=DEV)
    return fa.fa_cache8_attn(
        c["q"].to(DEV), torch.from_numpy(c["cache"]).to(DEV), i32(c["table"]),
        i32(c["lens"]), c["scale"], None if c["q_lens"] is None else i32(c["q_lens"]),
        c["window"], out, lse, workspace)


def check_attn(c, o, lse, rows_left=7.0):
    q = f64(c["q"])
    B, H, T, d = q.shape
    Hkv = c["cache"].shape[1]
    ro, rl, mag = cache8.attention(q, c["cache"], c["table"], c["lens"],
                                   c["q_lens"], c["scale"], c["window"])
    o, lse = f64(o), f64(lse)
    left = np.isnan(rl)                    # past the request's new tokens
    assert (o[left] == rows_left).all() and (lse[left] == rows_left).all()
    none = np.isneginf(rl)
    assert (o[none] == 0).all() and np.isneginf(lse[none]).all()
    live = ~left & ~none
    assert np.isfinite(o[live]).all() and np.isfinite(lse[live]).all()
    k, _ = cache8.values(c["cache"])
    kmax = np.nan_to_num(np.abs(k)).max((0, 2)).repeat(H // Hkv, 0)[None, :, None]
    es = (d + 8) * 2.0 ** -24 * c["scale"] * (np.abs(q) * kmax).sum(-1)
    room = es + 2.0 ** -20 * (1 + np.abs(np.where(live, rl, 0)))
    assert (np.abs(lse[live] - rl[live]) <= room[live]).all()
    # The largest product of the row is at most its weight times 448 2^e; some
    # dim of some value of its head reaches an eighth of that here.
    w = 2.0 ** -11 + 2 * es + 2.0 ** -20
    top = mag.max(-1, keepdims=True) * 448 / 2 ** -3
    room = (2.0 ** -8 * np.abs(np.where(live[..., None], ro, 0)) + w[..., None] * mag
            + int(max(c["lens"])) * 2.0 ** -32 * top)
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
    (3, 6, 2, 4, 128, 16, [4, 3, 100], None, -1),        # rows before the start
    (4, 8, 2, 5, 64, 32, [40, 9, 0, 77], [5, 1, 2, 0], 20),
    (2, 10, 2, 5, 128, 64, [300, 70], [3, 5], -1),       # 25 rows
    (2, 4, 1, 33, 64, 16, [33, 129], [33, 20], 40),
    (1, 8, 1, 40, 128, 32, [400], None, -1),             # many row blocks
    (3, 8, 2, 70, 128, 64, [500, 70, 130], [70, 70, 1], 90),
    (2, 5, 1, 64, 64, 16, [64, 300], [64, 31], -1),
    (2, 16, 2, 150, 128, 64, [600, 151], None, -1),      # rows of several tiles
    (1, 3, 1, 129, 64, 128, [1000], None, 77),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hkv,T,d,page,lens,q_lens,window", ATTN)
def test_attention_matches_oracle(B, H, Hkv, T, d, page, lens, q_lens, window):
    c = attn_case(B, H, Hkv, T, d, page, lens, q_lens, window)
    check_attn(c, *gpu_attn(c))
    assert fa.fa_check_device_status(DEV) == OK


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 3, 40, 130])
def test_exponents_far_apart(T):
    """Values whose groups differ by 2^40: the largest products decide."""
    c = attn_case(2, 4, 2, T, 128, 32, [200, 131], None, -1, exps=(-3, -3))
    rng = np.random.default_rng(3)
    e = rng.integers(-20, 21, c["cache"][..., 0].shape)
    c["cache"][..., 32 * 128 + 1] = e.astype(np.int8).view(np.uint8)
    check_attn(c, *gpu_attn(c))


@pytest.mark.gpu
@pytest.mark.parametrize("ke,ve", [(-60, 60), (60, -60), (20, 0), (-128, 127)])
@pytest.mark.parametrize("T", [1, 140])
def test_exponents_at_the_ends(ke, ve, T):
    """All of one size, and bytes that no append writes (brought into range)."""
    c = attn_case(1, 2, 1, T, 64, 16, [150], None, -1)
    c["cache"][..., 32 * 64] = np.int8(ke).view(np.uint8)
    c["cache"][..., 32 * 64 + 1] = np.int8(ve).view(np.uint8)
    if ke > 0:                             # scores of an ordinary size
        c["q"] = (c["q"].float() * 2.0 ** -min(ke, 60)).bfloat16()
    check_attn(c, *gpu_attn(c))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 4, 20, 130])
@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_reaches_the_rows_that_see_it(T, d):
    """Everything that no row sees is NaN; a seen NaN key spoils its rows, a
    seen NaN value its dim of them, and nothing else."""
    L, page = 180 + T, 32
    c = attn_case(1, 4, 2, T, d, page, [L], None, -1)
    cache, table = c["cache"], c["table"][0]
    clean = cache.copy()
    held = set(table[:-(-L // page)])
    for pg in range(cache.shape[0]):
        if pg not in held:
            cache[pg] = 0xff
    last = table[L // page] if L % page else None
    if last is not None:
        for tok in range(L % page, page):
            for at in cache8.places(d, tok % 16):
                cache[last, :, tok // 16, at] = 0x7f
    check_attn(c, *gpu_attn(c))
    # Token L - 2 is seen by all rows but those before it.
    tok = L - 2
    grp = cache[table[tok // page], 0, tok % page // 16]
    ka, va = cache8.places(d, tok % 16)
    grp[va[5]] = 0xff
    o, lse = (f64(x) for x in gpu_attn(c))
    sees = np.arange(T) + L - T >= tok
    assert np.isfinite(lse).all()
    bad = np.zeros(o.shape, bool)
    bad[0, :2, sees, 5] = True
    assert np.array_equal(np.isnan(o), bad)
    grp[va[5]] = clean[table[tok // page], 0, tok % page // 16, va[5]]
    grp[ka[7]] = 0x7f
    o, lse = (f64(x) for x in gpu_attn(c))
    bad = np.zeros(lse.shape, bool)
    bad[0, :2, sees] = True
    assert np.array_equal(np.isnan(lse), bad)
    assert np.array_equal(np.isnan(o), np.broadcast_to(bad[..., None], o.shape))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 6, 150])
def test_pages_outside_the_cache_hide_their_tokens(T):
    c = attn_case(2, 4, 2, T, 128, 16, [100, 170], None, -1)
    c["table"][0, 2], c["table"][1, 0] = 2 ** 30, -7
    c["table"][1, 9] = c["cache"].shape[0]
    check_attn(c, *gpu_attn(c))


@pytest.mark.gpu
def test_lengths_are_brought_into_range():
    c = attn_case(3, 4, 2, 2, 64, 16, [64, 20, 5], [2, 1, 2], -1, extra=0)
    c["lens"][:] = [2 ** 31 - 1, -3, 5]
    c["q_lens"][:] = [-4, 1, 2 ** 31 - 1]
    c["lens"][0] = 2 ** 31 - 1
    check_attn(c, *gpu_attn(c))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 9, 200])
def test_same_result_every_time_and_with_a_used_workspace(T):
    c = attn_case(5, 8, 2, T, 128, 64, [900, 1, 300, 2500, 64], None, -1)
    need = fa.fa_cache8_attn_workspace_size(5, 8, 2, T, 128)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    o, lse = gpu_attn(c)
    for _ in range(3):
        o2, lse2 = gpu_attn(c, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.gpu
def test_zeros_hold_zeros():
    c = attn_case(1, 2, 1, 1, 128, 16, [40], None, -1)
    c["cache"][...] = 0
    o, lse = gpu_attn(c)
    assert (o == 0).all()
    assert np.abs(f64(lse) - np.log(40)).max() <= 2.0 ** -18


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes, its last pages in use."""
    d, Hkv, page = 128, 8, 256
    pages = 2 ** 32 // (Hkv * 16 * 4112) + 40
    cache = torch.zeros((pages, Hkv, page // 16, 32 * d + 16), dtype=torch.uint8, device=DEV)
    assert cache.numel() > 2 ** 32
    n, T = 300, 2
    table = i32([[pages - 1, pages - 2]])
    pos = np.arange(n)
    slots = np.where(pos < page, (pages - 1) * page + pos, (pages - 2) * page + pos - page)[None]
    k, v = (rows(Hkv * n, d, s, special=False).view(1, Hkv, n, d) for s in (1, 2))
    fa.fa_cache8_append(k.to(DEV), v.to(DEV), cache, i32(slots))
    small = cache[-2:].cpu().numpy()
    want = np.zeros_like(small)
    cache8.append(want, slots - (pages - 2) * page, f64(k), f64(v))
    assert same_cache(cache[-2:], want, d) and not cache[:-2].any()
    gk, gv = fa.fa_cache8_read(cache, table, i32([n]), n)
    wk, wv, _ = cache8.read(small, [[1, 0]], [n], None, n)
    assert same(gk, wk) and same(gv, wv)
    q = (torch.randn((1, 8, T, d), generator=torch.Generator().manual_seed(1))).bfloat16()
    o, lse = fa.fa_cache8_attn(q.to(DEV), cache, table, i32([n]), 0.05)
    c = dict(q=q, cache=small, table=np.array([[1, 0]]), lens=np.array([n]), q_lens=None,
             window=-1, scale=0.05)
    check_attn(c, o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("T,site", [(1, 0x521)] + [(300, s) for s in range(
    0x531, 0x53e)])
def test_a_stopped_attention_reports_and_recovers(T, site):
    """The kernels' stopping paths, by the test hook (no fault, no hang)."""
    c = attn_case(2, 8, 1, T, 128, 64, [30000, 700], None, -1)
    o, lse = gpu_attn(c)
    torch.cuda.synchronize()
    fa.fa_debug_expire_at(site)
    try:
        gpu_attn(c)
        assert fa.fa_check_device_status(DEV) == 4
        assert fa.fa_last_failure_site() == site
    finally:
        torch.cuda.synchronize()
        fa.fa_debug_expire_at(0)
    o2, lse2 = gpu_attn(c)
    assert fa.fa_check_device_status(DEV) == OK
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
