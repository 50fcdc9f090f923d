"""The attention over the 8-bit cache within what its roundings allow, on
histories whose every unit of 128 keys can be missed.

Tolerances.  K, V and Q enter the products exactly.  A score is within es =
(d + 8) 2^-24 scale sum |q||k| of its value, so a weight is within 2 es + 2^-20
of its own (exponential and reference; test_cache8.py).  Sums over L keys are
taken 16 keys at a time, in L / 16 steps at most and some to join parts, each
off by half a step of fp32, or a whole one inside a matrix product: n 2^-24 of l
and n 2^-23 of the terms of O, n = L / 16 + 64.

P is f16 of p 2^e_v over a reference that the row's largest product stands
2^8 to 2^15 above.  Products down to 2^-22 of the largest are normal numbers in
f16: off by half a step, 2^-11 of each.  Smaller ones are off by at most half of
f16's smallest step, 2^-25, times a code of at most 448, in units 2^-8 of the
largest: 448 2^-33 of it each.  O is rounded to bf16 (2^-8).
"""
import numpy as np
import pytest
import torch

from oracle import cache8
from test_cache8 import ATTN, DEV, OK, attn_case, f64, gpu_attn
from test_cache8_split import MIXED, TURNS
from tiled_attention_bwd_gb300 import fa

UNIT = 128


def allowed(c):
    """O and LSE in float64, and how far either may be off."""
    q = f64(c["q"])
    d, Hkv = q.shape[-1], c["cache"].shape[1]
    ro, rl, mag, top, few = cache8.products(q, c["cache"], c["table"], c["lens"], c["q_lens"],
                                            c["scale"], c["window"])
    k, _ = cache8.values(c["cache"])
    kmax = np.nan_to_num(np.abs(k)).max((0, 2)).repeat(q.shape[1] // Hkv, 0)[None, :, None]
    es = (d + 8) * 2.0 ** -24 * c["scale"] * (np.abs(q) * kmax).sum(-1)
    n = max(c["lens"]) / 16 + 64
    live = np.isfinite(rl)
    room_l = es + 2.0 ** -20 * (1 + np.abs(np.where(live, rl, 0))) + n * 2.0 ** -24
    w = 2.0 ** -11 + 2 * es + 2.0 ** -20 + n * (2.0 ** -24 + 2.0 ** -23)
    room_o = (2.0 ** -8 * np.abs(np.where(live[..., None], ro, 0)) + w[..., None] * mag
              + (few * top * 448 * 2.0 ** -33)[..., None])
    return ro, rl, room_o, room_l


def check(c, o, lse, rows_left=7.0, within=None):
    ro, rl, room_o, room_l = within or allowed(c)
    o, lse = f64(o), f64(lse)
    left, none = np.isnan(rl), np.isneginf(rl)
    assert (o[left] == rows_left).all() and (lse[left] == rows_left).all()
    assert (o[none] == 0).all() and np.isneginf(lse[none]).all()
    live = ~left & ~none
    # (Not a number compares false.)
    assert (np.abs(lse[live] - rl[live]) <= room_l[live]).all()
    err = np.abs(o[live] - ro[live])
    assert (err <= room_o[live]).all(), (err / room_o[live]).max()


def one_sign(c):
    """Values of one sign per dim: O is not far below its terms."""
    d = c["q"].shape[-1]
    for tok in range(16):
        at = cache8.places(d, tok)[1]
        signs = np.where(np.arange(d) % 3 == 0, 0x80, 0).astype(np.uint8)
        c["cache"][..., at] = (c["cache"][..., at] & 0x7f) | signs
    return c


def marked(c):
    """The same, and a dim has values in every d-th unit of keys only: a unit
    that is missing, or counts twice, is much of that dim's O."""
    one_sign(c)
    d, page = c["q"].shape[-1], 16 * c["cache"].shape[2]
    at = np.stack([cache8.places(d, tok)[1] for tok in range(16)])
    for row, n in zip(c["table"], c["lens"]):
        for tok in range(0, n, 16):
            off = np.arange(d) != tok // UNIT % d
            c["cache"][row[tok // page], :, tok % page // 16, at[:, off]] = 0
    return c


# ------------------------------------------------------------------- on CPU
def test_the_matrix_form_is_the_plain_one():
    for case in (ATTN[7], ATTN[8], ATTN[5]):
        c = attn_case(*case)
        args = (f64(c["q"]), c["cache"], c["table"], c["lens"], c["q_lens"], c["scale"], c["window"])
        for a, b in zip(cache8.attention(*args), cache8.products(*args)):
            assert np.allclose(a, b, rtol=1e-12, atol=1e-14, equal_nan=True)


@pytest.mark.parametrize("make", [one_sign, marked])
@pytest.mark.parametrize("d,T,L", [(128, 2, 40000), (64, 1, 30000)])
def test_the_check_misses_nothing(make, d, T, L):
    """An output with its roundings passes; one that lacks a part, or has it
    twice, is refused."""
    c = make(attn_case(1, 1, 1, T, d, 256, [L], None, -1))
    c["q"] = c["q"] * 0.25
    within = ro, rl, _, _ = allowed(c)
    lse = torch.from_numpy(rl).float()
    check(c, torch.from_numpy(ro).bfloat16(), lse, within=within)
    # Keys lo .. hi - 1 in float64, as they count in O.
    k, v = cache8.values(c["cache"])
    at = np.arange(L)
    pg = c["table"][0][at // 256]
    K, V = k[pg, 0, at % 256], v[pg, 0, at % 256]
    pos = L - T + np.arange(T)
    s = np.where(at <= pos[:, None], f64(c["q"])[0, 0] @ K.T * c["scale"], -np.inf)
    p = np.exp(s - rl[0, 0][:, None])

    def part(lo, hi):
        return (p[:, lo:hi] @ V[lo:hi])[None, None]

    wrong = [ro - part(0, L // 2), 1.5 * ro, 1.01 * ro]
    share = -(-L // 148)                   # of a block
    wrong += [ro - part(7 * share, 8 * share), ro + part(0, share)]
    if make is marked:
        wrong += [ro - part(40 * UNIT, 41 * UNIT), ro - part(L // UNIT * UNIT, L),
                  ro + part(UNIT, 2 * UNIT), ro - part(50 * UNIT, 50 * UNIT + 32)]
    for o in wrong:
        with pytest.raises(AssertionError):
            check(c, torch.from_numpy(o).bfloat16(), lse, within=within)
    with pytest.raises(AssertionError):    # one unit of l
        check(c, torch.from_numpy(ro).bfloat16(),
              lse + torch.from_numpy(np.log1p(-p[:, :UNIT].sum(1))).float(), within=within)


# ------------------------------------------------------------------- on GPU
@pytest.mark.gpu
@pytest.mark.parametrize("make", [lambda c: c, one_sign])
@pytest.mark.parametrize("case", ATTN + MIXED + TURNS)
def test_calls_of_every_kind(case, make):
    c = make(attn_case(*case))
    check(c, *gpu_attn(c))
    assert fa.fa_check_device_status(DEV) == OK


LONG = [  # H, Hkv, T, d, page, lens, q_lens
    # One token: parts of every block, and of a few.
    (8, 1, 1, 128, 256, [100000], None),
    (4, 4, 1, 64, 64, [60000, 3000, 129], None),
    (3, 1, 5, 64, 128, [40000, 7], [5, 2]),
    (32, 1, 1, 128, 256, [50000], None),
    # Units taken in turn: odd and even shares.
    (8, 1, 14, 128, 256, [40000], None), (16, 2, 14, 64, 256, [30000, 14], None),
    (24, 3, 14, 128, 256, [9000, 129, 12000], None), (1, 1, 64, 64, 256, [30000], None),
    (2, 2, 100, 128, 128, [20000, 100], [100, 3]),
    # Items of 256 rows, some with a last one of a few.
    (8, 1, 40, 128, 256, [20000], None), (2, 1, 300, 64, 64, [15000, 300], None),
    (8, 2, 33, 64, 256, [9000, 5000], [33, 1]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("make", [one_sign, marked])
@pytest.mark.parametrize("H,Hkv,T,d,page,lens,q_lens", LONG)
def test_long_histories_miss_nothing(H, Hkv, T, d, page, lens, q_lens, make):
    c = make(attn_case(len(lens), H, Hkv, T, d, page, lens, q_lens, -1))
    c["q"] = c["q"] * 0.25
    o, lse = gpu_attn(c)
    assert fa.fa_check_device_status(DEV) == OK
    # Some of the new tokens (the float64 form takes a second for 64 rows).
    few = sorted({0, 1, T // 2, T - 1} & set(range(T)))
    n = np.full(len(lens), T) if q_lens is None else c["q_lens"]
    for t in few:
        one = dict(c, q=c["q"][:, :, t:t + 1].contiguous(), lens=c["lens"] - n + t + 1,
                   q_lens=(n > t).astype(np.int32))
        check(one, o[:, :, t:t + 1], lse[:, :, t:t + 1])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_the_last_pages_of_a_cache_past_32_bits(d):
    """Each kernel on pages beyond 2^32 bytes: the bits that it has on a cache of
    these pages alone."""
    H, Hkv, page, lens = 16, 2, 64, [900, 333]
    small = one_sign(attn_case(2, H, Hkv, 1, d, page, lens, None, -1))
    n = small["cache"].shape[0]
    pages = 2 ** 32 // small["cache"][0].size + n + 1
    big = torch.zeros((pages, *small["cache"].shape[1:]), dtype=torch.uint8, device=DEV)
    big[-n:] = torch.from_numpy(small["cache"]).to(DEV)
    assert big[:-n].numel() > 2 ** 32
    for T, q_lens in ((1, None), (4, None), (9, None), (40, None), (40, [40, 1])):
        c = attn_case(2, H, Hkv, T, d, page, lens, q_lens, -1)
        c.update(cache=small["cache"], table=small["table"])
        want = gpu_attn(c)
        check(c, *want)
        table = np.where(c["table"] < 0, -1, c["table"] + pages - n).astype(np.int32)
        dev = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
        out = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)
        fa.fa_cache8_attn(c["q"].to(DEV), big, dev(table), dev(c["lens"]), c["scale"],
                          None if q_lens is None else dev(c["q_lens"]), out=out[0], lse=out[1])
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert fa.fa_check_device_status(DEV) == OK


MANY_HEADS = [  # B, H, Hkv, T, d, page, lens, q_lens, window
    # Items that end within a token; a token of several items.
    (2, 300, 1, 1, 128, 16, [700, 33], None, -1), (2, 300, 1, 2, 64, 64, [300, 5], [2, 1], -1),
    (3, 100, 2, 2, 128, 32, [260, 1, 90], None, 40), (1, 130, 1, 1, 64, 16, [400], None, -1),
    (2, 520, 4, 3, 128, 128, [129, 400], [1, 3], -1), (2, 40, 1, 1, 128, 16, [300, 2], None, -1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", MANY_HEADS)
def test_many_heads_of_one_key_value_head(case):
    c = one_sign(attn_case(*case))
    check(c, *gpu_attn(c))
    assert fa.fa_check_device_status(DEV) == OK


@pytest.mark.gpu
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("T,d", [(1, 128), (4, 64), (9, 128), (40, 64), (40, 128)])
def test_a_query_that_is_no_number_spoils_its_row_only(T, d, value):
    c = attn_case(2, 8, 1, T, d, 32, [700, 150], None, -1)
    good = c["q"].clone()
    c["q"][0, 3, T // 2, 5] = value
    o, lse = gpu_attn(c)
    assert torch.isnan(lse[0, 3, T // 2]) and torch.isnan(o[0, 3, T // 2]).all()
    c["q"] = good
    want = gpu_attn(c)
    o[0, 3, T // 2], lse[0, 3, T // 2] = want[0][0, 3, T // 2], want[1][0, 3, T // 2]
    check(c, o, lse)


@pytest.mark.gpu
def test_more_requests_than_threads():
    """A thread sums up several requests; most have no work."""
    B = 1500
    rng = np.random.default_rng(4)
    lens = np.where(rng.random(B) < 0.7, 0, rng.integers(1, 40, B)).tolist()
    for T, q in ((1, None), (6, 1), (9, None), (33, 2)):
        q_lens = None if q is None else [min(q, n) if i % 50 else min(T, n) for i, n in enumerate(lens)]
        c = one_sign(attn_case(B, 8, 1, T, 64, 16, lens, q_lens, -1))
        check(c, *gpu_attn(c))
