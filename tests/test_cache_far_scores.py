"""Cache attention with scores far from zero, up to the 2^22 that the header
names.

Exact cases: queries of one nonzero dim, so that a score is one product and the
keys' scores are equal or apart, and one power of two for all values.  A score's
distance from the row's reference then is rounded once and the scale's two
roundings move all scores of a row alike, so the weights are those of float64.  O
is off by P's rounding to f16 and its own to bf16, 2^-11 and 2^-8, by some 2^-18
for sums, and by what P cannot hold, 2^-32 a key times the largest value that
it may have; the LSE by the roundings of the scale, the score and its own, 2^-21.

Of any queries: a score of fp32 may be off by more than one there, so that only
this holds: O lies among the values that its row sees (the same roundings off),
and the LSE within (d + 8) 2^-24 scale sum |q||k| of its value.
"""
import numpy as np
import pytest
import torch

import test_cache4
import test_cache8
from oracle import cache8, serve
from test_cache8 import DEV, OK, f64
from tiled_attention_bwd_gb300 import fa

# Rows before the cache's start, several units, a window.
CASES = [(1, -1), (5, -1), (14, 60), (33, -1), (140, -1)]
LENS = [300, 77, 3]
LIMIT = 2.0 ** 22


def case8(T, d, window):
    c = test_cache8.attn_case(3, 8, 2, T, d, 32, LENS, None, window, exps=(-3, -3))
    # Several powers of two for keys.
    rng = np.random.default_rng(T)
    ke = rng.integers(-3, 3, c["cache"][..., 0].shape)
    c["cache"][..., 32 * d] = ke.astype(np.int8).view(np.uint8)
    return c, test_cache8.gpu_attn


def case4(T, d, window):
    return test_cache4.attn_case(3, 8, 2, T, d, 32, LENS, None, window), full4


def full4(c):
    out = torch.full(c["q"].shape, 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(c["q"].shape[:3], 7.0, device=DEV)
    return test_cache4.gpu_attn(c, out, lse)


def values_of(c):
    if "gk" in c:
        return serve.cache_values(c["cache"], c["gk"], c["gv"])
    return cache8.values(c["cache"])


def exact(c):
    """O, LSE, sum of weight times |value|; least and largest value that a row
    sees; sum of |q||k|'s bound."""
    q = f64(c["q"])
    B, H, T, d = q.shape
    k, v = values_of(c)
    Hkv, page = k.shape[1], k.shape[2]
    o, mag, lo, hi = (np.zeros(q.shape) for _ in range(4))
    lse = np.full((B, H, T), -np.inf)
    for b, L in enumerate(c["lens"]):
        at = np.arange(L)
        pg = c["table"][b][at // page]
        for h in range(H):
            K, V = (x[pg, h // (H // Hkv), at % page] for x in (k, v))
            for t in range(T):
                i = L - T + t
                see = (at <= i) & ((at >= i - c["window"]) | (c["window"] < 0))
                if not see.any():
                    continue
                s = K[see] @ q[b, h, t] * c["scale"]
                m = s.max()
                p = np.exp(s - m)
                o[b, h, t], mag[b, h, t] = (p @ x / p.sum() for x in (V[see], np.abs(V[see])))
                lse[b, h, t] = m + np.log(p.sum())
                lo[b, h, t], hi[b, h, t] = V[see].min(0), V[see].max(0)
    es = (d + 8) * 2.0 ** -24 * c["scale"] * (np.abs(q) * np.abs(k).max((0, 1, 2))).sum(-1)
    return o, lse, mag, lo, hi, es


def scaled(c, to):
    """Queries times a power of two, the largest score within [to / 2, to]."""
    k, _ = values_of(c)
    q, k = f64(c["q"]), k.reshape(-1, k.shape[1], c["q"].shape[-1])
    H, Hkv = q.shape[1], k.shape[1]
    most = max(np.abs(q[:, h] @ k[:, h // (H // Hkv)].T).max() for h in range(H)) * c["scale"]
    return dict(c, q=(c["q"].float() * 2.0 ** np.floor(np.log2(to / most))).bfloat16())


@pytest.mark.gpu
@pytest.mark.parametrize("make", [case8, case4])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,window", CASES)
def test_scores_of_one_product(T, window, d, make):
    c, call = make(T, d, window)
    for to in (2.0 ** 12, 2.0 ** 19, LIMIT):
        for sign in (1, -1):
            q = torch.zeros_like(c["q"])
            q[:, :, torch.arange(T), (torch.arange(T) * 5 + 1) % d] = sign
            one = scaled(dict(c, q=q), to)
            o, lse = (f64(x) for x in call(one))
            ro, rl, mag, lo, hi, _ = exact(one)
            some = np.isfinite(rl)
            assert (o[~some] == 0).all() and np.isneginf(lse[~some]).all()
            assert (np.abs(lse[some] - rl[some]) <= 2.0 ** -21 * (1 + np.abs(rl[some]))).all(), to
            room = (2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2.0 ** -18) * mag
                    + max(LENS) * 2.0 ** -32 * np.maximum(np.abs(lo), np.abs(hi)))
            assert (np.abs(o - ro) <= room).all(), (to, sign)
    assert fa.fa_check_device_status(DEV) == OK


@pytest.mark.gpu
@pytest.mark.parametrize("make", [case8, case4])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,window", CASES)
def test_outputs_stay_among_the_values(T, window, d, make):
    c, call = make(T, d, window)
    for to in (2.0 ** 14, 2.0 ** 20, LIMIT):
        one = scaled(c, to)
        o, lse = (f64(x) for x in call(one))
        _, rl, _, lo, hi, es = exact(one)
        some = np.isfinite(rl)
        assert (o[~some] == 0).all() and np.isneginf(lse[~some]).all()
        room = es + 2.0 ** -20 * (1 + np.abs(np.where(some, rl, 0)))
        assert (np.abs(lse[some] - rl[some]) <= room[some]).all(), to
        room = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18) * np.maximum(np.abs(lo), np.abs(hi))
        assert (o >= lo - room).all() and (o <= hi + room).all(), to
    assert fa.fa_check_device_status(DEV) == OK


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 14, 140])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_beside_values_of_any_size_count_in_lse(T, d):
    """Exponents of the values at both ends: the smaller products are 2^-120 of
    the larger ones times the ratio of their weights, here above 2^-14."""
    c = test_cache8.attn_case(2, 4, 2, T, d, 16, [300 + T, 40 + T], None, -1, exps=(-3, -3))
    rng = np.random.default_rng(T)
    ve = rng.choice([-60, 60], c["cache"][..., 0].shape)
    c["cache"][..., 32 * d + 1] = ve.astype(np.int8).view(np.uint8)
    c = scaled(c, 4.0)                     # weights within 2^(8 / ln 2), 2^12
    o, lse = test_cache8.gpu_attn(c)
    _, rl, _, _, _, es = exact(c)
    assert (np.abs(f64(lse) - rl) <= es + 2.0 ** -20 * (1 + 60 + np.abs(rl))).all()
    assert np.isfinite(f64(o)).all()
