"""Calls whose outputs lie on one another or on an input (CPU only: the C ABI
refuses them before it touches a GPU).

Where a call is in order, it gets past the checks to the device, which is not
there: FA_ERR_CUDA then, and on a machine with a GPU these tests do not run.
"""
import ctypes
import itertools

import pytest
import torch

from tiled_attention_bwd_gb300 import build as fa_build
from tiled_attention_bwd_gb300 import fa

INVALID, CUDA = 1, 3

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="made-up addresses: no GPU may read them")


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fa.load_library()


def p(x):
    return ctypes.c_void_p(x) if x else None


M = 1 << 20


def bwd(lib, B=2, N=3, H=3, Hkv=1, d=128, rot=128, rows=8, sb=None, sn=None,
        dsb=None, dsn=None, norm=True, **at):
    """fa_qk_norm_rope_bwd on addresses a megabyte apart, but for `at`."""
    width = (H + 2 * Hkv) * d
    sn = width if sn is None else sn
    sb = N * sn if sb is None else sb
    dsn = width if dsn is None else dsn
    dsb = N * dsn if dsb is None else dsb
    names = ["qkv", "rope", "pos", "qw", "kw", "dq", "dk", "dv", "dqkv", "dqw",
             "dkw", "ws"]
    a = {n: (16 + i) * 16 * M for i, n in enumerate(names)}
    if not norm:
        a.update(qw=0, kw=0, dqw=0, dkw=0, ws=0)
    a.update(at)
    return lib.fa_qk_norm_rope_bwd(
        p(a["qkv"]), sb, sn, p(a["rope"]), rows, rot, p(a["pos"]), p(a["qw"]),
        p(a["kw"]), 0, 1e-6, 0, p(a["dq"]), p(a["dk"]), p(a["dv"]), p(a["dqkv"]),
        dsb, dsn, p(a["dqw"]), p(a["dkw"]), p(a["ws"]), 1 << 24, B, N, H, Hkv,
        d, None)


W = 5 * 128                                # elements of a token above


def tokens_meet(B, N, sb, sn, width):
    at = sorted(b * sb + n * sn for b in range(B) for n in range(N))
    return any(y - x < width for x, y in zip(at, at[1:]))


@pytest.mark.parametrize("B,N", [(1, 1), (1, 4), (4, 1), (2, 2), (2, 3), (3, 2), (3, 5), (6, 4)])
def test_tokens_of_the_gradient_that_lie_on_one_another(lib, B, N):
    """Every pair of strides of up to a few rows, in half rows, both signs."""
    seen = set()
    steps = [s * W // 2 for s in range(-9, 10)] + [W - 8, W + 8, 1 << 40]
    for sb, sn in itertools.product(steps, steps):
        meet = tokens_meet(B, N, sb, sn, W)
        got = bwd(lib, B, N, dsb=sb, dsn=sn, dqkv=1 << 50, norm=False)
        assert got == (INVALID if meet else CUDA), (sb, sn)
        seen.add(meet)
    assert B * N == 1 or seen == {False, True}


def test_tokens_on_one_another_in_many_entries(lib):
    """Strides of the same size: entry 0's second token is entry 1's first."""
    for B, N in ((2, 2), (64, 4096), (4096, 64)):
        assert bwd(lib, B, N, dsb=W, dsn=W, dqkv=1 << 50, norm=False) == INVALID
        assert bwd(lib, B, N, dsb=W, dsn=-W, dqkv=1 << 50, norm=False) == INVALID
        assert bwd(lib, B, N, dsb=N * W, dsn=W, dqkv=1 << 50, norm=False) == CUDA
        assert bwd(lib, B, N, dsb=W, dsn=B * W, dqkv=1 << 50, norm=False) == CUDA
        # (The last token on the next entry's first.)
        assert bwd(lib, B, N, dsb=(N - 1) * W, dsn=W, dqkv=1 << 50, norm=False) == INVALID


def fwd(lib, B=2, N=3, H=3, Hkv=1, d=128, rot=128, rows=8, sb=None, sn=None,
        bf16=0, **at):
    """fa_qk_norm_rope on addresses 16 megabytes apart, but for `at`."""
    width = (H + 2 * Hkv) * d
    sn = width if sn is None else sn
    sb = N * sn if sb is None else sb
    a = {n: (16 + i) * 16 * M for i, n in enumerate(
        ["qkv", "rope", "pos", "qw", "kw", "q", "k", "v"])}
    a.update(at)
    return lib.fa_qk_norm_rope(
        p(a["qkv"]), sb, sn, p(a["rope"]), rows, rot, p(a["pos"]), p(a["qw"]),
        p(a["kw"]), bf16, 1e-6, 0, p(a["q"]), p(a["k"]), p(a["v"]), B, N, H,
        Hkv, d, None)


def touching(x, size, y, other):
    """Addresses of a piece of `size` bytes at x: just before, over either
    end of, within and just behind a piece of `other` bytes at y."""
    return [(y - size, False), (y - size + 16, True), (y, True),
            (y + other - 16, True), (y + other, False)]


def test_forward_outputs_on_one_another_and_on_inputs(lib):
    at = {n: (16 + i) * 16 * M for i, n in enumerate(
        ["qkv", "rope", "pos", "qw", "kw", "q", "k", "v"])}
    # B, N, H, Hkv, d = 2, 3, 3, 1, 128: six tokens
    size = {"qkv": 6 * 2 * W, "rope": 8 * 128 * 4, "pos": 32, "qw": 512,
            "kw": 512, "q": 6 * 768, "k": 6 * 256, "v": 6 * 256}
    assert fwd(lib) == CUDA
    for out in ("q", "k", "v"):
        for other in at:
            if other == out:
                continue
            for x, bad in touching(at[out], size[out], at[other], size[other]):
                assert fwd(lib, **{out: x}) == (INVALID if bad else CUDA), (out, other, x)
    # Weights of two bytes, no positions, no weights: nothing to meet.
    assert fwd(lib, bf16=1, q=at["qw"] + 256) == CUDA
    assert fwd(lib, bf16=1, q=at["qw"] + 240) == INVALID
    assert fwd(lib, pos=0, q=at["pos"]) == CUDA
    assert fwd(lib, qw=0, kw=0, q=at["qw"]) == CUDA
    assert fwd(lib, H=0, q=0) == CUDA
    assert fwd(lib, H=0, k=at["v"]) == INVALID


def test_forward_outputs_between_the_tokens_of_a_wide_input(lib):
    """qkv as columns of wider rows: outputs may lie in the gaps."""
    qkv, row = 1 << 30, 2 * 4096           # bytes from token to token
    ok = dict(qkv=qkv, sn=4096, sb=3 * 4096)
    tok, q, k = 2 * W, 6 * 768, 6 * 256    # bytes of a token, of q, of k or v
    # One request of one token: nothing behind it.
    assert fwd(lib, B=1, N=1, qkv=qkv, q=qkv + tok, sn=0, sb=0) == CUDA
    assert fwd(lib, q=qkv + tok, k=qkv + row + tok, v=qkv + row + tok + k, **ok) == CUDA
    assert fwd(lib, q=qkv + tok - 16, **ok) == INVALID
    assert fwd(lib, q=qkv + row - q, **ok) == CUDA
    assert fwd(lib, q=qkv + row - q + 16, **ok) == INVALID
    assert fwd(lib, k=qkv + 5 * row + tok, **ok) == CUDA
    assert fwd(lib, k=qkv + 5 * row + tok - 16, **ok) == INVALID
    assert fwd(lib, k=qkv - k, **ok) == CUDA
    assert fwd(lib, k=qkv - k + 16, **ok) == INVALID
    # Negative strides: tokens lie before the address.
    back = dict(qkv=qkv, sn=-4096, sb=-3 * 4096)
    assert fwd(lib, k=qkv - row - k, **back) == CUDA
    assert fwd(lib, k=qkv - row - k + 16, **back) == INVALID
    assert fwd(lib, k=qkv - 5 * row + tok, **back) == CUDA
    assert fwd(lib, k=qkv - 5 * row, **back) == INVALID


NAMES = ["qkv", "rope", "pos", "qw", "kw", "dq", "dk", "dv", "dqkv", "dqw",
         "dkw", "ws"]


def test_backward_outputs_on_one_another_and_on_inputs(lib):
    at = {n: (16 + i) * 16 * M for i, n in enumerate(NAMES)}
    size = {"qkv": 6 * 2 * W, "rope": 8 * 128 * 4, "pos": 32, "qw": 512,
            "kw": 512, "dq": 6 * 768, "dk": 6 * 256, "dv": 6 * 256,
            "dqkv": 6 * 2 * W, "dqw": 512, "dkw": 512,
            "ws": lib.fa_qk_norm_rope_bwd_workspace_size(128)}
    assert bwd(lib) == CUDA
    for out in ("dqkv", "dqw", "dkw", "ws"):
        for other in at:
            if other == out:
                continue
            for x, bad in touching(at[out], size[out], at[other], size[other]):
                if (out, other) == ("dqkv", "qkv") and x == at[other]:
                    bad = False            # the one input that it may be
                assert bwd(lib, **{out: x}) == (INVALID if bad else CUDA), (out, other, x)
    # Without weights there is no sum, and qkv is not read.
    assert bwd(lib, norm=False, dqkv=at["qkv"] + 16) == CUDA
    assert bwd(lib, norm=False, dqkv=at["dq"]) == INVALID
    assert bwd(lib, norm=False, dqkv=at["rope"]) == INVALID
    # Without tokens only the weights' gradients are written.
    empty = dict(N=0, qkv=0, dq=0, dk=0, dv=0, dqkv=0, rope=0, pos=0)
    assert bwd(lib, **empty) == CUDA
    assert bwd(lib, dqw=at["dkw"], **empty) == INVALID
    assert bwd(lib, dkw=at["qw"] + 256, **empty) == INVALID


def test_gradient_in_place_and_beside_its_input(lib):
    """dqkv as qkv itself needs qkv's strides; as other columns of the same
    wide rows it shares nothing."""
    x, row, tok = 1 << 30, 2 * 4096, 2 * W
    wide = dict(qkv=x, sn=4096, sb=3 * 4096, dsn=4096, dsb=3 * 4096)
    assert bwd(lib, dqkv=x, **wide) == CUDA
    assert bwd(lib, dqkv=x + tok, **wide) == CUDA
    assert bwd(lib, dqkv=x + row - tok, **wide) == CUDA
    for off in (16, tok - 16, row, row - tok + 16, 3 * row, 5 * row, -row + 16,
                -5 * row, 2 * row + tok - 16):
        assert bwd(lib, dqkv=x + off, **wide) == INVALID, off
    for off in (6 * row, 5 * row + tok, -5 * row - tok, -6 * row, 3 * row + tok):
        assert bwd(lib, dqkv=x + off, **wide) == CUDA, off
    # Other strides on the same memory: refused, whatever lies between.
    other = dict(wide, dsn=4096 + 8)
    assert bwd(lib, dqkv=x, **other) == INVALID
    assert bwd(lib, dqkv=x + 6 * row, **other) == CUDA
    # A single entry or token has no stride.
    assert bwd(lib, B=1, qkv=x, dqkv=x, sb=0, dsb=77 * 8) == CUDA
    assert bwd(lib, B=1, N=1, qkv=x, dqkv=x, sn=0, dsn=8) == CUDA
    # Entries within the tokens' gaps of one another.
    loose = dict(B=2, N=3, qkv=x, sb=1024, sn=4096, dsb=1024, dsn=4096)
    assert bwd(lib, dqkv=x, **loose) == CUDA
    assert bwd(lib, dqkv=x + 2 * 2048, **loose) == CUDA
    assert bwd(lib, dqkv=x + 2048, **loose) == INVALID


ATTN = ["q", "cache", "table", "lens", "ql", "o", "lse", "ws"]


def attn(lib, B=2, H=4, Hkv=2, T=3, d=64, blocks=2, pages=3, page=32, **at):
    """fa_cache4_attn on addresses 64 megabytes apart, but for `at`."""
    a = {n: (16 + i) * 64 * M for i, n in enumerate(ATTN)}
    a.update(at)
    return lib.fa_cache4_attn(
        p(a["q"]), p(a["cache"]), p(a["table"]), p(a["lens"]), p(a["ql"]),
        p(a["o"]), p(a["lse"]), p(a["ws"]), 1 << 40, B, H, Hkv, T, d, blocks,
        pages, page, -1, 0.1, 1.0, 1.0, None)


def test_attention_outputs_on_one_another_and_on_inputs(lib):
    at = {n: (16 + i) * 64 * M for i, n in enumerate(ATTN)}
    B, H, T, d = 4, 4, 3, 64
    rows = B * H * T
    size = {"q": rows * d * 2, "cache": 3 * 2 * 2 * 18 * d, "table": B * 2 * 4,
            "lens": B * 4, "ql": B * 4, "o": rows * d * 2, "lse": rows * 4,
            "ws": lib.fa_cache4_attn_workspace_size(B, H, 2, T, d)}
    assert attn(lib, B) == CUDA
    for out in ("o", "lse", "ws"):
        for other in at:
            if other == out:
                continue
            if out == "ws":                # 256-byte aligned
                up = lambda n: -(-n // 256) * 256  # noqa: E731
                places = [(at[other] - up(size["ws"]), False),
                          (at[other] + 256 - up(size["ws"]), True),
                          (at[other], True), (at[other] + up(size[other]), False)]
            else:
                places = touching(at[out], size[out], at[other], size[other])
            for x, bad in places:
                assert attn(lib, B, **{out: x}) == (INVALID if bad else CUDA), (out, other, x)
    assert attn(lib, B, ql=0, lse=at["ql"]) == CUDA
    assert attn(lib, B, ql=at["lens"]) == CUDA  # inputs may share what they read


APPEND = ["k", "v", "cache", "slots", "ko", "vo"]


def append(lib, B=2, Hkv=2, N=4, d=64, pages=3, page=32, **at):
    """fa_cache4_append on addresses 16 megabytes apart, but for `at`."""
    a = {n: (16 + i) * 16 * M for i, n in enumerate(APPEND)}
    a.update(at)
    return lib.fa_cache4_append(
        p(a["k"]), p(a["v"]), p(a["cache"]), p(a["slots"]), 1.0, 1.0,
        p(a["ko"]), p(a["vo"]), B, Hkv, N, d, pages, page, None)


def test_append_outputs_on_one_another_and_on_inputs(lib):
    at = {n: (16 + i) * 16 * M for i, n in enumerate(APPEND)}
    rows = 2 * 2 * 4 * 64 * 2
    size = {"k": rows, "v": rows, "cache": 3 * 2 * 2 * 18 * 64, "slots": 32,
            "ko": rows, "vo": rows}
    assert append(lib) == CUDA
    for out in ("cache", "ko", "vo"):
        for other in at:
            if other == out:
                continue
            for x, bad in touching(at[out], size[out], at[other], size[other]):
                if out[1:] == "o" and other == out[0] and x == at[other]:
                    bad = False            # values may replace their own input
                assert append(lib, **{out: x}) == (INVALID if bad else CUDA), (out, other, x)
    both = dict(ko=at["k"], vo=at["v"])
    assert append(lib, **both) == CUDA
    for other in ("k", "v"):
        assert append(lib, cache=at[other], **both) == INVALID
        assert append(lib, cache=at[other], ko=0, vo=0) == INVALID
        assert append(lib, slots=at[other], **both) == INVALID
    assert append(lib, cache=at["slots"], ko=0, vo=0) == INVALID
    assert append(lib, v=at["k"], ko=0, vo=0) == CUDA
    assert append(lib, v=at["k"], **dict(both, vo=at["vo"])) == INVALID
