"""The cache attention where requests of one call have very different numbers
of new tokens, against the float64 oracle (tolerances: test_cache4.py)."""
import numpy as np
import pytest
import torch

from test_cache4 import attn_case, check_attn, gpu_attn
from tiled_attention_bwd_gb300 import fa_check_device_status

CASES = [  # B, H, Hkv, T, d, page, lens, q_lens, window
    # A chunk beside single tokens, and requests without any.
    (6, 8, 1, 96, 128, 32, [300, 77, 1, 500, 0, 129], [96, 1, 1, 0, 0, 1], -1),
    (5, 6, 2, 64, 64, 16, [64, 200, 33, 90, 7], [64, 1, 2, 63, 1], -1),
    (4, 12, 4, 50, 128, 64, [400, 60, 50, 51], [3, 50, 50, 1], 37),
    # More new tokens than cached ones: rows before the start.
    (3, 8, 2, 40, 128, 16, [7, 40, 0], [40, 40, 5], -1),
    (2, 16, 1, 33, 64, 32, [20, 333], [33, 2], 5),
    # Heads that are no power of two; items that end inside a token.
    (2, 7, 1, 19, 128, 32, [150, 19], [19, 7], -1),
    (2, 10, 2, 21, 64, 16, [21, 210], None, 64),
    # A window of one key, and of more than all.
    (2, 4, 1, 30, 128, 16, [100, 30], [30, 11], 0),
    (2, 4, 1, 30, 64, 16, [100, 30], [30, 11], 1000),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_mixed_calls_match_the_oracle(case):
    c = attn_case(*case)
    out = torch.full(c["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda:0")
    lse = torch.full(c["q"].shape[:3], 7.0, device="cuda:0")
    gpu_attn(c, out, lse)
    assert fa_check_device_status("cuda:0") == 0
    check_attn(c, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES[:3])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38])
def test_rows_without_a_token_change_nothing(case, value):
    """Query rows past a request's new tokens may hold anything."""
    c = attn_case(*case)
    c["q"][:] = c["q"].clamp(-8, 8)
    want = [torch.full(c["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda:0"),
            torch.full(c["q"].shape[:3], 7.0, device="cuda:0")]
    got = [t.clone() for t in want]
    gpu_attn(c, *want)
    for b, n in enumerate(c["q_lens"]):
        c["q"][b, :, n:] = value
    gpu_attn(c, *got)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_a_chunk_equals_its_tokens_one_by_one():
    """Each of a chunk's rows against a call for that token alone, its history
    cut there: the same keys in other tiles (tolerances of either, twice)."""
    c = attn_case(1, 6, 2, 45, 128, 16, [160], None, -1, seed=21)
    o, lse = gpu_attn(c)
    for t in (0, 1, 20, 44):
        one = dict(c, q=c["q"][:, :, t:t + 1].contiguous(),
                   lens=np.array([160 - 44 + t], np.int32))
        po, pl = gpu_attn(one)
        v = float(torch.maximum(o[:, :, t].abs().max(), po.abs().max()))
        assert (po[:, :, 0].float() - o[:, :, t].float()).abs().max() <= 2.0 ** -7 * v + 2.0 ** -9
        assert (pl[:, :, 0] - lse[:, :, t]).abs().max() <= 1e-4
