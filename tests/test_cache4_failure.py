"""The cache attention's stopping path, without a GPU fault: the test hook
makes the first warp of every block treat its first wait for copies as
expired.  Its block goes on to the end without it, the copies in flight land
before the block leaves, and the next call is right.
"""
import pytest
import torch

from test_cache4 import attn_case, check_attn, gpu_attn
from tiled_attention_bwd_gb300 import (fa_check_device_status,
                                       fa_debug_expire_at,
                                       fa_last_failure_site)

FA_ERR_DEVICE_TIMEOUT = 4
SITE = 0x511

CASES = [  # B, H, Hkv, T, d, page, lens, q_lens, window
    (1, 8, 1, 1, 128, 64, [20], None, -1),             # one block, one unit
    (5, 16, 2, 1, 128, 32, [1500, 3, 0, 700, 4000], None, -1),
    (400, 2, 2, 2, 128, 16, [(9 * i) % 50 for i in range(400)], None, 20),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_an_expired_wait_stops_the_call_and_no_other(case):
    dev = torch.device("cuda:0")
    c = attn_case(*case)
    assert fa_check_device_status(dev) == 0
    try:
        fa_debug_expire_at(SITE)
        gpu_attn(c)
        assert fa_check_device_status(dev) == FA_ERR_DEVICE_TIMEOUT
        assert fa_last_failure_site() == SITE
    finally:
        fa_debug_expire_at(0)
    assert fa_check_device_status(dev) == 0    # reported once, then cleared
    check_attn(c, *gpu_attn(c))
    assert fa_check_device_status(dev) == 0


@pytest.mark.gpu
def test_calls_without_the_hook_ignore_it():
    dev = torch.device("cuda:0")
    for case in ((2, 8, 1, 1, 64, 32, [300, 77], None, -1),
                 (2, 16, 1, 1, 128, 32, [300, 77], None, -1)):
        c = attn_case(*case)
        try:
            fa_debug_expire_at(SITE)
            check_attn(c, *gpu_attn(c))
            assert fa_check_device_status(dev) == 0
        finally:
            fa_debug_expire_at(0)
