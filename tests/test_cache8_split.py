"""Cache attention calls whose requests go to different kernels by their number
of rows: the division of work (CPU only, the kernels' own header), and mixed
calls against the float64 oracle (tolerances: test_cache8.py)."""
import ctypes
import random
import subprocess

import numpy as np
import pytest
import torch

import test_cache4_work as base
from test_cache8 import DEV, OK, attn_case, check_attn, gpu_attn
from tiled_attention_bwd_gb300 import build as fa_build
from tiled_attention_bwd_gb300 import fa

# The same harness with limits to the live rows.
OLD = "  const c4::Call c = {B, Hkv, T, window, heads, rows, (heads * T - 1) / rows + 1, max_len,\n" \
      "                      FastDiv::of(heads)};\n"
NEW = "  c4::Call c = {B, Hkv, T, window, heads, rows, (heads * T - 1) / rows + 1, max_len,\n" \
      "                FastDiv::of(heads)};\n  c.least_rows = g_least, c.most_rows = g_most;\n" \
      "  if (g_most < heads * T) c.row_blocks = (g_most - 1) / rows + 1;\n"


@pytest.fixture(scope="module")
def work(tmp_path_factory):
    assert base.HARNESS.count(OLD) == 1
    text = base.HARNESS.replace(OLD, NEW).replace(
        "using namespace fa;\n", "using namespace fa;\nstatic int g_least = 0, g_most = 1 << 30;\n"
        "extern \"C\" void limits(int least, int most) { g_least = least, g_most = most; }\n")
    d = tmp_path_factory.mktemp("split")
    (d / "work.cpp").write_text(text)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-I", fa_build.CSRC,
                    str(d / "work.cpp"), "-o", str(d / "work.so")], check=True)
    return ctypes.CDLL(str(d / "work.so"))


@pytest.mark.parametrize("seed", range(30))
def test_every_request_goes_to_one_kernel(work, seed):
    rng = random.Random(seed)
    for _ in range(20):
        B, heads = rng.choice([1, 2, 7, 40]), rng.choice([1, 3, 8, 16, 64])
        T, most = rng.choice([2, 5, 40, 150]), 32
        if B > 7 and T > 5:
            T = 5
        lens = [rng.randint(-1, rng.choice([40, 700])) for _ in range(B)]
        q_lens = [rng.choice([0, 1, T, rng.randint(-1, T + 1)]) for _ in range(B)]
        window, Hkv = rng.choice([-1, 0, 100]), rng.choice([1, 2])
        live = [min(max(q, 0), T) * heads for q in q_lens]
        for least, top, rows in ((0, most, rng.choice([8, 16, 32])), (most + 1, 1 << 30, 256)):
            work.limits(least, top)
            mine = [q if least <= n <= top else 0 for q, n in zip(q_lens, live)]
            segs, _ = base.deal(work, Hkv, T, window, heads, rows, lens, q_lens, 304)
            work.limits(0, 1 << 30)
            want, _ = base.deal(work, Hkv, T, window, heads, rows, lens, mine, 304)
            assert [s[2:] for s in segs] == [s[2:] for s in want]


MIXED = [  # B, H, Hkv, T, d, page, lens, q_lens, window
    # A chunk beside single tokens, and requests without any.
    (6, 8, 1, 96, 128, 32, [300, 77, 1, 500, 0, 129], [96, 1, 1, 0, 0, 1], -1),
    (5, 6, 2, 64, 64, 16, [64, 200, 33, 90, 7], [64, 1, 2, 63, 1], -1),
    (4, 12, 4, 50, 128, 64, [400, 60, 50, 51], [3, 50, 50, 1], 37),
    # More new tokens than cached ones: rows before the start.
    (3, 8, 2, 40, 128, 16, [7, 40, 0], [40, 40, 5], -1),
    (2, 16, 1, 33, 64, 32, [20, 333], [33, 2], 5),
    # On either side of the limit between the kernels, and of a tile's rows.
    (4, 4, 1, 9, 128, 32, [150, 19, 90, 200], [8, 9, 7, 0], -1),
    (5, 8, 1, 33, 64, 16, [200, 210, 220, 230, 33], [16, 17, 32, 33, 4], -1),
    # Heads that are no power of two; tokens across tiles; one head of many.
    (2, 7, 1, 40, 128, 32, [150, 40], [40, 37], -1),
    (2, 33, 1, 1, 128, 16, [300, 1], None, -1),
    (2, 64, 1, 5, 64, 64, [300, 90], [5, 4], 33),
    # A window of one key, and of more than all.
    (2, 4, 1, 30, 128, 16, [100, 30], [30, 11], 0),
    (2, 4, 1, 30, 64, 16, [100, 30], [30, 11], 1000),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", MIXED)
def test_mixed_calls_match_the_oracle(case):
    c = attn_case(*case)
    check_attn(c, *gpu_attn(c))
    assert fa.fa_check_device_status(DEV) == OK


@pytest.mark.gpu
@pytest.mark.parametrize("case", MIXED[:3])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38])
def test_rows_without_a_token_change_nothing(case, value):
    """Query rows past a request's new tokens may hold anything."""
    c = attn_case(*case)
    want = gpu_attn(c)
    for b, n in enumerate(c["q_lens"]):
        c["q"][b, :, n:] = value
    for a, b in zip(gpu_attn(c), want):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_a_chunk_equals_its_tokens_one_by_one():
    """Each of a chunk's rows against a call for that token alone, by the other
    kernel (tolerances of either, twice)."""
    c = attn_case(1, 6, 2, 45, 128, 16, [160], None, -1, seed=21)
    o, lse = gpu_attn(c)
    for t in (0, 1, 20, 44):
        one = dict(c, q=c["q"][:, :, t:t + 1].contiguous(),
                   lens=np.array([160 - 44 + t], np.int32))
        po, pl = gpu_attn(one)
        v = float(torch.maximum(o[:, :, t].abs().max(), po.abs().max()))
        assert (po[:, :, 0].float() - o[:, :, t].float()).abs().max() <= 2.0 ** -7 * v + 2.0 ** -9
        assert (pl[:, :, 0] - lse[:, :, t]).abs().max() <= 1e-4


@pytest.mark.gpu
@pytest.mark.parametrize("Hkv,T,lens", [(1, 64, [30000]), (2, 40, [20000, 5])])
def test_long_histories_are_joined_from_many_parts(Hkv, T, lens):
    """Few rows over a long history: every block has a part of each item."""
    c = attn_case(len(lens), Hkv, Hkv, T, 64, 256, lens, None, -1)
    c["q"] = c["q"] * 0.25
    o, lse = gpu_attn(c)
    o2, lse2 = gpu_attn(c)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    some = [0, T // 2, T - 1]              # of the rows: the oracle is slow
    for t in some:
        n = T - 1 - t
        one = dict(c, q=c["q"][:, :, t:t + 1].contiguous(), lens=c["lens"] - n)
        check_attn(one, o[:, :, t:t + 1], lse[:, :, t:t + 1])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 300])
def test_scores_that_grow_along_the_history(T):
    """Each key's scores above all before it: the maximum moves every unit."""
    c = attn_case(1, 8, 1, T, 128, 32, [700 + T], None, -1)
    cache = c["cache"]
    cache[..., :16 * 128] = 0x30           # keys of a half
    cache[..., 32 * 128] = 0
    order = {int(p): i for i, p in enumerate(c["table"][0]) if p >= 0}
    for p, i in order.items():             # a power of two a page
        cache[p, :, :, 32 * 128] = np.int8(i // 3 - 4).view(np.uint8)
    c["q"] = c["q"].abs()
    check_attn(c, *gpu_attn(c))


@pytest.mark.gpu
def test_calls_that_run_together():
    """Calls of both kernels on several streams, workspaces of their own."""
    cases = [attn_case(3, 8, 2, t, 128, 64, [9000 - 97 * s, 3000, 500 + s], q, -1, seed=s)
             for s, (t, q) in enumerate([(1, None), (60, [60, 1, 33]), (200, None)])]
    args = [(c["q"].to(DEV), torch.from_numpy(c["cache"]).to(DEV),
             torch.from_numpy(c["table"]).to(DEV), torch.from_numpy(c["lens"]).to(DEV), c["scale"],
             None if c["q_lens"] is None else torch.from_numpy(c["q_lens"]).to(DEV)) for c in cases]

    def outs(a):
        return torch.zeros_like(a[0]), torch.zeros(a[0].shape[:3], device=DEV)

    want = [fa.fa_cache8_attn(*a, out=o, lse=lse) for a in args for o, lse in [outs(a)]]
    streams = [torch.cuda.Stream() for _ in args]
    got = [[outs(a) for _ in range(8)] for a in args]
    torch.cuda.synchronize()
    for i in range(8):
        for s, a, g in zip(streams, args, got):
            with torch.cuda.stream(s):
                fa.fa_cache8_attn(*a, out=g[i][0], lse=g[i][1])
    torch.cuda.synchronize()
    assert fa.fa_check_device_status(DEV) == OK
    for w, g in zip(want, got):
        for o, lse in g:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])
