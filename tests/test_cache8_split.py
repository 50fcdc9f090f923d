"""Cache attention calls whose requests go to different kernels by their number
of rows: the division of work (CPU only, the kernels' own header), and mixed
calls against the float64 oracle (tolerances: test_cache8.py)."""
import ctypes
import random
import subprocess
import tempfile
from pathlib import Path

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


# Calls whose items' units two tiles of the same rows take in turn (up to 128
# rows a request).
TURNS = [
    # One unit, two, three: the second tile has none, one, fewer than the first.
    (4, 8, 1, 16, 128, 16, [16, 129, 300, 257], None, -1),
    (4, 8, 1, 9, 64, 32, [9, 128, 256, 385], None, -1),
    # Fewer rows than the items have; lengths of the new tokens around the limits.
    (6, 7, 1, 7, 128, 64, [900, 12, 640, 7, 0, 77], [7, 6, 2, 7, 5, 1], -1),
    (5, 24, 2, 9, 64, 16, [500, 90, 9, 30, 1000], [9, 5, 8, 3, 1], -1),
    (3, 65, 1, 1, 128, 16, [130, 1, 0], None, -1),
    (2, 128, 1, 1, 64, 256, [1500, 255], [1, 1], -1),
    # More new tokens than cached ones; windows that end before a unit, within
    # one and within the item's own tokens.
    (3, 16, 2, 15, 128, 16, [7, 15, 3], [15, 15, 15], -1),
    (2, 8, 1, 16, 128, 32, [700, 300], None, 0),
    (2, 8, 1, 16, 128, 32, [700, 300], [16, 13], 3),
    (2, 12, 1, 10, 64, 16, [900, 140], None, 127),
    (3, 16, 2, 8, 128, 64, [600, 513, 8], None, 200),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", TURNS)
def test_units_taken_in_turn_match_the_oracle(case):
    c = attn_case(*case)
    check_attn(c, *gpu_attn(c))
    assert fa.fa_check_device_status(DEV) == OK


@pytest.mark.gpu
@pytest.mark.parametrize("d,Hkv,lens", [(128, 1, [40000]), (64, 2, [30000, 5]),
                                        (128, 3, [9000, 129, 12000])])
def test_turns_over_many_blocks(d, Hkv, lens):
    """A block begins and ends inside an item: odd and even shares, and joins of
    few and of many parts; the same twice, and each row as the oracle's."""
    T = 14
    c = attn_case(len(lens), 8 * Hkv, Hkv, T, d, 256, lens, None, -1)
    c["q"] = c["q"] * 0.25
    o, lse = gpu_attn(c)
    o2, lse2 = gpu_attn(c)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for t in (0, T - 1):
        one = dict(c, q=c["q"][:, :, t:t + 1].contiguous(), lens=c["lens"] - (T - 1 - t))
        check_attn(one, o[:, :, t:t + 1], lse[:, :, t:t + 1])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tok", [0, 127, 128, 300, 511, 519, 525])
def test_nan_values_of_either_tile(d, tok):
    """A NaN value reaches the rows that see its token, whichever tile took its
    unit, and no others."""
    c = attn_case(1, 8, 1, 14, d, 16, [526], None, 300)
    page = int(c["table"][0, tok // 16])
    dim = 70 % d
    at = (page, 0, 0, v_at(d, tok % 16, dim))
    c["cache"][at] = 0
    want = gpu_attn(c)
    check_attn(c, *want)
    c["cache"][at] = 0x7f
    o, lse = gpu_attn(c)
    pos = 526 - 14 + np.arange(14)
    seen = torch.from_numpy((tok <= pos) & (tok >= pos - 300)).to(DEV)
    assert torch.equal(lse, want[1])
    assert (torch.isnan(o[0, :, :, dim]) == seen).all()
    want[0][0, :, :, dim].masked_fill_(seen, 0)
    o[0, :, :, dim].masked_fill_(seen, 0)
    assert torch.equal(o, want[0])


def v_at(d, tok, dim):
    """Byte of a value in its group, from the documented axes."""
    return 16 * d + ((((dim // 64 * 2 + tok // 8) * 8 + dim % 64 // 8) * 4 + tok % 8 // 2) * 8
                     + dim % 8) * 2 + tok % 2


@pytest.mark.gpu
@pytest.mark.parametrize("site", range(0x531, 0x53f))
def test_a_stop_between_turns_reports_and_recovers(site):
    """By the test hook (no fault, no hang), at every wait."""
    c = attn_case(2, 8, 1, 12, 128, 64, [30000, 700], None, -1)
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


def test_few_rows_are_fewer_than_the_calls():
    """The first kernel leaves the second every request with all of a call's rows:
    a call without lengths runs the second alone."""
    src = (Path(fa_build.CSRC) / "fa_cache8_attn.cu").read_text()
    rows_of = src[src.index("int cache8_attn_rows("):src.index("// Measured against")]
    few = src[src.index("int cache8_narrow_rows("):src.index("cudaError_t launch_cache8_attn(")]
    wide = (Path(fa_build.CSRC) / "fa_cache8_wide.cu").read_text()
    at = wide.index("int cache8_wide_rows(int rows) {")
    code = (rows_of + wide[at:wide.index("\n", at)] + "\n" + few
            + 'int main() { for (int d = 64; d <= 128; d += 64)\n'
            '  for (int heads = 1; heads <= 300; ++heads) for (int T = 1; T <= 400; ++T)\n'
            '    if (heads * T > cache8_narrow_rows(d) && cache8_few_rows(heads * T, heads, d) >= heads * T)\n'
            '      return 1;\n  return 0; }\n')
    with tempfile.TemporaryDirectory() as tmp:
        (Path(tmp) / "few.cpp").write_text(code)
        subprocess.run(["g++", "-O1", "-std=c++17", "few.cpp", "-o", "few"], cwd=tmp, check=True)
        assert subprocess.run([str(Path(tmp) / "few")]).returncode == 0


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
