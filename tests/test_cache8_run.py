"""The 8-bit cache and the rotation with axes as they are used together: plan,
norm and rotation by three axes, append, attention, read; captured steps; a
training step; and the binding's arguments (CPU only)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import serve
from test_cache8 import DEV, OK, f64, i32
from test_serve_marshal import Recorder, p, same, z
from tiled_attention_bwd_gb300 import build as fa_build
from tiled_attention_bwd_gb300 import fa

I32, F32, U8 = torch.int32, torch.float32, torch.uint8


@pytest.fixture
def recorder():
    """The binding, connected to entry points that note their arguments."""
    fa_build.build()
    lib, native = fa.load_library(), fa._native()
    r = Recorder(lib)
    size = lib.fa_cache8_attn_workspace_size
    r.fa_cache8_attn_workspace_size = ctypes.CFUNCTYPE(size.restype, *size.argtypes)(lambda *a: 512)
    fa._connect(native, r, host=True)
    yield r
    fa._connect(native, lib)
    assert not any(r.streams)              # CPU tensors have none


@pytest.fixture
def rec(recorder):
    return recorder.calls


# ------------------------------------------------------------------- on CPU
def test_cache_calls(rec):
    R, M, P, T = 3, 5, 9, 2
    table, lens = z(R, M, dtype=I32), z(R, dtype=I32)
    cache = z(P, 4, 2, 32 * 64 + 16, dtype=U8)
    k, v, slots = z(R, 4, T, 64), z(R, 4, T, 64), z(R, T, dtype=I32)
    assert fa.fa_cache8_append(k, v, cache, slots) is cache
    assert rec[-1] == ("fa_cache8_append", (p(k), p(v), p(cache), p(slots), None, None, R, 4, T,
                                            64, P, 32))
    fa.fa_cache8_append(k, v, cache, slots, k, v)
    assert rec[-1][1][4:6] == (p(k), p(v))
    ko, vo = fa.fa_cache8_read(cache, table, lens, 7, lens)
    assert rec[-1] == ("fa_cache8_read", (p(cache), p(table), p(lens), p(lens), p(ko), p(vo), R, 4,
                                          7, 64, M, P, 32))
    assert ko.shape == vo.shape == (R, 4, 7, 64)
    fa.fa_cache8_read(cache, table, lens, T, k_out=k, v_out=v)
    assert rec[-1][1][3:6] == (None, p(k), p(v))
    q = z(R, 8, T, 64)
    o, lse = fa.fa_cache8_attn(q, cache, table, lens, 0.25, lens, 7, workspace=z(256, dtype=U8))
    a = rec[-1][1]
    same(a, (p(q), p(cache), p(table), p(lens), p(lens), p(o), p(lse), a[7], 256, R, 8, 4, T, 64,
             M, P, 32, 7, 0.25))


def test_axes_calls(rec):
    B, N, H, Hkv, d = 2, 3, 4, 2, 64
    qkv, rope, w = z(B, N, 8, d), z(10, 32, dtype=F32), z(d, dtype=F32)
    pos, axes = z(3, B, N, dtype=I32), bytes([0, 1, 2, 1] * 4)
    q, k, v = fa.fa_qk_norm_rope_axes(qkv, H, Hkv, rope, pos, axes, w, w, interleaved=True)
    assert rec[-1][0] == "fa_qk_norm_rope_axes"
    a = rec[-1][1]
    same(a, (p(qkv), N * 8 * d, 8 * d, p(rope), 10, 32, p(pos), 3, a[8], p(w), p(w), 0, 1e-6, 1,
             p(q), p(k), p(v), B, N, H, Hkv, d))
    out = fa.fa_qk_norm_rope_axes_bwd(qkv, H, Hkv, rope, q, k, v, pos, list(axes))
    assert rec[-1][0] == "fa_qk_norm_rope_axes_bwd" and rec[-1][1][7] == 3
    assert out[0].shape == qkv.shape and out[1:] == (None, None)


def test_refusals(rec):
    table, lens = z(3, 5, dtype=I32), z(3, dtype=I32)
    cache, four = z(9, 4, 2, 2064, dtype=U8), z(9, 4, 2, 18 * 64, dtype=U8)
    k, slots, q = z(3, 4, 2, 64), z(3, 2, dtype=I32), z(3, 8, 2, 64)
    qkv, rope, pos = z(2, 3, 8, 64), z(10, 32, dtype=F32), z(3, 2, 3, dtype=I32)
    for bad in (
            lambda: fa.fa_cache8_append(k, k, four, slots),
            lambda: fa.fa_cache4_append(k, k, cache, slots),
            lambda: fa.fa_cache8_append(k, k, cache[..., :8], slots),
            lambda: fa.fa_cache8_append(k, k, cache[:, :2], slots),
            lambda: fa.fa_cache8_append(k, k[:, :2], cache, slots),
            lambda: fa.fa_cache8_append(k, k, cache, slots.long()),
            lambda: fa.fa_cache8_append(k, k, cache, slots, k_out=k),
            lambda: fa.fa_cache8_read(four, table, lens, 2),
            lambda: fa.fa_cache8_read(cache, table, lens[:2], 2),
            lambda: fa.fa_cache8_read(cache, table, lens, -1),
            lambda: fa.fa_cache8_read(cache, table, lens, 1 << 40),
            lambda: fa.fa_cache8_read(cache, table, lens, 2, lens.long()),
            lambda: fa.fa_cache8_read(cache, table, lens, 3, k_out=k, v_out=k),
            lambda: fa.fa_cache8_attn(q, four, table, lens, 0.1),
            lambda: fa.fa_cache8_attn(q, cache, table[:2], lens, 0.1),
            lambda: fa.fa_cache8_attn(q, cache, table, lens, 0.1, lens.long()),
            lambda: fa.fa_cache8_attn(q, cache, table, lens, 0.1, window=1 << 31),
            lambda: fa.fa_cache8_attn(q, cache, table, lens, 0.1, out=q.float()),
            lambda: fa.fa_qk_norm_rope_axes(qkv, 4, 2, rope, pos[0], [0] * 16),
            lambda: fa.fa_qk_norm_rope_axes(qkv, 4, 2, rope, pos, [0] * 15),
            lambda: fa.fa_qk_norm_rope_axes(qkv, 4, 2, rope, pos, [300] * 16),
            lambda: fa.fa_qk_norm_rope_axes(qkv, 4, 2, rope, pos[:, :, :2], [0] * 16),
            lambda: fa.fa_qk_norm_rope_axes(qkv, 4, 2, rope, None, [0] * 16)):
        with pytest.raises(ValueError):
            bad()
    for axes in (None, 16):
        with pytest.raises(TypeError):
            fa.fa_qk_norm_rope_axes(qkv, 4, 2, rope, pos, axes)
    assert rec == []


def test_errors_carry_the_status(recorder):
    recorder.status = 5
    table, lens, cache = z(3, 5, dtype=I32), z(3, dtype=I32), z(9, 4, 2, 2064, dtype=U8)
    k, slots, q = z(3, 4, 2, 64), z(3, 2, dtype=I32), z(3, 8, 2, 64)
    qkv, rope, pos = z(2, 3, 8, 64), z(10, 32, dtype=F32), z(3, 2, 3, dtype=I32)
    for call in (
            lambda: fa.fa_cache8_append(k, k, cache, slots),
            lambda: fa.fa_cache8_read(cache, table, lens, 4),
            lambda: fa.fa_cache8_attn(q, cache, table, lens, 0.1),
            lambda: fa.fa_qk_norm_rope_axes(qkv, 4, 2, rope, pos, [0] * 16),
            lambda: fa.fa_qk_norm_rope_axes_bwd(qkv, 4, 2, rope, z(2, 4, 3, 64), z(2, 2, 3, 64),
                                                z(2, 2, 3, 64), pos, [0] * 16)):
        with pytest.raises(fa.FAError) as e:
            call()
        assert e.value.status == 5


# ----------------------------------------------------------- a run of them all
class Serving:
    """Requests over one layer, positions with three axes."""

    def __init__(self, R, H, Hkv, d, page, pages, max_blocks, T, seed=0):
        self.H, self.Hkv, self.page, self.T = H, Hkv, page, T
        self.lens, self.table = i32([0] * R), i32([[-1] * max_blocks] * R)
        self.free, self.count = i32(list(range(pages))), i32([pages])
        self.cache = torch.full((pages, Hkv, page // 16, 32 * d + 16), 0xff, dtype=U8, device=DEV)
        self.rope = torch.from_numpy(serve.rope_table(max_blocks * page, d)).to(DEV)
        self.axes = bytes(i % 3 for i in range(d // 2))
        g = torch.Generator().manual_seed(seed)
        self.qw, self.kw = ((1 + 0.1 * torch.randn(d, generator=g)).to(DEV) for _ in range(2))
        self.scale = d ** -0.5
        self.new = i32([0] * R)
        self.qkv = torch.zeros((R, T, H + 2 * Hkv, d), dtype=torch.bfloat16, device=DEV)
        self.out = torch.zeros((R, H, T, d), dtype=torch.bfloat16, device=DEV)
        self.lse = torch.zeros((R, H, T), device=DEV)

    def step(self):
        slots, pos, granted = fa.fa_cache4_plan(self.new, self.lens, self.table, self.free,
                                                self.count, self.page, self.T)
        places = torch.stack([pos, pos // 7, pos % 7]).contiguous()
        q, k, v = fa.fa_qk_norm_rope_axes(self.qkv, self.H, self.Hkv, self.rope, places,
                                          self.axes, self.qw, self.kw)
        fa.fa_cache8_append(k, v, self.cache, slots)
        fa.fa_cache8_attn(q, self.cache, self.table, self.lens, self.scale, granted, out=self.out,
                          lse=self.lse)
        return slots, granted, q, k, v


@pytest.mark.gpu
def test_a_run_of_requests():
    """Prompts, decode steps, drafts taken back, an end and a new request.
    Every step's output equals the attention of what read returns, and that is
    within the format's rounding of the tokens so far."""
    R, H, Hkv, d, T = 3, 4, 2, 64, 50
    s = Serving(R, H, Hkv, d, 16, 24, 8, T)
    rng = np.random.default_rng(2)
    hist = [[], [], []]
    for new in [[50, 20, 0], [1, 1, 33], [1, 1, 1], [-200, 3, 1], [40, -2, 1], [5, 5, 5], [1, 2, 20]]:
        s.new.copy_(i32(new))
        s.qkv.copy_(torch.from_numpy(rng.standard_normal(s.qkv.shape)).bfloat16())
        s.out.fill_(7.0), s.lse.fill_(7.0)
        _, granted, q, k, v = s.step()
        assert fa.fa_check_device_status(DEV) == OK
        granted = granted.tolist()
        assert granted == [max(0, n) for n in new]
        rk, rv = (f64(x) for x in fa.fa_cache8_read(s.cache, s.table, s.lens, 128))
        for r in range(R):
            if new[r] < 0:
                del hist[r][max(0, len(hist[r]) + new[r]):]
            for t in range(granted[r]):
                hist[r].append((f64(k[r, :, t]), f64(v[r, :, t])))
            L = len(hist[r])
            assert s.lens[r].item() == L
            for held, which in ((rk, 0), (rv, 1)):
                for j in range(L):
                    x = hist[r][j][which]
                    # A group's largest is below 448 2^e <= 4 times this
                    # layer's largest value here: steps of 2^-17 of that.
                    assert (np.abs(held[r, :, j] - x) <= np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -12)).all()
            for h in range(H):
                for t in range(T):
                    if t >= granted[r]:
                        assert (s.out[r, h, t] == 7).all() and s.lse[r, h, t] == 7
                        continue
                    n = L - granted[r] + t + 1
                    K, V = rk[r, h // 2, :n], rv[r, h // 2, :n]
                    x = K @ f64(q[r, h, t]) * s.scale
                    w = np.exp(x - x.max())
                    o = w @ V / w.sum()
                    # f16 weights, fp32 scores, bf16 output.
                    room = 2.0 ** -8 * np.abs(o) + 2.0 ** -10 * np.abs(V).max(0)
                    assert (np.abs(f64(s.out[r, h, t]) - o) <= room).all()
                    assert abs(s.lse[r, h, t].item() - (x.max() + np.log(w.sum()))) <= 1e-4


@pytest.mark.gpu
def test_prompt_through_the_cache_equals_the_attention_forward():
    """fa_fwd_varlen on what read returns, against fa_cache8_attn over the
    cache: the same operation, twice."""
    s = Serving(2, 4, 2, 128, 32, 20, 8, 200)
    s.new.copy_(i32([200, 131]))
    s.qkv.copy_(torch.randn(s.qkv.shape, generator=torch.Generator().manual_seed(1)))
    _, granted, q, _, _ = s.step()
    k, v = (torch.zeros((2, 2, 200, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    fa.fa_cache8_read(s.cache, s.table, s.lens, 200, k_out=k, v_out=v)
    o, lse = fa.fa_fwd_varlen(q, k, v, granted, True, s.scale)
    for r, n in enumerate([200, 131]):
        # Either side is within its own rounding of P (bf16: 2^-8 of the
        # weights there) and O.
        a, b = f64(s.out[r, :, :n]), f64(o[r, :, :n])
        vmax = np.abs(f64(v[r, :, :n])).max((1, 2)).repeat(2, 0)[:, None, None]
        assert (np.abs(a - b) <= 2.0 ** -7 * np.abs(b) + (2.0 ** -8 + 2.0 ** -10) * vmax).all()
        assert np.abs(f64(s.lse[r, :, :n]) - f64(lse[r, :, :n])).max() <= 1e-4


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 40])
def test_captured_steps(T):
    """One captured step, replayed while the requests grow, equals eager ones;
    with T = 40 chunks and single tokens in one call."""
    a, b = (Serving(4, 8, 2, 128, 16, 120, 60, T) for _ in range(2))
    first = [1, 1, 0, 1] if T == 1 else [40, 1, 0, 33]
    for s in (a, b):
        s.new.copy_(i32(first))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.step()
    side.synchronize()
    b.step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side, capture_error_mode="thread_local"):
        a.step()
    for i in range(12):
        x = torch.randn(a.qkv.shape, generator=torch.Generator().manual_seed(i)).bfloat16()
        new = i32([1, min(T, 1 + i), i % 2, -1 if i % 5 == 4 else T])
        for s in (a, b):
            s.qkv.copy_(x)
            s.new.copy_(new)
        g.replay()
        b.step()
        torch.cuda.synchronize()
        for n in ("out", "lse", "lens", "table", "free", "count", "cache"):
            assert torch.equal(getattr(a, n), getattr(b, n)), (i, n)


@pytest.mark.gpu
def test_captured_training_step_on_another_stream():
    """Norm and rotation by axes, attention, its backward and theirs, captured
    once and replayed on other inputs, equal the eager calls."""
    B, N, H, Hkv, d = 2, 150, 6, 2, 64
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn((B, N, H + 2 * Hkv, d), generator=g).bfloat16().to(DEV)
    do = torch.randn((B, H, N, d), generator=g).bfloat16().to(DEV)
    rope = torch.from_numpy(serve.rope_table(300, d)).to(DEV)
    pos = torch.randint(0, 300, (3, B, N), generator=g, dtype=I32).to(DEV)
    w = torch.linspace(0.5, 1.5, d, device=DEV)
    axes = bytes([0] * 8 + [1] * 12 + [2] * 12)

    def step():
        q, k, v = fa.fa_qk_norm_rope_axes(qkv, H, Hkv, rope, pos, axes, w, w)
        o, lse = fa.fa_fwd_ext(q, k, v, True, 0.125)
        dq, dk, dv = fa.fa_bwd_ext(q, k, v, o, lse, do, True, 0.125)
        return (o,) + fa.fa_qk_norm_rope_axes_bwd(qkv, H, Hkv, rope, dq, dk, dv, pos, axes, w, w)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s, capture_error_mode="thread_local"):
        out = step()
    for _ in range(2):
        qkv.copy_(torch.randn(qkv.shape, generator=g))
        pos.copy_(torch.randint(0, 300, pos.shape, generator=g, dtype=I32))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        # (dQ's fp32 additions come in any order: the attention backward is
        # not bitwise repeatable, everything else here is.)
        assert torch.equal(out[0], want[0])
        for a, b in zip(out[1:], want[1:]):
            a, b = f64(a), f64(b)
            assert np.linalg.norm(a - b) <= 4 * 2.0 ** -8 * np.linalg.norm(b)
