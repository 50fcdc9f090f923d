"""The binding of the norm with rotation and of the 4-bit cache: the arguments
that reach the C ABI, and what the binding refuses (CPU only: the compiled
binding is connected to entry points that record their arguments, and then
takes CPU tensors)."""
import ctypes

import numpy as np
import pytest
import torch

from tiled_attention_bwd_gb300 import build as fa_build
from tiled_attention_bwd_gb300 import fa

I32, BF16, F32 = torch.int32, torch.bfloat16, torch.float32


def z(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


class Recorder:
    """Stands in for libfa.so: every entry point notes its arguments."""

    def __init__(self, lib):
        self.calls, self.streams, self.status = [], [], 0
        sizes = {"fa_qk_norm_rope_bwd_workspace_size": 1024,
                 "fa_cache4_attn_workspace_size": 512}
        for name in fa._NATIVE:
            real = getattr(lib, name)
            kind = ctypes.CFUNCTYPE(real.restype, *real.argtypes)
            if name in sizes:
                f = kind(lambda *a, n=sizes[name]: n)
            else:
                f = kind(lambda *a, n=name: self.note(n, a))
            setattr(self, name, f)

    def note(self, name, args):
        self.calls.append((name, args[:-1]))
        self.streams.append(args[-1])
        return self.status


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fa.load_library()


@pytest.fixture
def recorder(lib):
    native = fa._native()
    r = Recorder(lib)
    fa._connect(native, r, host=True)
    yield r
    fa._connect(native, lib)
    assert not any(r.streams)              # CPU tensors have none


@pytest.fixture
def rec(recorder):
    return recorder.calls


def same(got, want):
    """Equal arguments, floats as the C side's fp32 rounds them."""
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert a == (float(np.float32(b)) if isinstance(b, float) else b)


def p(t):
    return t.data_ptr()


def test_rope_calls(rec):
    B, N, H, Hkv, d = 2, 3, 4, 2, 64
    qkv, rope = z(B, N, 8, d), z(10, 32, dtype=F32)
    pos, w = z(B, N, dtype=I32), z(d, dtype=F32)
    q, k, v = fa.fa_qk_norm_rope(qkv, H, Hkv, rope, pos, w, w, eps=0.5,
                                 interleaved=True)
    assert rec[-1][0] == "fa_qk_norm_rope"
    same(rec[-1][1], (
        p(qkv), N * 8 * d, 8 * d, p(rope), 10, 32, p(pos), p(w), p(w), 0, 0.5,
        1, p(q), p(k), p(v), B, N, H, Hkv, d))
    assert q.shape == (B, H, N, d) and v.shape == (B, Hkv, N, d)
    dqkv, dqw, dkw = fa.fa_qk_norm_rope_bwd(qkv, H, Hkv, rope, q, k, v, None,
                                            w.bfloat16(), w.bfloat16())
    name, a = rec[-1]
    assert name == "fa_qk_norm_rope_bwd" and a[6] is None and a[9] == 1
    same(a[10:], (1e-6, 0, p(q), p(k), p(v), p(dqkv), N * 8 * d, 8 * d,
                  p(dqw), p(dkw), a[20], 1024, B, N, H, Hkv, d))
    assert fa.fa_qk_norm_rope_bwd(qkv, H, Hkv, rope, q, k, v)[1:] == (None, None)


def test_rope_strides_and_refusals(rec):
    wide = z(2, 7, 11, 64)
    rope = z(10, 32, dtype=F32)
    part = wide[:, 2:5, 1:9]
    fa.fa_qk_norm_rope(part, 4, 2, rope)
    assert rec[-1][1][:3] == (p(part), 7 * 11 * 64, 11 * 64)
    n = len(rec)
    w, q = z(64, dtype=F32), z(2, 4, 3, 64)
    k = z(2, 2, 3, 64)
    for bad in (
            lambda: fa.fa_qk_norm_rope(wide[..., ::2], 5, 3, rope),
            lambda: fa.fa_qk_norm_rope(wide[:, :, ::2], 2, 2, rope),
            lambda: fa.fa_qk_norm_rope(part, 4, 3, rope),
            lambda: fa.fa_qk_norm_rope(part, 10, -1, rope),
            lambda: fa.fa_qk_norm_rope(part.float(), 4, 2, rope),
            lambda: fa.fa_qk_norm_rope(part, 4, 2, rope.double()),
            lambda: fa.fa_qk_norm_rope(part, 4, 2, rope[:, ::2]),
            lambda: fa.fa_qk_norm_rope(part, 4, 2, rope, z(2, 4, dtype=I32)),
            lambda: fa.fa_qk_norm_rope(part, 4, 2, rope, z(2, 3, dtype=F32)),
            lambda: fa.fa_qk_norm_rope(part, 4, 2, rope, None, w),
            lambda: fa.fa_qk_norm_rope(part, 4, 2, rope, None, w, w.bfloat16()),
            lambda: fa.fa_qk_norm_rope(part, 4, 2, rope, None, w[:32], w[:32]),
            lambda: fa.fa_qk_norm_rope(part, 4, 2, rope, q=q.float()),
            lambda: fa.fa_qk_norm_rope(part, 4, 2, rope, q=q.transpose(1, 2)),
            lambda: fa.fa_qk_norm_rope_bwd(part, 4, 2, rope, k, k, k),
            lambda: fa.fa_qk_norm_rope_bwd(part, 4, 2, rope, q, k, k, dqkv=wide)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fa.fa_qk_norm_rope_bwd(part, 4, 2, rope, q, None, k),
                lambda: fa.fa_qk_norm_rope_bwd(part, 4, 2, rope, q, k, k, None,
                                               w, w, workspace=1024)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(ValueError):        # a workspace on another device
        fa.fa_qk_norm_rope_bwd(part, 4, 2, rope, q, k, k, None, w, w,
                               workspace=torch.empty(1 << 20, device="meta"))
    assert len(rec) == n


def test_cache_calls(rec):
    R, M, P, T = 3, 5, 9, 2
    new, lens, table = z(R, dtype=I32), z(R, dtype=I32), z(R, M, dtype=I32)
    free, count = z(P, dtype=I32), z(1, dtype=I32)
    s, pos, g = fa.fa_cache4_plan(new, lens, table, free, count, 32, T)
    assert rec[-1] == ("fa_cache4_plan", (p(new), p(lens), p(table), p(free),
                                          p(count), p(s), p(pos), p(g), R, M,
                                          P, 32, T))
    cache = z(P, 4, 2, 18 * 64, dtype=torch.uint8)
    k, v = z(R, 4, T, 64), z(R, 4, T, 64)
    slots = z(R, T, dtype=I32)
    fa.fa_cache4_append(k, v, cache, slots, 2.0, 0.5)
    assert rec[-1] == ("fa_cache4_append", (p(k), p(v), p(cache), p(slots),
                                            2.0, 0.5, None, None, R, 4, T, 64,
                                            P, 32))
    fa.fa_cache4_append(k, v, cache, slots, k_out=k, v_out=v)
    assert rec[-1][1][6:8] == (p(k), p(v))
    q = z(R, 8, T, 64)
    o, lse = fa.fa_cache4_attn(q, cache, table, lens, 0.25, new, 7, 2.0, 0.5)
    a = rec[-1][1]
    same(a, (p(q), p(cache), p(table), p(lens), p(new), p(o), p(lse), a[7],
             512, R, 8, 4, T, 64, M, P, 32, 7, 0.25, 2.0, 0.5))
    assert lse.shape == (R, 8, T) and lse.dtype == F32


def test_cache_refusals(rec):
    new, table = z(3, dtype=I32), z(3, 5, dtype=I32)
    free, one = z(9, dtype=I32), z(1, dtype=I32)
    cache = z(9, 4, 2, 18 * 64, dtype=torch.uint8)
    k, slots, q = z(3, 4, 2, 64), z(3, 2, dtype=I32), z(3, 8, 2, 64)
    for bad in (
            lambda: fa.fa_cache4_plan(new, one, table, free, one, 16, 1),
            lambda: fa.fa_cache4_plan(new, new, table.T, free, one, 16, 1),
            lambda: fa.fa_cache4_plan(new, new, table, free, new, 16, 1),
            lambda: fa.fa_cache4_plan(new, new, table, free[::2], one, 16, 1),
            lambda: fa.fa_cache4_plan(new.long(), new, table, free, one, 16, 1),
            lambda: fa.fa_cache4_plan(new, new, table, free, one, 16, -1),
            lambda: fa.fa_cache4_plan(new, new, table, free, one, 16, 1, slots=slots),
            lambda: fa.fa_cache4_append(k, k, cache[..., :100], slots),
            lambda: fa.fa_cache4_append(k, k, cache[:, :2], slots),
            lambda: fa.fa_cache4_append(k, k[:, :2], cache, slots),
            lambda: fa.fa_cache4_append(k.half(), k, cache, slots),
            lambda: fa.fa_cache4_append(k, k, cache, slots.T.contiguous()),
            lambda: fa.fa_cache4_append(k, k, cache, slots.long()),
            lambda: fa.fa_cache4_attn(q[..., :32], cache, table, new, 0.1),
            lambda: fa.fa_cache4_attn(q, cache, table[:2], new, 0.1),
            lambda: fa.fa_cache4_attn(q, cache, table, new[:2], 0.1),
            lambda: fa.fa_cache4_attn(q, cache, table, new, 0.1, new.long()),
            lambda: fa.fa_cache4_attn(q, cache, table, new, 0.1,
                                      workspace=torch.empty(9, device="meta")),
            lambda: fa.fa_cache4_attn(q, cache, table, new, 0.1, out=q.float())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ValueError):
        fa.fa_cache4_append(k, k, cache, slots, k_out=k)
    for bad in (lambda: fa.fa_cache4_append(k, None, cache, slots),
                lambda: fa.fa_cache4_append(k, [1.0], cache, slots),
                lambda: fa.fa_cache4_attn(q, cache, table, new, "0.1"),
                lambda: fa.fa_cache4_plan(new, None, table, free, one, 16, 1)):
        with pytest.raises(TypeError):
            bad()
    assert rec == []


def test_errors_carry_the_status(recorder):
    recorder.status = 5
    new, table = z(3, dtype=I32), z(3, 5, dtype=I32)
    cache = z(9, 4, 2, 18 * 64, dtype=torch.uint8)
    k, slots, q = z(3, 4, 2, 64), z(3, 2, dtype=I32), z(3, 8, 2, 64)
    rope, qkv = z(10, 32, dtype=F32), z(2, 3, 8, 64)
    for call in (
            lambda: fa.fa_cache4_plan(new, new, table, new, z(1, dtype=I32), 16, 1),
            lambda: fa.fa_cache4_append(k, k, cache, slots),
            lambda: fa.fa_cache4_attn(q, cache, table, new, 0.1),
            lambda: fa.fa_qk_norm_rope(qkv, 4, 2, rope),
            lambda: fa.fa_qk_norm_rope_bwd(qkv, 4, 2, rope, z(2, 4, 3, 64),
                                           z(2, 2, 3, 64), z(2, 2, 3, 64))):
        with pytest.raises(fa.FAError) as e:
            call()
        assert e.value.status == 5 and "FA_ERR_WORKSPACE" in str(e.value)


def test_values_out_of_an_int_are_refused(rec):
    new, table = z(3, dtype=I32), z(3, 5, dtype=I32)
    cache, q = z(9, 4, 2, 18 * 64, dtype=torch.uint8), z(3, 8, 2, 64)
    for bad in (
            lambda: fa.fa_cache4_plan(new, new, table, new, z(1, dtype=I32), 1 << 40, 1),
            lambda: fa.fa_cache4_plan(new, new, table, new, z(1, dtype=I32), 16, 1 << 40),
            lambda: fa.fa_cache4_attn(q, cache, table, new, 0.1, window=1 << 31)):
        with pytest.raises(ValueError):
            bad()
    assert rec == []


def test_cpu_tensors_are_refused(lib):
    new, table = z(3, dtype=I32), z(3, 5, dtype=I32)
    with pytest.raises(ValueError):
        fa.fa_cache4_plan(new, new, table, new, z(1, dtype=I32), 16, 1)
    with pytest.raises(ValueError):
        fa.fa_qk_norm_rope(z(1, 1, 3, 64), 1, 1, z(4, 64, dtype=F32))
