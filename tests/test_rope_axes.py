"""Norm of query and key heads with a rotation whose positions have several
axes, and backward: the oracle against differences, the kernels against the
oracle, refusals.

Tolerances.  The kernels compute in fp32 and round once to bf16, an error of
at most half a step, 2^-8 of the value.  Before that, a value is a product of
a norm (a sum of d squares: at most d + 4 roundings of 2^-24) and two
rotation terms: within (d + 16) 2^-24 of the row's largest value.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import serve
from tiled_attention_bwd_gb300 import build as fa_build
from tiled_attention_bwd_gb300 import fa

BF16 = 2.0 ** -8
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5
DEV = "cuda:0"


def f64(t):
    return t.detach().to("cpu").double().numpy()


def sections(half, sizes):
    out = [i for i, n in enumerate(sizes) for _ in range(n)]
    assert len(out) == half
    return out


# ------------------------------------------------------------------- on CPU
@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_gradient_against_differences(interleaved):
    B, N, H, Hkv, d, rot = 1, 2, 2, 1, 64, 32
    rng = np.random.default_rng(5)
    x = rng.standard_normal((B, N, H + 2 * Hkv, d))
    w = [1 + 0.2 * rng.standard_normal(d) for _ in range(2)]
    pos = np.array([[[3, 11]], [[0, 7]], [[15, 2]]])
    table, at = serve.axes_table(serve.rope_table(16, rot), pos, [i % 3 for i in range(16)])
    dz = [rng.standard_normal((B, h, N, d)) for h in (H, Hkv, Hkv)]

    def loss(x, qw, kw):
        out = serve.norm_rope(x, H, Hkv, table, at, qw, kw, 1e-3, interleaved)
        return sum((a * b).sum() for a, b in zip(out, dz))

    g = serve.norm_rope_bwd(x, H, Hkv, table, at, *w, 1e-3, interleaved, *dz)
    h = 1e-6
    for _ in range(12):
        u = rng.standard_normal(x.shape)
        num = (loss(x + h * u, *w) - loss(x - h * u, *w)) / (2 * h)
        assert abs(num - (g[0] * u).sum()) <= 1e-6 * (1 + abs(num))
    for k in range(2):
        u = rng.standard_normal(d)
        up, dn = list(w), list(w)
        up[k], dn[k] = w[k] + h * u, w[k] - h * u
        num = (loss(x, *up) - loss(x, *dn)) / (2 * h)
        assert abs(num - (g[1 + k] * u).sum()) <= 1e-6 * (1 + abs(num))


def test_oracle_with_equal_axes_is_the_plain_one():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((2, 3, 4, 64))
    pos = rng.integers(0, 20, (2, 3))
    table = serve.rope_table(20, 64)
    t2, at = serve.axes_table(table, np.stack([pos] * 4), [i % 4 for i in range(32)])
    for a, b in zip(serve.norm_rope(x, 2, 1, t2, at, None, None, 0, False),
                    serve.norm_rope(x, 2, 1, table, pos, None, None, 0, False)):
        assert np.array_equal(a, b)


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fa.load_library()


def p(x):
    return ctypes.c_void_p(x) if x else None


def _axes(axes):
    return None if axes is None else ctypes.cast(ctypes.create_string_buffer(bytes(axes), 64),
                                                 ctypes.c_void_p)


def _fwd(lib, qkv=16, rope=16, pos=16, n=3, axes=(0, 1, 2, 0), qw=16, kw=16, q=16,
         k=16, v=16, B=1, N=1, H=2, Hkv=1, d=128, rot=128, rows=8):
    return lib.fa_qk_norm_rope_axes(p(qkv), 512, 512, p(rope), rows, rot, p(pos), n,
                                    _axes(axes), p(qw), p(kw), 0, 1e-6, 0, p(q), p(k),
                                    p(v), B, N, H, Hkv, d, None)


def _bwd(lib, ptr=16, pos=16, n=3, axes=(0, 1, 2, 0), ws=16, B=1, N=1, d=128, rot=128, dw=16):
    return lib.fa_qk_norm_rope_axes_bwd(p(16), 512, 512, p(16), 8, rot, p(pos), n, _axes(axes),
                                        p(16), p(16), 0, 1e-6, 0, p(ptr), p(ptr), p(ptr), p(ptr),
                                        512, 512, p(dw), p(dw), p(ws), 1 << 30, B, N, 2, 1, d,
                                        None)


REFUSED = [
    (INVALID, dict(n=0)), (INVALID, dict(n=-1)), (UNSUPPORTED, dict(n=5)),
    (INVALID, dict(axes=None)), (INVALID, dict(axes=(0, 3))), (INVALID, dict(n=2)),
    (INVALID, dict(axes=(255,))), (INVALID, dict(axes=(0,) * 63 + (3,))),
    (INVALID, dict(pos=0)), (INVALID, dict(pos=2)), (INVALID, dict(rot=24)),
    (UNSUPPORTED, dict(d=96)),
]


@pytest.mark.parametrize("want,bad", REFUSED + [
    (INVALID, dict(qw=0)), (INVALID, dict(q=0)), (INVALID, dict(rows=0)),
    # The third axis's positions lie on an output.
    (INVALID, dict(pos=4096, q=4096 + 1024, B=1, N=100, k=1 << 20, v=1 << 21)),
])
def test_forward_refusals(lib, want, bad):
    assert _fwd(lib, **bad) == want


@pytest.mark.parametrize("want,bad", REFUSED + [(WORKSPACE, dict(ws=0)), (INVALID, dict(dw=0))])
def test_backward_refusals(lib, want, bad):
    assert _bwd(lib, **bad) == want


def test_empty_calls(lib):
    assert _fwd(lib, N=0, qkv=0, q=0, k=0, v=0, pos=0) == 0
    assert _fwd(lib, H=0, Hkv=0, qkv=0, pos=0) == 0
    assert _fwd(lib, N=0, n=9) == UNSUPPORTED and _fwd(lib, N=0, axes=None) == INVALID


def test_binding_refusals():
    z = torch.zeros
    with pytest.raises(ValueError):        # not on a GPU
        fa.fa_qk_norm_rope_axes(z((1, 1, 4, 64), dtype=torch.bfloat16), 2, 1, z((4, 64)),
                                z((3, 1, 1), dtype=torch.int32), [0] * 32)
    with pytest.raises(ValueError):        # an axis that is no byte
        fa.fa_qk_norm_rope_axes(z((1, 1, 4, 64), dtype=torch.bfloat16), 2, 1, z((4, 64)),
                                z((3, 1, 1), dtype=torch.int32), [256] * 32)


def test_axes_of_any_sequence():
    """Their elements count, not the memory or the size that they stand for."""
    want = bytes([0, 2, 1, 0])
    for axes in ([0, 2, 1, 0], (0, 2, 1, 0), bytearray(want), np.array([0, 2, 1, 0]),
                 np.array([0, 2, 1, 0], dtype=np.int32), torch.tensor([0, 2, 1, 0]),
                 (x for x in (0, 2, 1, 0))):
        assert fa._axis_bytes(axes) == want
    assert fa._axis_bytes(np.array([3])) == b"\3"
    assert fa._axis_bytes(torch.tensor([3])) == b"\3"
    for axes in (4, True, np.int64(4), np.array(4), torch.tensor(4), "0210", [0.0], None):
        with pytest.raises(TypeError):
            fa._axis_bytes(axes)
    for axes in ([-1], [256]):
        with pytest.raises(ValueError):
            fa._axis_bytes(axes)


# ------------------------------------------------------------------- on GPU
CASES = [  # B, N, H, Hkv, d, rot, interleaved, weights, axes, strided
    (1, 1, 1, 1, 128, 128, False, "f32", sections(64, (16, 24, 24)), False),
    (2, 3, 5, 1, 128, 128, False, "bf16", [i % 3 for i in range(64)], False),
    (1, 7, 4, 4, 64, 64, True, "f32", sections(32, (8, 12, 12)), True),
    (3, 33, 9, 3, 64, 32, False, "f32", sections(16, (3, 5, 8)), False),
    (2, 65, 6, 2, 128, 96, True, "bf16", [i * 7 % 4 for i in range(48)], True),
    (2, 40, 8, 2, 128, 16, False, None, sections(8, (7, 1)), False),
    (1, 129, 3, 3, 128, 48, False, "f32", sections(24, (24,)), True),
    (1, 50, 7, 7, 64, 48, True, None, [3] * 12 + [1] * 12, False),
    (5, 301, 12, 4, 128, 128, False, "f32", sections(64, (16, 24, 24)), False),
    (2, 200, 8, 0, 64, 64, False, "f32", [i % 2 for i in range(32)], False),
    (2, 200, 0, 5, 128, 64, False, "f32", [i % 3 for i in range(32)], False),
]


def setup(case, seed=0):
    B, N, H, Hkv, d, rot, inter, weights, axes, strided = case
    rows = 300
    g = torch.Generator().manual_seed(1000 + seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    A = max(axes) + 1
    x = {"qkv": r(B, N, H + 2 * Hkv, d).bfloat16(), "qw": 1 + 0.2 * r(d), "kw": 1 + 0.2 * r(d),
         "rope": torch.from_numpy(serve.rope_table(rows, rot)),
         "pos": torch.randint(0, rows, (A, B, N), generator=g, dtype=torch.int32),
         "dq": r(B, H, N, d).bfloat16(), "dk": r(B, Hkv, N, d).bfloat16(),
         "dv": r(B, Hkv, N, d).bfloat16()}
    if B * N > 2:                          # clamped to the table's ends
        x["pos"][0, 0, 0], x["pos"][-1, -1, -1] = -5, 1 << 30
    if weights == "bf16":
        x["qw"], x["kw"] = x["qw"].bfloat16(), x["kw"].bfloat16()
    if weights is None:
        x["qw"] = x["kw"] = None
    table, at = serve.axes_table(x["rope"].numpy(), x["pos"].numpy(), axes)
    qw, kw = (None, None) if weights is None else (f64(x["qw"]), f64(x["kw"]))
    ref = (f64(x["qkv"]), H, Hkv, table, at, qw, kw, 1e-6, inter)
    gpu = {n: None if t is None else t.to(DEV) for n, t in x.items()}
    if strided:                            # a slice of wider, longer rows
        wide = torch.full((B, N + 2, H + 2 * Hkv + 3, d), float("nan"), dtype=torch.bfloat16,
                          device=DEV)
        view = wide[:, 1:N + 1, 2:2 + H + 2 * Hkv]
        view.copy_(gpu["qkv"])
        gpu["qkv"] = view
    args = (gpu["qkv"], H, Hkv, gpu["rope"])
    rest = dict(q_weight=gpu["qw"], k_weight=gpu["kw"], interleaved=inter)
    return x, gpu, args, rest, ref


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_forward_matches_oracle(case):
    x, gpu, args, rest, ref = setup(case)
    d = case[4]
    got = fa.fa_qk_norm_rope_axes(*args, gpu["pos"], case[8], **rest)
    want = serve.norm_rope(*ref)
    for a, b in zip(got[:2], want[:2]):
        a = f64(a)
        if b.size == 0:
            continue
        room = BF16 * np.abs(b) + (d + 16) * 2.0 ** -24 * np.abs(b).max(-1, keepdims=True)
        # Both members of a rotated pair are of the pair's size.
        room = room + 4 * 2.0 ** -24 * np.linalg.norm(b, axis=-1, keepdims=True)
        assert (np.abs(a - b) <= room).all(), np.max(np.abs(a - b) - room)
    assert np.array_equal(f64(got[2]), want[2])


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_backward_matches_oracle(case):
    B, N, H, Hkv, d = case[:5]
    x, gpu, args, rest, ref = setup(case)
    got = fa.fa_qk_norm_rope_axes_bwd(*args, gpu["dq"], gpu["dk"], gpu["dv"], gpu["pos"],
                                      bytes(case[8]), **rest)
    grads = [f64(x[n]) for n in ("dq", "dk", "dv")]
    dx, dqw, dkw = serve.norm_rope_bwd(*ref, *grads)
    # dx = r (gw - xh mean(gw xh)): each term's fp32 error is within
    # (d + 16) 2^-24 of r (max |gw| + max |xh| mean |gw xh|).
    size = np.abs(np.concatenate([g.transpose(0, 2, 1, 3) for g in grads], 2)).max(
        -1, keepdims=True) * 2
    if rest["q_weight"] is not None:
        r = 1 / np.sqrt((ref[0] ** 2).mean(-1, keepdims=True) + 1e-6)
        xh = np.abs(ref[0] * r).max(-1, keepdims=True)
        wm = max(np.abs(ref[5]).max(), np.abs(ref[6]).max())
        size = np.maximum(size, r * size * wm * (1 + xh ** 2))
    room = BF16 * np.abs(dx) + (d + 16) * 2.0 ** -24 * size
    err = np.abs(f64(got[0]) - dx)
    assert (err <= room).all(), np.max(err - room)
    if rest["q_weight"] is None:
        assert got[1] is None and got[2] is None
        return
    # A sum of n terms, in any order, is within n 2^-24 of the sum of their
    # sizes, each term within (d + 16) 2^-24 of its own.
    for g, want, heads, x0, dz in ((got[1], dqw, H, 0, grads[0]), (got[2], dkw, Hkv, H, grads[1])):
        part = ref[0][:, :, x0:x0 + heads]
        r = 1 / np.sqrt((part ** 2).mean(-1, keepdims=True) + 1e-6)
        top = np.abs(dz).transpose(0, 2, 1, 3).max(-1, keepdims=True, initial=0) * 2
        sizes = (np.abs(part) * r * top).sum((0, 1, 2))
        assert g.dtype == torch.float32
        assert (np.abs(f64(g) - want) <= (B * N * heads + d + 16) * 2.0 ** -24 * sizes).all()


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("axes", [[0] * 64, [i % 3 for i in range(64)],
                                  sections(64, (16, 24, 24))])
def test_equal_axes_are_the_plain_call(inter, axes):
    """Bit for bit, whichever way the angles come."""
    x, gpu, args, rest, ref = setup((3, 70, 6, 2, 128, 128, inter, "f32", axes, False))
    pos = gpu["pos"][0].contiguous()
    many = pos[None].repeat(max(axes) + 1, 1, 1)
    grads = gpu["dq"], gpu["dk"], gpu["dv"]
    for a, b in zip(fa.fa_qk_norm_rope_axes(*args, many, axes, **rest),
                    fa.fa_qk_norm_rope(*args, pos, **rest)):
        assert torch.equal(a, b)
    for a, b in zip(fa.fa_qk_norm_rope_axes_bwd(*args, *grads, many, axes, **rest),
                    fa.fa_qk_norm_rope_bwd(*args, *grads, pos, **rest)):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_backward_in_place():
    case = CASES[8]
    x, gpu, args, rest, ref = setup(case)
    grads = gpu["dq"], gpu["dk"], gpu["dv"]
    first = fa.fa_qk_norm_rope_axes_bwd(*args, *grads, gpu["pos"], case[8], **rest)
    over = fa.fa_qk_norm_rope_axes_bwd(*args, *grads, gpu["pos"], case[8], dqkv=gpu["qkv"], **rest)
    assert over[0].data_ptr() == gpu["qkv"].data_ptr()
    for a, b in zip(first, over):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_no_tokens_give_zero_weight_gradients():
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    w = torch.ones(128, device=DEV)
    _, a, b = fa.fa_qk_norm_rope_axes_bwd(
        z(2, 0, 6, 128), 4, 1, torch.zeros((4, 128), device=DEV), z(2, 4, 0, 128), z(2, 1, 0, 128),
        z(2, 1, 0, 128), torch.zeros((3, 2, 0), dtype=torch.int32, device=DEV), [0, 1] * 32, w, w)
    assert not a.any() and not b.any()


@pytest.mark.gpu
def test_binding_checks_shapes():
    x, gpu, args, rest, ref = setup(CASES[1])
    for pos, axes in ((gpu["pos"][0], CASES[1][8]), (gpu["pos"], CASES[1][8][:-1]),
                      (gpu["pos"][:, :1], CASES[1][8]), (gpu["pos"].long(), CASES[1][8])):
        with pytest.raises(ValueError):
            fa.fa_qk_norm_rope_axes(*args, pos, axes, **rest)
    with pytest.raises(fa.FAError):        # an axis that positions do not have
        fa.fa_qk_norm_rope_axes(*args, gpu["pos"][:2].contiguous(), CASES[1][8], **rest)
