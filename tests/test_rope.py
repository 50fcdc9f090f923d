"""Norm of query and key heads with the rotation of positions, and backward:
the oracle against differences, the kernels against the oracle, refusals.

Tolerances.  The kernels compute in fp32 and round once to bf16, an error of
at most half a step, 2^-8 of the value.  Before that, a value is a product of
a norm (a sum of d squares: at most d + 4 roundings of 2^-24) and two
rotation terms: within FP32 = (d + 16) 2^-24 of the row's largest value.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import serve
from tiled_attention_bwd_gb300 import build as fa_build
from tiled_attention_bwd_gb300 import fa

BF16 = 2.0 ** -8


def f64(t):
    return t.detach().to("cpu").double().numpy()


def make(B, N, H, Hkv, d, rot, rows=300, seed=0):
    g = torch.Generator().manual_seed(1000 + seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return {"qkv": r(B, N, H + 2 * Hkv, d).bfloat16(),
            "qw": 1 + 0.2 * r(d), "kw": 1 + 0.2 * r(d),
            "rope": torch.from_numpy(serve.rope_table(rows, rot)),
            "pos": torch.randint(0, rows, (B, N), generator=g,
                                 dtype=torch.int32),
            "dq": r(B, H, N, d).bfloat16(), "dk": r(B, Hkv, N, d).bfloat16(),
            "dv": r(B, Hkv, N, d).bfloat16()}


# ------------------------------------------------------------------- on CPU
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_oracle_gradient_against_differences(interleaved, norm):
    B, N, H, Hkv, d, rot = 1, 2, 2, 1, 64, 32
    rng = np.random.default_rng(5)
    x = rng.standard_normal((B, N, H + 2 * Hkv, d))
    w = [1 + 0.2 * rng.standard_normal(d) for _ in range(2)] if norm else [None, None]
    table = serve.rope_table(16, rot)
    pos = np.array([[3, 11]])
    dz = [rng.standard_normal((B, h, N, d)) for h in (H, Hkv, Hkv)]

    def loss(x, qw, kw):
        out = serve.norm_rope(x, H, Hkv, table, pos, qw, kw, 1e-3, interleaved)
        return sum((a * b).sum() for a, b in zip(out, dz))

    g = serve.norm_rope_bwd(x, H, Hkv, table, pos, *w, 1e-3, interleaved, *dz)
    h = 1e-6
    for _ in range(12):
        u = rng.standard_normal(x.shape)
        num = (loss(x + h * u, *w) - loss(x - h * u, *w)) / (2 * h)
        assert abs(num - (g[0] * u).sum()) <= 1e-6 * (1 + abs(num))
    if norm:
        for k in range(2):
            u = rng.standard_normal(d)
            up, dn = list(w), list(w)
            up[k], dn[k] = w[k] + h * u, w[k] - h * u
            num = (loss(x, *up) - loss(x, *dn)) / (2 * h)
            assert abs(num - (g[1 + k] * u).sum()) <= 1e-6 * (1 + abs(num))


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fa.load_library()


def _fwd(lib, qkv=16, rope=16, pos=16, qw=16, kw=16, q=16, k=16, v=16, B=1,
         N=1, H=2, Hkv=1, d=128, rot=128, rows=8, bf16=0, eps=1e-6, inter=0,
         sb=512, sn=512):
    p = lambda x: ctypes.c_void_p(x) if x else None  # noqa: E731
    return lib.fa_qk_norm_rope(p(qkv), sb, sn, p(rope), rows, rot, p(pos),
                               p(qw), p(kw), bf16, eps, inter, p(q), p(k),
                               p(v), B, N, H, Hkv, d, None)


def _bwd(lib, ptr=16, qkv=16, ws=16, ws_bytes=1 << 30, dw=16, qw=16, kw=16, B=1, N=1,
         H=2, Hkv=1, d=128, rot=128, dsn=512, dsb=512):
    p = lambda x: ctypes.c_void_p(x) if x else None  # noqa: E731
    return lib.fa_qk_norm_rope_bwd(p(qkv), 512, 512, p(16), 8, rot, p(16),
                                   p(qw), p(kw), 0, 1e-6, 0, p(ptr), p(ptr),
                                   p(ptr), p(ptr), dsb, dsn, p(dw), p(dw),
                                   p(ws), ws_bytes, B, N, H, Hkv, d, None)


INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5


@pytest.mark.parametrize("want,bad", [
    (UNSUPPORTED, dict(d=96)), (INVALID, dict(d=0)), (INVALID, dict(rot=0)),
    (INVALID, dict(rot=24)), (INVALID, dict(rot=144)), (INVALID, dict(rows=0)),
    (INVALID, dict(qw=0)), (INVALID, dict(kw=0)), (INVALID, dict(eps=-1.0)),
    (INVALID, dict(eps=float("nan"))), (INVALID, dict(bf16=2)),
    (INVALID, dict(inter=2)), (INVALID, dict(qkv=0)), (INVALID, dict(qkv=8)),
    (INVALID, dict(rope=0)), (INVALID, dict(rope=8)), (INVALID, dict(pos=2)),
    (INVALID, dict(q=0)), (INVALID, dict(v=24)), (INVALID, dict(sn=12)),
    (INVALID, dict(sb=4)), (INVALID, dict(B=-1)), (INVALID, dict(H=-1)),
    (UNSUPPORTED, dict(B=1 << 20, N=1 << 20)), (UNSUPPORTED, dict(H=1 << 17)),
    (UNSUPPORTED, dict(B=1 << 15, N=1 << 15, H=8)),
])
def test_forward_refusals(lib, want, bad):
    assert _fwd(lib, **bad) == want


@pytest.mark.parametrize("want,bad", [
    (INVALID, dict(ptr=0)), (INVALID, dict(ptr=8)), (INVALID, dict(dw=0)),
    (INVALID, dict(dsn=4)), (INVALID, dict(N=2, dsn=0)),
    (INVALID, dict(N=2, dsn=504)), (INVALID, dict(N=2, dsn=-504)),
    (INVALID, dict(B=2, dsb=0)), (WORKSPACE, dict(ws=0)), (WORKSPACE, dict(ws=8)),
    (WORKSPACE, dict(ws_bytes=1000)), (UNSUPPORTED, dict(d=80)),
    (INVALID, dict(qkv=0)), (INVALID, dict(kw=0)),
])
def test_backward_refusals(lib, want, bad):
    assert _bwd(lib, **bad) == want


def test_empty_calls(lib):
    assert _fwd(lib, N=0, qkv=0, q=0, k=0, v=0) == 0
    assert _fwd(lib, H=0, Hkv=0, qkv=0, q=0, k=0, v=0) == 0
    assert _bwd(lib, B=0, ptr=0, qw=0, kw=0) == 0
    assert lib.fa_qk_norm_rope_bwd_workspace_size(96) == 0


def test_binding_refusals():
    x = make(1, 2, 2, 1, 64, 64)
    with pytest.raises(ValueError):        # not on a GPU
        fa.fa_qk_norm_rope(x["qkv"], 2, 1, x["rope"])
    with pytest.raises(TypeError):
        fa.fa_qk_norm_rope(None, 2, 1, x["rope"])


# ------------------------------------------------------------------- on GPU
CASES = [  # B, N, H, Hkv, d, rot, interleaved, weights, positions, strided
    (1, 1, 1, 1, 128, 128, False, "f32", True, False),
    (2, 3, 5, 1, 128, 128, False, "bf16", True, False),
    (1, 7, 4, 4, 64, 64, True, "f32", True, True),
    (3, 33, 9, 3, 64, 32, False, "f32", False, False),
    (2, 65, 6, 2, 128, 96, True, "bf16", True, True),
    (2, 40, 8, 2, 128, 16, False, None, True, False),
    (1, 129, 3, 3, 128, 48, False, "f32", True, True),
    (1, 50, 7, 7, 64, 48, True, None, False, False),
    (5, 301, 12, 4, 128, 128, False, "f32", True, False),
]


def setup(case, seed=0):
    B, N, H, Hkv, d, rot, inter, weights, positions, strided = case
    dev = torch.device("cuda:0")
    x = make(B, N, H, Hkv, d, rot, rows=max(300, N), seed=seed)
    if positions and B * N > 2:            # clamped to the table's ends
        x["pos"][0, 0], x["pos"][-1, -1] = -5, 1 << 30
    if weights == "bf16":
        x["qw"], x["kw"] = x["qw"].bfloat16(), x["kw"].bfloat16()
    if weights is None:
        x["qw"] = x["kw"] = None
    pos = x["pos"].numpy() if positions else np.broadcast_to(np.arange(N), (B, N))
    qw, kw = (None, None) if weights is None else (f64(x["qw"]), f64(x["kw"]))
    ref = (f64(x["qkv"]), H, Hkv, x["rope"].numpy(), pos, qw, kw, 1e-6, inter)
    gpu = {n: None if t is None else t.to(dev) for n, t in x.items()}
    if strided:                            # a slice of wider, longer rows
        wide = torch.full((B, N + 2, H + 2 * Hkv + 3, d), float("nan"),
                          dtype=torch.bfloat16, device=dev)
        view = wide[:, 1:N + 1, 2:2 + H + 2 * Hkv]
        view.copy_(gpu["qkv"])
        gpu["qkv"] = view
    args = (gpu["qkv"], H, Hkv, gpu["rope"])
    kw_ = dict(positions=gpu["pos"] if positions else None,
               q_weight=gpu["qw"], k_weight=gpu["kw"], interleaved=inter)
    return x, gpu, args, kw_, ref


def close(got, want, d):
    fp32 = (d + 16) * 2.0 ** -24
    room = BF16 * np.abs(want) + fp32 * np.abs(want).max(-1, keepdims=True)
    # Both members of a rotated pair are of the pair's size.
    room = room + 4 * 2.0 ** -24 * np.linalg.norm(want, axis=-1, keepdims=True)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= room).all(), np.max(np.abs(got - want) - room)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_forward_matches_oracle(case):
    x, gpu, args, kw, ref = setup(case)
    q, k, v = fa.fa_qk_norm_rope(*args, **kw)
    rq, rk, rv = serve.norm_rope(*ref)
    close(f64(q), rq, case[4])
    close(f64(k), rk, case[4])
    assert np.array_equal(f64(v), rv)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_backward_matches_oracle(case):
    B, N, H, Hkv, d = case[:5]
    x, gpu, args, kw, ref = setup(case)
    got = fa.fa_qk_norm_rope_bwd(*args, gpu["dq"], gpu["dk"], gpu["dv"], **kw)
    grads = [f64(x[n]) for n in ("dq", "dk", "dv")]
    dx, dqw, dkw = serve.norm_rope_bwd(*ref, *grads)
    # dx = r (gw - xh mean(gw xh)): each term's fp32 error is within
    # (d + 16) 2^-24 of r (max |gw| + max |xh| mean |gw xh|).
    xq = ref[0]
    size = np.abs(np.concatenate(
        [g.transpose(0, 2, 1, 3) for g in grads], 2)).max(-1, keepdims=True) * 2
    if kw["q_weight"] is not None:
        r = 1 / np.sqrt((xq ** 2).mean(-1, keepdims=True) + 1e-6)
        xh = np.abs(xq * r).max(-1, keepdims=True)
        wm = max(np.abs(ref[5]).max(), np.abs(ref[6]).max())
        size = np.maximum(size, r * size * wm * (1 + xh ** 2))
    room = BF16 * np.abs(dx) + (d + 16) * 2.0 ** -24 * size
    err = np.abs(f64(got[0]) - dx)
    assert (err <= room).all(), np.max(err - room)
    if kw["q_weight"] is None:
        assert got[1] is None and got[2] is None
        return
    # A sum of n terms, in any order, is within n 2^-24 of the sum of their
    # sizes, each term within (d + 16) 2^-24 of its own.
    for g, want, heads, x0, dz in ((got[1], dqw, H, 0, grads[0]), (got[2], dkw, Hkv, H, grads[1])):
        part = xq[:, :, x0:x0 + heads]
        r = 1 / np.sqrt((part ** 2).mean(-1, keepdims=True) + 1e-6)
        top = np.abs(dz).transpose(0, 2, 1, 3).max(-1, keepdims=True) * 2
        sizes = (np.abs(part) * r * top).sum((0, 1, 2))
        assert g.dtype == torch.float32
        assert (np.abs(f64(g) - want) <= (B * N * heads + d + 16) * 2.0 ** -24 * sizes).all()


@pytest.mark.gpu
def test_backward_in_place_and_repeatable():
    case = CASES[-1]
    x, gpu, args, kw, ref = setup(case)
    first = fa.fa_qk_norm_rope_bwd(*args, gpu["dq"], gpu["dk"], gpu["dv"], **kw)
    again = fa.fa_qk_norm_rope_bwd(*args, gpu["dq"], gpu["dk"], gpu["dv"], **kw)
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    over = fa.fa_qk_norm_rope_bwd(*args, gpu["dq"], gpu["dk"], gpu["dv"],
                                  dqkv=gpu["qkv"], **kw)
    assert over[0].data_ptr() == gpu["qkv"].data_ptr()
    for a, b in zip(first, over):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hkv,d", [(3, 1, 128), (5, 2, 64)])
def test_weight_gradients_without_eps(H, Hkv, d):
    """Heads that do not fill a warp, eps = 0: as with an eps far below the
    rows' squares, whose effect is below fp32's rounding."""
    x, gpu, args, kw, ref = setup((2, 9, H, Hkv, d, d, False, "f32", True, False))
    grads = gpu["dq"], gpu["dk"], gpu["dv"]
    want = fa.fa_qk_norm_rope_bwd(*args, *grads, eps=1e-30, **kw)
    for a, b in zip(fa.fa_qk_norm_rope_bwd(*args, *grads, eps=0.0, **kw), want):
        assert torch.isfinite(b).all() and torch.equal(a, b)


@pytest.mark.gpu
def test_no_tokens_give_zero_weight_gradients():
    dev = torch.device("cuda:0")
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    w = torch.ones(128, device=dev)
    _, a, b = fa.fa_qk_norm_rope_bwd(
        z(2, 0, 6, 128), 4, 1, torch.zeros((4, 128), device=dev),
        z(2, 4, 0, 128), z(2, 1, 0, 128), z(2, 1, 0, 128), None, w, w)
    assert not a.any() and not b.any()


@pytest.mark.gpu
def test_strided_output_leaves_the_rest():
    case = CASES[4]
    B, N, H, Hkv, d = case[:5]
    x, gpu, args, kw, ref = setup(case)
    want = fa.fa_qk_norm_rope_bwd(*args, gpu["dq"], gpu["dk"], gpu["dv"], **kw)
    wide = torch.full((B, N + 3, H + 2 * Hkv + 1, d), 7.0, dtype=torch.bfloat16,
                      device="cuda:0")
    view = wide[:, 2:N + 2, 1:]
    fa.fa_qk_norm_rope_bwd(*args, gpu["dq"], gpu["dk"], gpu["dv"], dqkv=view, **kw)
    assert torch.equal(view, want[0])
    assert (wide[:, :2] == 7).all() and (wide[:, N + 2:] == 7).all()
    assert (wide[:, :, 0] == 7).all()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """More than 2^31 elements: the last tokens as in a call of their own."""
    N, H, Hkv, d, tail = 150000, 96, 16, 128, 40
    dev = torch.device("cuda:0")
    assert N * (H + 2 * Hkv) * d > 1 << 31
    qkv = torch.empty((1, N, H + 2 * Hkv, d), dtype=torch.bfloat16, device=dev).normal_()
    rope = torch.from_numpy(serve.rope_table(64, d)).to(dev)
    pos = (torch.arange(N, dtype=torch.int32, device=dev) % 64)[None].contiguous()
    w = torch.linspace(0.5, 1.5, d, device=dev)
    full = fa.fa_qk_norm_rope(qkv, H, Hkv, rope, pos, w, w)
    part = fa.fa_qk_norm_rope(qkv[:, -tail:], H, Hkv, rope, pos[:, -tail:].contiguous(), w, w)
    for a, b in zip(full, part):
        assert torch.equal(a[:, :, -tail:], b)
    dqkv, dqw, dkw = fa.fa_qk_norm_rope_bwd(qkv, H, Hkv, rope, *full, pos, w, w)
    last = fa.fa_qk_norm_rope_bwd(qkv[:, -tail:], H, Hkv, rope, *part,
                                  pos[:, -tail:].contiguous(), w, w)
    assert torch.equal(dqkv[:, -tail:], last[0])
    # dw = sum of xh^2 w over all rows of about unit mean square.
    for g, heads in ((dqw, H), (dkw, Hkv)):
        assert torch.allclose(g / (N * heads), w, rtol=1e-2)


@pytest.mark.gpu
def test_captured_training_step_on_another_stream():
    """Norm and rotation, attention, its backward and theirs, captured once
    and replayed on other inputs, equal the eager calls."""
    B, N, H, Hkv, d = 2, 150, 6, 2, 64
    case = (B, N, H, Hkv, d, 64, False, "f32", True, False)
    x, gpu, args, kw, ref = setup(case)
    do = gpu["dq"]

    def step():
        q, k, v = fa.fa_qk_norm_rope(*args, **kw)
        o, lse = fa.fa_fwd_ext(q, k, v, True, 0.125)
        dq, dk, dv = fa.fa_bwd_ext(q, k, v, o, lse, do, True, 0.125)
        return (o,) + fa.fa_qk_norm_rope_bwd(*args, dq, dk, dv, **kw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s, capture_error_mode="thread_local"):
        out = step()
    for seed in (1, 2):
        gpu["qkv"].copy_(make(B, N, H, Hkv, d, 64, seed=seed)["qkv"])
        g.replay()
        want = step()
        torch.cuda.synchronize()
        # (dQ's fp32 additions come in any order: the attention backward is
        # not bitwise repeatable, everything else here is.)
        assert torch.equal(out[0], want[0])
        for a, b in zip(out[1:], want[1:]):
            a, b = f64(a), f64(b)
            assert np.linalg.norm(a - b) <= 4 * BF16 * np.linalg.norm(b)
