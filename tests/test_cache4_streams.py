"""Cache attention calls that run at the same time on several streams: every
input is on the device beforehand, all calls are queued behind one event, and
histories are long enough that each call fills the GPU and is joined from many
partial results."""
import pytest
import torch

from test_cache4 import attn_case, i32
from tiled_attention_bwd_gb300 import fa

STREAMS, CALLS = 3, 30


def on_device(c):
    return ((c["q"].cuda(), torch.from_numpy(c["cache"]).cuda(), i32(c["table"]),
             i32(c["lens"]), c["scale"]),
            dict(k_scale=c["gk"], v_scale=c["gv"]))


@pytest.mark.gpu
@pytest.mark.parametrize("own_workspace", [False, True])
def test_calls_that_run_together(own_workspace):
    """With a workspace of the call's own, and with one kept per stream."""
    cases = [attn_case(3, 8, 2, 1, 128, 64, [30000 - 97 * s, 9000, 500 + s], None, -1, seed=s)
             for s in range(STREAMS)]
    args = [on_device(c) for c in cases]
    want = [fa.fa_cache4_attn(*a, **k) for a, k in args]
    size = fa.fa_cache4_attn_workspace_size(3, 8, 2, 1, 128)
    spaces = [torch.empty(size, dtype=torch.uint8, device="cuda:0") if own_workspace else None
              for _ in args]
    outs = [[(torch.empty_like(w[0]), torch.empty_like(w[1])) for _ in range(CALLS)] for w in want]
    streams = [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    # Something that holds the streams back until all calls are queued.
    big = torch.empty((16384, 16384), device="cuda:0").normal_()
    gate, hold = torch.cuda.Event(), torch.cuda.Stream()
    with torch.cuda.stream(hold):
        for _ in range(4):
            big = (big @ big).clamp_(-1, 1)
        gate.record()
    for s in streams:
        s.wait_event(gate)
    for i in range(CALLS):
        for s, (a, k), w, o in zip(streams, args, spaces, outs):
            with torch.cuda.stream(s):
                fa.fa_cache4_attn(*a, out=o[i][0], lse=o[i][1], workspace=w, **k)
    torch.cuda.synchronize()
    assert fa.fa_check_device_status("cuda:0") == 0
    for w, per_call in zip(want, outs):
        for o, lse in per_call:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])


@pytest.mark.gpu
def test_two_graphs_with_workspaces_of_their_own_run_together():
    """Two captured calls, replayed on two streams at once."""
    cases = [attn_case(2, 8, 1, 1, 64, 64, [20000 + 311 * s, 700], None, -1, seed=s) for s in (1, 2)]
    args = [on_device(c) for c in cases]
    want = [fa.fa_cache4_attn(*a, **k) for a, k in args]
    graphs, outs, streams = [], [], []
    torch.cuda.synchronize()
    for a, k in args:
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        o = torch.empty_like(a[0]), torch.empty(a[0].shape[:3], device="cuda:0")
        w = torch.empty(fa.fa_cache4_attn_workspace_size(2, 8, 1, 1, 64), dtype=torch.uint8,
                        device="cuda:0")
        with torch.cuda.graph(g, stream=s, capture_error_mode="thread_local"):
            for _ in range(10):
                fa.fa_cache4_attn(*a, out=o[0], lse=o[1], workspace=w, **k)
        graphs.append(g), outs.append(o), streams.append(s)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
