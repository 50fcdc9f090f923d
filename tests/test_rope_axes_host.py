"""The rotation's axes are read on the host: what lies on a device is refused and
not waited for."""
import pytest
import torch

from tiled_attention_bwd_gb300 import fa


def refused(axes):
    with pytest.raises(ValueError, match="host"):
        fa._axis_bytes(axes)


def test_axes_on_a_device_are_refused():
    # ("meta" stands in for a device: its elements cannot be had either.)
    t = torch.zeros(4, dtype=torch.int32, device="meta")
    refused(t)
    refused([t[0], 1, 2, 0])
    refused((t[i] for i in range(4)))
    assert fa._axis_bytes(torch.tensor([0, 2, 1])) == b"\0\2\1"
    assert fa._axis_bytes([torch.tensor(1), 2]) == b"\1\2"


@pytest.mark.gpu
def test_axes_on_the_gpu_are_refused_in_a_capture_too():
    B, N, H, Hkv, d = 1, 3, 2, 1, 64
    dev = "cuda:0"
    qkv = torch.randn((B, N, H + 2 * Hkv, d), device=dev).bfloat16()
    rope = torch.rand((8, d), device=dev)
    pos = torch.zeros((2, B, N), dtype=torch.int32, device=dev)
    axes = torch.zeros(d // 2, dtype=torch.int32, device=dev)
    out = fa.fa_qk_norm_rope_axes(qkv, H, Hkv, rope, pos, bytes(d // 2))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        with pytest.raises(ValueError, match="host"):
            fa.fa_qk_norm_rope_axes(qkv, H, Hkv, rope, pos, axes)
        again = fa.fa_qk_norm_rope_axes(qkv, H, Hkv, rope, pos, bytes(d // 2))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, again):
        assert torch.equal(a, b)
