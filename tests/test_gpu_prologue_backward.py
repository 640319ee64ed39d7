"""Gradient of the input prologue on the GPU against the float64 oracle, within
the bound that the oracle carries for a float32 evaluation."""
import pytest
import torch

from gated_delta_rule_98_b200 import kda
from layer_testutil import close, cu_of, cuda, draw
from oracle import scan

pytestmark = pytest.mark.gpu


def make(lens, C, W, dtype, seed=0, pad=0):
    T = sum(lens) + pad
    return dict(x=draw(seed, dtype, T, C), dy=draw(seed + 1, dtype, T, C),
                w=draw(seed + 2, "f32", C, W, std=W ** -0.5), cu=cu_of(lens), T=sum(lens),
                L=max(lens))


def check(p, dx, dw):
    T = p["T"]
    o = scan.conv_backward(p["x"][:T], p["w"], p["cu"].tolist(), p["dy"][:T])
    close(dx[:T], o["dx"], o["e_dx"], "dx")
    close(dw, o["dw"], o["e_dw"], "dw")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("lens", [
    [1], [3], [31], [32], [33], [255, 2], [700], [1] * 9, [2, 1, 3, 0, 0, 4, 1], [0, 30, 2, 32, 0],
    [29, 1, 1, 1, 32, 3, 90],
], ids=lambda v: "_".join(map(str, v))[:24])
def test_packed_lengths(lens, W, dtype):
    p = make(lens, 24, W, dtype, seed=W)
    dx, dw = kda.short_conv_swish_backward(cuda(p["x"]), cuda(p["w"]), cuda(p["dy"]),
                                           cu_seqlens=cuda(p["cu"]), max_seqlen=p["L"])
    check(p, dx, dw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C,N", [(8, 1), (136, 3), (1000, 2), (2048, 1)])
def test_channels_and_equal_sequences(C, N, dtype):
    p = make([90] * N, C, 4, dtype, seed=C)
    dx, dw = kda.short_conv_swish_backward(cuda(p["x"]), cuda(p["w"]), cuda(p["dy"]), num_seqs=N)
    check(p, dx, dw)


def test_large_values():
    p = make([200], 16, 4, "f32", seed=3)
    p["x"] *= 60
    dx, dw = kda.short_conv_swish_backward(cuda(p["x"]), cuda(p["w"]), cuda(p["dy"]), num_seqs=1)
    check(p, dx, dw)


def test_padded_batch_and_neighbours():
    """Rows behind the last sequence are not read or written; a NaN stays in its sequence."""
    p = make([50, 41], 24, 4, "bf16", seed=4, pad=37)
    x, dy = cuda(p["x"]).clone(), cuda(p["dy"]).clone()
    x[91:] = float("nan")
    dy[91:] = float("nan")
    how = dict(cu_seqlens=cuda(p["cu"]), max_seqlen=50)
    dx = torch.full_like(x, 7.0)
    _, dw = kda.short_conv_swish_backward(x, cuda(p["w"]), dy, dx=dx, **how)
    assert (dx[91:] == 7).all()
    check(p, dx, dw)
    x[49, 3] = float("nan")
    dy[50, 5] = float("nan")
    bad, _ = kda.short_conv_swish_backward(x, cuda(p["w"]), dy, **how)
    keep = torch.ones_like(bad, dtype=torch.bool)
    keep[46:50, 3] = keep[50:54, 5] = False
    keep[91:] = False
    assert torch.equal(bad[keep], dx[keep])
    assert torch.isnan(bad[46:50, 3]).all()


def test_repeated_captured_and_side_stream():
    p = make([400, 300], 72, 4, "bf16", seed=5)
    x, w, dy, cu = cuda(p["x"]), cuda(p["w"]), cuda(p["dy"]), cuda(p["cu"])
    f = lambda: kda.short_conv_swish_backward(x, w, dy, cu_seqlens=cu, max_seqlen=400)
    want = f()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a = f()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = f()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for got in (a, b):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_empty_problem():
    x = torch.zeros(0, 16, device="cuda")
    dx, dw = kda.short_conv_swish_backward(x, torch.ones(16, 4, device="cuda"), x, num_seqs=0)
    assert dx.shape == x.shape and (dw == 0).all()


def test_trains_the_recurrent_block():
    """Prologue, recurrence, and the gradients back through both, as a training
    step uses them: against the oracle's chain on the same rounded tensors."""
    from oracle import prologue
    lens, C = [90, 1, 64], 40
    p = make(lens, C, 4, "f32", seed=6)
    z, A = draw(9, "f32", p["T"], C, mean=-3.0), draw(10, "f32", C, std=0.3)
    cu = p["cu"].tolist()
    how = dict(cu_seqlens=cuda(p["cu"]), max_seqlen=p["L"])
    u = kda.short_conv_swish(cuda(p["x"]), cuda(p["w"]), **how)
    y, h, st = kda.gated_scan(u, cuda(z), cuda(A), save_states=True, **how)
    du, dz, dA, _ = kda.gated_scan_backward(u, cuda(z), cuda(A), st, cuda(p["dy"]), **how)
    dx, dw = kda.short_conv_swish_backward(cuda(p["x"]), cuda(p["w"]), du, **how)
    u64 = prologue.short_conv_swish(p["x"], p["w"], cu)
    # the prologue's own error: 32 units of its terms, at most 8 in magnitude here
    eu = 32 * 8 * scan.U
    f = scan.forward(u.cpu(), cu, z=z, A=A)
    close(u, u64, eu + 0 * u64, "u")
    close(y, f["y"], f["e_y"], "y")
    b = scan.backward(u.cpu(), cu, p["dy"], z=z, A=A)
    close(du, b["dx"], b["e_dx"], "du")
    close(dz, b["dz"], b["e_dz"], "dz")
    close(dA, b["dA"], b["e_dA"], "dA")
    o = scan.conv_backward(p["x"], p["w"], cu, du.cpu())
    close(dx, o["dx"], o["e_dx"], "dx")
    close(dw, o["dw"], o["e_dw"], "dw")


def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the last sequence, alone, gives the same bits."""
    T, C, tail = 65600, 32768, 96
    x, dy = (torch.zeros(T, C, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[-tail:], dy[-tail:] = draw(40, "bf16", tail, C).cuda(), draw(41, "bf16", tail, C).cuda()
    w = draw(42, "f32", C, 4, std=0.5).cuda()
    cu = torch.tensor([0, T - tail, T], dtype=torch.int32, device="cuda")
    dx, dw = kda.short_conv_swish_backward(x, w, dy, cu_seqlens=cu, max_seqlen=T)
    dx1, dw1 = kda.short_conv_swish_backward(x[-tail:].clone(), w, dy[-tail:].clone())
    assert torch.equal(dx[-tail:], dx1) and (dx[:100] == 0).all()
    # dw's sums are grouped otherwise: tail terms of magnitude |du x|, each rounded
    assert ((dw - dw1).abs() <= tail * 2.0 ** -24 * 30).all()
