"""Gradient of the input prologue on the GPU against the float64 oracle, within
the bound that the oracle carries for a float32 evaluation."""
import numpy as np
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


# What one run of a warp holds (the longest of 8 to 128 tokens that still gives enough
# blocks: 240 of bf16, 120 of fp32; a block has 8 runs of 128 channels): more groups of
# 8 tokens than the warp has slots, so that every slot is filled again.
RUNS = [
    ("bf16", 1100, 3840, 16), ("bf16", 1100, 7680, 32), ("bf16", 1100, 12808, 64),
    ("bf16", 1100, 15368, 128), ("f32", 1100, 1920, 16), ("f32", 1100, 3840, 32),
    ("f32", 1100, 6408, 64), ("f32", 1100, 7688, 128),
]


def check_channels(p, dx, dw, seed, n=40):
    """check() on some channels alone (the prologue does not mix channels)."""
    C, rng = p["x"].shape[1], np.random.default_rng(seed)
    idx = torch.tensor(sorted({*range(4), *range(C - 8, C),
                               *rng.choice(C, min(n, C), replace=False).tolist()}))
    q = dict(p, x=p["x"][:, idx], dy=p["dy"][:, idx], w=p["w"][idx])
    check(q, dx[:, idx.cuda()], dw[idx.cuda()])


@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("dtype,T,C,run", RUNS)
def test_every_length_of_a_run(dtype, T, C, run, W):
    """Runs that cross no sequence start, and starts in a run's first, middle and last
    groups, at every offset in a group."""
    lens = [3 * run + 5, 1, 2, 8, 7, 9, 40, 3, 0, 1, 1, 25]
    if sum(lens) < T:
        lens.append(T - sum(lens))
    p = make(lens, C, W, dtype, seed=run + W, pad=T - sum(lens))
    dx, dw = kda.short_conv_swish_backward(cuda(p["x"]), cuda(p["w"]), cuda(p["dy"]),
                                           cu_seqlens=cuda(p["cu"]), max_seqlen=p["L"])
    check_channels(p, dx, dw, seed=run)
    q = make([T], C, W, dtype, seed=run + W + 50)
    dx, dw = kda.short_conv_swish_backward(cuda(q["x"]), cuda(q["w"]), cuda(q["dy"]))
    check_channels(q, dx, dw, seed=run)


@pytest.mark.parametrize("dtype,W", [("bf16", 4), ("f32", 3)])
def test_blocks_that_take_a_second_tile(dtype, W):
    """More tokens than 512 blocks of 8 runs of 128: a block goes on with the next tile.
    Against the definition in 64 bits, shifted tensors instead of loops; the bound is
    the oracle's, 32 units of 2^-24 of every term."""
    T, C, U = 512 * 8 * 128 + 12345, 8, scan.U
    x, dy, w = draw(70, dtype, T, C), draw(71, dtype, T, C), draw(72, "f32", C, W, std=W ** -0.5)
    starts = [0, 128, 129, 1024, 300001, T - 12345, T - 12340, T - 1]
    cu = torch.tensor([*starts, T], dtype=torch.int32)
    dx, dw = kda.short_conv_swish_backward(x.cuda(), w.cuda(), dy.cuda(), cu_seqlens=cu.cuda(),
                                           max_seqlen=T)
    x, dy, w = x.double(), dy.double(), w.double()
    seq = torch.zeros(T, dtype=torch.int64)
    seq[torch.tensor(starts)] = 1
    seq = seq.cumsum(0)

    def earlier(v, j):                  # row t: v of token t - j of the same sequence, or 0
        out = torch.zeros_like(v)
        out[j:] = v[:T - j] * (seq[j:] == seq[:T - j])[:, None] if j else v
        return out

    def later(v, j):
        out = torch.zeros_like(v)
        out[:T - j] = v[j:] * (seq[j:] == seq[:T - j])[:, None] if j else v
        return out

    terms = [w[:, W - 1 - j] * earlier(x, j) for j in range(W)]
    u, e_u = sum(terms), 32 * U * sum(t.abs() for t in terms)
    p = torch.sigmoid(u)
    du = dy * p * (1 + u * (1 - p))
    e_du = dy.abs() * (0.5 * e_u + 32 * U * p * (1 + u.abs() * (1 - p)))
    want = sum(w[:, W - 1 - j] * later(du, j) for j in range(W))
    bound = sum(w[:, W - 1 - j].abs() * later(e_du + 32 * U * du.abs(), j) for j in range(W))
    close(dx, want.numpy(), bound.numpy(), "dx")
    want = torch.stack([(du * earlier(x, j)).sum(0) for j in reversed(range(W))], 1)
    bound = torch.stack([((e_du + 64 * U * du.abs()) * earlier(x, j).abs()).sum(0)
                         for j in reversed(range(W))], 1)
    close(dw, want.numpy(), bound.numpy(), "dw")
