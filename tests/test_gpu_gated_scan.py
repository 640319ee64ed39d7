"""Gated linear recurrence on the GPU (kda_gated_scan, kda_gated_scan_g, their
gradients, kda_gated_scan_step) against the float64 oracle, within the bound
that the oracle carries for a float32 evaluation."""
import numpy as np
import pytest
import torch

from gated_delta_rule_98_b200 import kda
from layer_testutil import close, cu_of, cuda, draw
from oracle import scan

pytestmark = pytest.mark.gpu


def make(lens, C, dtype, entry, seed=0, state=True, mean=-3.0, pad=0):
    T, N = sum(lens), len(lens)
    p = dict(x=draw(seed, dtype, T + pad, C), dy=draw(seed + 1, dtype, T + pad, C),
             cu=cu_of(lens), L=max(lens), T=T)
    if entry == "z":
        p.update(z=draw(seed + 2, dtype, T + pad, C, mean=mean, std=1.5),
                 A=draw(seed + 3, "f32", C, std=0.3))
    else:
        p["g"] = -torch.exp(draw(seed + 2, "f32", T + pad, C, mean=mean, std=1.5))
    if state:
        p.update(h0=draw(seed + 4, "f32", N, C), dh=draw(seed + 5, "f32", N, C))
    return p


def gate_of(p):
    return (cuda(p["z"]), cuda(p["A"])) if "z" in p else (cuda(p["g"]),)


def run(p, equal=None, **kw):
    """(y, h_final, states), gradients; ``equal``: so many equal sequences without cu_seqlens."""
    fwd, bwd = ((kda.gated_scan, kda.gated_scan_backward) if "z" in p else
                (kda.gated_scan_g, kda.gated_scan_g_backward))
    how = dict(num_seqs=equal) if equal else dict(cu_seqlens=cuda(p["cu"]), max_seqlen=p["L"])
    x, gate, h0 = cuda(p["x"]), gate_of(p), cuda(p.get("h0"))
    out = fwd(x, *gate, h0=h0, save_states=True, **how, **kw)
    grads = bwd(x, *gate, out[2], cuda(p["dy"]), h0=h0, dh_final=cuda(p.get("dh")), **how)
    torch.cuda.synchronize()
    return out, grads


def check(p, out, grads):
    T = p["T"]
    cu = p["cu"].tolist()
    by = {k: p[k][:T] if k in "zg" else p[k] for k in ("z", "A", "g") if k in p}
    f = scan.forward(p["x"][:T], cu, h0=p.get("h0"), **by)
    b = scan.backward(p["x"][:T], cu, p["dy"][:T], h0=p.get("h0"), dh_final=p.get("dh"), **by)
    close(out[0][:T], f["y"], f["e_y"], "y")
    close(out[1], f["h_final"], f["e_h_final"], "h_final")
    names = ("dx", "dz", "dA", "dh0") if "z" in p else ("dx", "dg", "dh0")
    for name, got in zip(names, grads):
        got = got[:T] if name in ("dx", "dz", "dg") else got
        close(got, b[name], b["e_" + name], name)


LENS = [
    [1], [2], [63], [64], [65], [129], [1000],
    [1, 1, 1, 1, 1], [0, 5, 0, 0, 64, 1, 0], [64, 64, 128], [63, 65, 1, 127, 200, 0],
    [300, 31, 33, 500], [3] * 200,
]


@pytest.mark.parametrize("entry", ["z", "g"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", LENS, ids=lambda v: "_".join(map(str, v))[:24])
def test_packed_lengths(lens, dtype, entry):
    p = make(lens, 40, dtype, entry, seed=len(lens))
    check(p, *run(p))


@pytest.mark.parametrize("entry", ["z", "g"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [8, 16, 24, 72, 264, 2056])
def test_channels(C, dtype, entry):
    p = make([70, 0, 133], C, dtype, entry, seed=C, state=C % 3 == 0)
    check(p, *run(p))


@pytest.mark.parametrize("entry", ["z", "g"])
@pytest.mark.parametrize("N,L", [(1, 5000), (3, 1700), (7, 1), (1, 9001)])
def test_equal_sequences_and_long_axes(N, L, entry):
    """Few channels over many tokens (the token axis is split over blocks), with long memories."""
    p = make([L] * N, 16, "f32", entry, seed=N + L, mean=-5.0)
    check(p, *run(p, equal=N))


def test_long_packed_split():
    p = make([2500, 0, 40, 3100, 1, 1, 1800], 24, "bf16", "z", seed=77, mean=-6.0)
    check(p, *run(p))


@pytest.mark.parametrize("entry", ["z", "g"])
def test_padded_batch_leaves_rows_behind_the_last_sequence(entry):
    p = make([70, 9], 24, "bf16", entry, seed=5, pad=60)
    how = dict(cu_seqlens=cuda(p["cu"]), max_seqlen=p["L"])
    x, gate = cuda(p["x"]).clone(), [t.clone() for t in gate_of(p)]
    x[79:] = float("nan")
    gate[0][79:] = float("nan")
    y = torch.full_like(x, 7.0)
    fwd = kda.gated_scan if entry == "z" else kda.gated_scan_g
    out = fwd(x, *gate, h0=cuda(p["h0"]), save_states=True, y=y, **how)
    torch.cuda.synchronize()
    assert (y[79:] == 7).all()
    bwd = kda.gated_scan_backward if entry == "z" else kda.gated_scan_g_backward
    grads = bwd(x, *gate, out[2], cuda(p["dy"]), h0=cuda(p["h0"]), dh_final=cuda(p["dh"]), **how)
    check(p, out, grads)


def test_nothing_leaks_between_sequences():
    """Infinities and NaN of one sequence and channel stay there; in it they last."""
    p = make([70, 30, 200, 5], 16, "f32", "z", seed=6)
    clean_out, clean_grads = run(p)
    p["x"][80, 3] = float("nan")
    p["x"][120, 5] = float("inf")
    p["dy"][85, 7] = float("nan")
    out, grads = run(p)
    y = out[0].cpu()
    assert torch.isnan(y[80:100, 3]).all() and torch.isinf(y[120:300, 5]).all()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[80:100, 3] = keep[100:300, 5] = False
    assert torch.equal(y[keep], clean_out[0].cpu()[keep])
    dx = grads[0].cpu()
    assert torch.isnan(dx[70:86, 7]).all()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[70:100, 7] = False
    assert torch.equal(dx[keep], clean_grads[0].cpu()[keep])


def test_gate_extremes():
    """z from -inf to +inf: nothing is forgotten, or e^-5 is kept; log-decay -inf clears."""
    T, C = 130, 8
    p = make([T], C, "f32", "z", seed=8)
    p["A"][:] = 0
    for c, v in enumerate((-300.0, 300.0, -80.0, 80.0, -20.0, 20.0, 0.0, 5.0)):
        p["z"][:, c] = v
    check(p, *run(p))
    p["z"][:, 0], p["z"][:, 1] = -float("inf"), float("inf")
    out, grads = run(p)
    assert torch.equal(out[0][:, 0].cpu(), p["h0"][0, 0].expand(T))
    a = np.exp(-5.0)
    want = scan.forward(p["x"][:, 1:2], [0, T], g=torch.full((T, 1), -5.0), h0=None)["y"] * (1 - a)
    want += p["h0"][0, 1].item() * a ** np.arange(1, T + 1)[:, None]
    close(out[0][:, 1:2], want, 64 * scan.U * (np.abs(want) + 4), "y at z = inf")
    q = make([100, 40], 16, "f32", "g", seed=9)
    q["g"][50, ::2] = -float("inf")
    q["g"][100, :] = -float("inf")
    q["g"][60, 1] = 0.0
    check(q, *run(q))


def test_long_memory_keeps_its_accuracy():
    """1 - a near 1e-6 over thousands of tokens: a bias of 1 - a would add up."""
    p = make([4000], 8, "f32", "z", seed=10)
    p["A"][:] = 0
    p["z"][:] = torch.linspace(-16, -8, 8)
    p["x"][:] = p["x"].abs() + 1
    p["h0"][:] = 0
    f = scan.forward(p["x"], [0, 4000], z=p["z"], A=p["A"], h0=p["h0"])
    out, _ = run(p)
    # per step: 32 units of its terms; they add up linearly at worst, which the oracle's
    # bound has; against a value built from 1 - a alone it is at most 32 * 4000 units
    close(out[0], f["y"], np.minimum(f["e_y"], 32 * 4000 * scan.U * np.abs(f["y"])), "y")


def test_repeated_calls_are_bit_identical():
    for C, lens in ((16, [5000, 3, 700]), (2048, [100, 300]), (264, [4099])):
        p = make(lens, C, "bf16", "z", seed=C)
        a, b = run(p), run(p)
        for s, t in zip((*a[0], *a[1]), (*b[0], *b[1])):
            if s is not a[0][2]:
                assert torch.equal(s, t)


def test_in_place_state_and_no_final_state():
    p = make([50, 0, 90], 24, "f32", "z", seed=12)
    h = cuda(p["h0"]).clone()
    how = dict(cu_seqlens=cuda(p["cu"]), max_seqlen=90)
    out, _ = run(p)
    y, hf = kda.gated_scan(cuda(p["x"]), *gate_of(p), h0=h, h_final=h, **how)
    assert hf is h and torch.equal(hf, out[1]) and torch.equal(y, out[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,C", [(1, 8), (3, 24), (256, 2048), (5, 1000)])
def test_step(B, C, dtype):
    x, z = draw(1, dtype, B, C), draw(2, dtype, B, C, mean=-2.0)
    A, h = draw(3, "f32", C, std=0.3), draw(4, "f32", B, C)
    hc = h.cuda()
    y = kda.gated_scan_step(x.cuda(), z.cuda(), A.cuda(), hc)
    f = scan.forward(x, list(range(B + 1)), z=z, A=A, h0=h)
    close(y, f["y"], f["e_y"], "y")
    close(hc, f["h_final"], f["e_h_final"], "h")


def test_steps_continue_a_prefill():
    """A prefill, then single steps, equals one longer prefill."""
    N, L, more, C = 4, 37, 5, 48
    x, z = draw(1, "bf16", N, L + more, C), draw(2, "bf16", N, L + more, C, mean=-3.0)
    A = draw(3, "f32", C, std=0.3)
    flat = lambda t, a, b: t[:, a:b].reshape(-1, C).contiguous().cuda()
    y, h = kda.gated_scan(flat(x, 0, L), flat(z, 0, L), A.cuda(), num_seqs=N)
    ys = [y.view(N, L, C)]
    for t in range(L, L + more):
        ys.append(kda.gated_scan_step(flat(x, t, t + 1), flat(z, t, t + 1), A.cuda(),
                                      h)[:, None])
    cu = [n * (L + more) for n in range(N + 1)]
    f = scan.forward(x.reshape(-1, C), cu, z=z.reshape(-1, C), A=A)
    close(torch.cat(ys, 1).reshape(-1, C), f["y"], f["e_y"], "y")
    close(h, f["h_final"], f["e_h_final"], "h")


def test_captured_graph_and_side_stream():
    p = make([300, 200], 24, "bf16", "z", seed=13)
    want_out, want_grads = run(p)
    x, gate, h0, dy, dh = (cuda(p["x"]), gate_of(p), cuda(p["h0"]), cuda(p["dy"]), cuda(p["dh"]))
    how = dict(cu_seqlens=cuda(p["cu"]), max_seqlen=300, h0=h0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out = kda.gated_scan(x, *gate, save_states=True, **how)
        grads = kda.gated_scan_backward(x, *gate, out[2], dy, dh_final=dh, **how)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gout = kda.gated_scan(x, *gate, save_states=True, **how)
        ggrads = kda.gated_scan_backward(x, *gate, gout[2], dy, dh_final=dh, **how)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for got in ((*out[:2], *grads), (*gout[:2], *ggrads)):
        for s, t in zip(got, (*want_out[:2], *want_grads)):
            assert torch.equal(s, t)


def test_empty_problem():
    A = torch.zeros(16, device="cuda")
    x = torch.zeros(0, 16, device="cuda")
    h0 = torch.randn(3, 16, device="cuda")
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    y, h, st = kda.gated_scan(x, x, A, h0=h0, cu_seqlens=cu, max_seqlen=0, save_states=True)
    assert torch.equal(h, h0) and y.shape == x.shape
    dx, dz, dA, dh0 = kda.gated_scan_backward(x, x, A, st, x, h0=h0, dh_final=h0, cu_seqlens=cu,
                                              max_seqlen=0)
    assert torch.equal(dh0, h0) and (dA == 0).all()
    y, h = kda.gated_scan_g(x, x, cu_seqlens=cu, max_seqlen=0)
    assert (h == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_state_of_sequences_inside_one_span(dtype):
    """A sequence's start and its end lie in one warp's span: h0 is read before
    h_final, which is the same tensor, is written."""
    p = make([10, 8, 20, 3, 1, 1, 30], 16, dtype, "z", seed=21)
    out, _ = run(p)
    h = cuda(p["h0"]).clone()
    y, hf = kda.gated_scan(cuda(p["x"]), *gate_of(p), h0=h, h_final=h, cu_seqlens=cuda(p["cu"]),
                           max_seqlen=30)
    assert torch.equal(hf, out[1]) and torch.equal(y, out[0])


def test_in_place_state_with_a_split_token_axis():
    p = make([3000, 5, 2900], 16, "bf16", "z", seed=22)
    f = scan.forward(p["x"], p["cu"].tolist(), z=p["z"], A=p["A"], h0=p["h0"])
    h = cuda(p["h0"]).clone()
    y, hf = kda.gated_scan(cuda(p["x"]), *gate_of(p), h0=h, h_final=h, cu_seqlens=cuda(p["cu"]),
                           max_seqlen=3000)
    close(hf, f["h_final"], f["e_h_final"], "h_final")
    close(y, f["y"], f["e_y"], "y")


@pytest.mark.parametrize("entry", ["z", "g"])
def test_thousands_of_short_sequences(entry):
    rng = np.random.default_rng(23)
    p = make([int(v) for v in rng.integers(0, 4, 3000)], 16, "f32", entry, seed=23)
    check(p, *run(p))


@pytest.mark.parametrize("entry", ["z", "g"])
def test_padded_batch_with_a_split_token_axis(entry):
    """The last sequence ends inside a segment; the segments behind it have nothing to do."""
    p = make([1500, 0, 700], 16, "bf16", entry, seed=24, pad=6000)
    y = torch.full_like(cuda(p["x"]), 7.0)
    out, grads = run(p, y=y)
    assert (y[2200:] == 7).all()
    check(p, out, grads)


def test_no_sequence_has_tokens():
    p = make([0, 0], 16, "bf16", "z", seed=25, pad=100) | dict(L=0)
    out, grads = run(p)
    assert torch.equal(out[1].cpu(), p["h0"]) and torch.equal(grads[3].cpu(), p["dh"])
    assert (grads[2] == 0).all()


def test_workspace_contents_do_not_matter():
    p = make([4000, 30, 2000], 24, "bf16", "z", seed=26)
    want, want_grads = run(p)
    n = kda.kda_gated_scan_workspace_size(p["T"], 24)
    how = dict(cu_seqlens=cuda(p["cu"]), max_seqlen=4000, h0=cuda(p["h0"]))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    out = kda.gated_scan(cuda(p["x"]), *gate_of(p), save_states=True, workspace=ws, **how)
    ws.fill_(255)
    grads = kda.gated_scan_backward(cuda(p["x"]), *gate_of(p), out[2], cuda(p["dy"]),
                                    dh_final=cuda(p["dh"]), workspace=ws, **how)
    for a, b in zip((*out[:2], *grads), (*want[:2], *want_grads)):
        assert torch.equal(a, b)


def test_stream_argument():
    p = make([4000, 200], 24, "bf16", "z", seed=27)
    want, want_grads = run(p)
    x, gate, h0, dy, dh = (cuda(p["x"]), gate_of(p), cuda(p["h0"]), cuda(p["dy"]), cuda(p["dh"]))
    how = dict(cu_seqlens=cuda(p["cu"]), max_seqlen=4000, h0=h0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = kda.gated_scan(x, *gate, save_states=True, stream=side, **how)
    grads = kda.gated_scan_backward(x, *gate, out[2], dy, dh_final=dh, stream=side, **how)
    # a workspace of the calls that was handed out again here would be overwritten now
    junk = [torch.full((1 << 16,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    for a, b in zip((*out[:2], *grads), (*want[:2], *want_grads)):
        assert torch.equal(a, b)
    del junk


def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the last sequence, alone, gives the same bits."""
    T, C, tail = 65600, 32768, 96          # the tail starts on a span
    x, z, dy = (torch.zeros(T, C, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    for i, t in enumerate((x, z, dy)):
        t[-tail:] = draw(30 + i, "bf16", tail, C, mean=-3.0 if t is z else 0.0).cuda()
    A = draw(33, "f32", C, std=0.3).cuda()
    cu = torch.tensor([0, T - tail, T], dtype=torch.int32, device="cuda")
    how = dict(cu_seqlens=cu, max_seqlen=T)
    y, h, st = kda.gated_scan(x, z, A, save_states=True, **how)
    dx, dz, _, dh0 = kda.gated_scan_backward(x, z, A, st, dy, **how)
    a, b, c = (t[-tail:].clone() for t in (x, z, dy))
    y1, h1, st1 = kda.gated_scan(a, b, A, save_states=True)
    dx1, dz1, _, dh1 = kda.gated_scan_backward(a, b, A, st1, c)
    assert torch.equal(y[-tail:], y1) and torch.equal(h[1:], h1)
    assert torch.equal(dx[-tail:], dx1) and torch.equal(dz[-tail:], dz1)
    assert torch.equal(dh0[1:], dh1) and (y[:100] == 0).all() and (y[-tail - 9:-tail] == 0).all()


@pytest.mark.parametrize("seed", range(6))
def test_gate_far_below_zero_keeps_its_accuracy(seed):
    """sigmoid(u) near e^u takes |u| times the relative error of u = e^A z."""
    p = make([120, 0, 77], 32, "f32", "z", seed=60 + 10 * seed, mean=-9.0, state=seed % 2 == 0)
    check(p, *run(p))


def check_channels(p, out, grads, idx):
    """check() on the channels ``idx`` alone (the recurrence does not mix channels)."""
    T, cut = p["T"], torch.as_tensor(idx)
    q = {k: v[..., cut] if torch.is_tensor(v) and k != "cu" else v for k, v in p.items()}
    on = lambda t: t.index_select(t.dim() - 1, cut.to(t.device))
    assert q["x"].shape == (T, len(idx))
    check(q, tuple(on(t) for t in out), tuple(on(t) for t in grads))


def some_channels(C, seed, n=48):
    """The first and last columns of channels, and some between."""
    rng = np.random.default_rng(seed)
    return sorted({*range(8), *range(C - 8, C), *rng.choice(C, min(n, C), replace=False).tolist()})


# Sequences of a long axis: one alone, or starts at every offset from a span's
# first token, some next to each other, with a long one last.
def long_axis(T, packed, seed):
    if not packed:
        return [T]
    rng = np.random.default_rng(seed)
    lens = [1, 0, 31, 32, 33, 63, 64, 65, 1, 1]
    while sum(lens) < T // 2:
        lens.append(int(rng.integers(1, T // 12)))
    return lens + [T - sum(lens)]


# Sizes by what a launch does with them: a block alone on its SM (channel groups times
# segments at most 148) or one of two, the token axis whole or cut, and many more spans
# a warp than it has slots, so that every slot is filled again several times.
LONG = [
    ("bf16", 3000, 1192),    # alone, whole: 94 spans over 12 or 15 warps
    ("f32", 6000, 600),
    ("bf16", 3000, 2400),    # paired, whole: 94 spans over 8 warps
    ("f32", 4000, 1208),
    ("bf16", 20000, 512),    # paired, 9 segments of 70 spans
    ("f32", 20000, 264),     # paired, 8 segments of 40 spans
    ("bf16", 6000, 512),     # paired, 9 segments of 21 spans
    ("f32", 4099, 264),      # paired, 8 segments of 9 spans
    ("bf16", 80000, 32),     # alone, 63 segments of 40 spans
    ("f32", 80000, 16),      # alone, 63 segments of 20 spans
]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("entry", ["z", "g"])
@pytest.mark.parametrize("dtype,T,C", LONG)
def test_long_axes_in_every_launch_form(dtype, T, C, entry, packed):
    seed = T + C + packed
    lens = long_axis(T, packed, seed)
    assert sum(lens) == T and min(lens) >= 0
    p = make(lens, C, dtype, entry, seed=seed, state=packed)
    check_channels(p, *run(p), some_channels(C, seed))


# Channels from one that forgets nothing to one that forgets in two tokens, over an axis
# on which the rounding of every decay to 2^-24 of itself would add up to thousands of
# units (0.4% of the state).  64 channels: the axis is cut; 1200: it is whole.
SLOW_T = 65536


def lasting(dtype):
    """Units of 2^-24 that a state which lasts may collect over the axis.  bf16, 32 tokens:
    half a unit for each of four runs' products and three products of them, one for the
    state.  fp32, 64 tokens: one for the state.  And 1024 for a span's own decays and the
    sums of logarithms."""
    return (4.5 * SLOW_T / 32 if dtype == "bf16" else SLOW_T / 64) + 1024


def slow_channels(C, lo, hi):
    return np.resize(np.logspace(np.log10(lo), np.log10(hi), 64), C)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [64, 1200])
def test_a_constant_does_not_drift(C, dtype):
    """h0 = x = 1 gives 1 whatever the gates: h stays between the extremes of h0 and x."""
    s = slow_channels(C, 1e-9, 0.4)
    z = torch.from_numpy(np.log(s / (1 - s))).to(draw(0, dtype, 1).dtype).cuda()
    z = z.expand(SLOW_T, C).contiguous()
    one, A = torch.ones_like(z), torch.zeros(C, device="cuda")
    h0 = torch.ones(1, C, device="cuda")
    y, h = kda.gated_scan(one, z, A, h0=h0)
    bound = lasting(dtype) * scan.U
    close(h, np.ones((1, C)), np.full((1, C), bound), "h_final")
    close(y, np.ones((SLOW_T, C)), np.full((SLOW_T, C), bound), "y")


@pytest.mark.parametrize("entry", ["z", "g"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [64, 1200])
def test_slow_channels_forget_at_their_rate(C, dtype, entry):
    """Without inputs h_final is the product of the decays, and so is dh0 for
    dh_final = 1: against the exponential of their sum in 64 bits.  Bound, of the result:
    as above, and the decays' own relative error (24 units, and 2 |u| for the rounding of
    u = e^A z, which the gate cannot tell from one of z) times the sum."""
    rate = slow_channels(C, 1e-9, 9e-4)          # of the log-decay; at most 60 in all
    zero = torch.zeros(SLOW_T, C, dtype=draw(0, dtype, 1).dtype, device="cuda")
    one = torch.ones(1, C, device="cuda")
    if entry == "z":
        z = torch.from_numpy(np.log(rate / 5 / (1 - rate / 5))).to(zero.dtype)
        gate = z.cuda().expand(SLOW_T, C).contiguous(), torch.zeros(C, device="cuda")
        u, log = np.abs(scan.f64(z)), -5.0 * scan.sigmoid(scan.f64(z))
        fwd, bwd = kda.gated_scan, kda.gated_scan_backward
    else:
        g = torch.from_numpy(-rate).float()
        gate = (g.cuda().expand(SLOW_T, C).contiguous(),)
        u, log = 0.0, scan.f64(g)
        fwd, bwd = kda.gated_scan_g, kda.gated_scan_g_backward
    want = np.exp(SLOW_T * log)[None]
    units = lasting(dtype) + SLOW_T * np.abs(log) * (24 + 2 * u)
    bound = units[None] * scan.U * want
    _, h, states = fwd(zero, *gate, h0=one, save_states=True)
    close(h, want, bound, "h_final")
    grads = bwd(zero, *gate, states, zero, h0=one, dh_final=one)
    close(grads[-1], want, bound, "dh0")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_do_not_drift(dtype):
    """One rounding of the state a step: 2000 steps leave a constant within 2000 units."""
    s = slow_channels(64, 1e-9, 0.4)
    z = torch.from_numpy(np.log(s / (1 - s))).to(draw(0, dtype, 1).dtype).cuda()
    z = z.expand(3, 64).contiguous()
    one, A, h = torch.ones_like(z), torch.zeros(64, device="cuda"), torch.ones(3, 64, device="cuda")
    for _ in range(2000):
        y = kda.gated_scan_step(one, z, A, h)
    close(h, np.ones((3, 64)), np.full((3, 64), 2000 * scan.U), "h")
    close(y, np.ones((3, 64)), np.full((3, 64), 2000 * scan.U), "y")


@pytest.mark.parametrize("entry", ["z", "g"])
@pytest.mark.parametrize("C", [16, 1200])
def test_slow_channels_next_to_fast_ones_and_starts(C, entry):
    """Slow and fast channels in one warp, starts inside, infinities: against the oracle."""
    lens = [700, 64, 0, 1, 2300, 31, 900]
    p = make(lens, C, "f32", entry, seed=90 + C)
    if entry == "z":
        p["A"][:] = 0
        p["z"][:, ::2] = torch.linspace(-18, -6, C // 2)
    else:
        p["g"][:, ::2] = -torch.exp(torch.linspace(-18, -4, C // 2))
        p["g"][1000, 4] = -float("inf")
    check_channels(p, *run(p), some_channels(C, 5))
    p["x"][900, 2] = float("inf")
    out, _ = run(p)
    assert torch.isinf(out[0][900:3065, 2]).all() and torch.isfinite(out[0][3065:, 2]).all()


def test_growing_states_keep_the_product():
    """A log-decay above 0 is outside of what the complement is for."""
    p = make([300, 90], 16, "f32", "g", seed=95)
    p["g"][:, ::3] = 1e-3
    p["g"][:, 1::3] = 0.0
    check(p, *run(p))


def _tail_check(got, want, units, what):
    """Relative to the value; results next to 2^-126 may be flushed."""
    g, ok = got.cpu().double().numpy(), np.abs(want) > 1e-36
    assert (np.abs(g[~ok]) <= 2e-36).all() and ok.sum() > 1000, what
    close(torch.from_numpy(g[ok]).to(got.dtype), want[ok], (units * scan.U * np.abs(want))[ok], what)


@pytest.mark.parametrize("mean", [-4, -9, -20, -40, -60])
def test_tail_of_the_gate(mean):
    """1 - a and the slope from thousands of first tokens with u down to -100: u = e^A z
    has two roundings, each of at most one unit of 2^-24 of itself, and the exponential
    takes |u| times that; 32 units for the rest (the slope: 64, it has both factors)."""
    N, C = 256, 1024
    z = draw(100 - mean, "f32", N, C, mean=mean, std=1.5)
    A = draw(200 - mean, "f32", C, std=0.3)
    u = np.exp(scan.f64(A)) * scan.f64(z)
    s, units = scan.sigmoid(u), 32 + 2 * np.abs(u)
    m = -np.expm1(-5 * s)
    one, zg, Ag = torch.ones(N, C, device="cuda"), z.cuda(), A.cuda()
    y = kda.gated_scan_step(one, zg, Ag, torch.zeros(N, C, device="cuda"))
    _tail_check(y, m, units, "step")
    how = dict(num_seqs=N)
    y, h, states = kda.gated_scan(one, zg, Ag, save_states=True, **how)
    _tail_check(y, m, units, "y")
    _tail_check(h, m, units, "h_final")
    dx, dz, _, _ = kda.gated_scan_backward(one, zg, Ag, states, one, **how)
    _tail_check(dx, m, units, "dx")
    # h_{t-1} - x = -1 and l = 1: dz = 5 s (1 - s) e^A a
    want = 5 * s * scan.sigmoid(-u) * np.exp(scan.f64(A)) * np.exp(-5 * s)
    _tail_check(dz, want, units + 32, "dz")


def test_tail_of_a_given_decay():
    """exp(g) takes g log2(e) in float32: a rounding of at most one unit of itself, and a
    quarter of one for the constant's; 32 units for the rest."""
    N, C = 256, 1024
    g = -torch.exp(draw(7, "f32", N, C, mean=2.0, std=1.0))
    one, zero = torch.ones(N, C, device="cuda"), torch.zeros(N, C, device="cuda")
    y, h = kda.gated_scan_g(zero, g.cuda(), h0=one, num_seqs=N)
    want = np.exp(scan.f64(g))
    _tail_check(y, want, 32 + 1.25 * np.abs(scan.f64(g)), "y")
    _tail_check(h, want, 32 + 1.25 * np.abs(scan.f64(g)), "h_final")


@pytest.mark.parametrize("entry", ["z", "g"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_states_with_strong_gates_stay_in_their_sequence(dtype, entry):
    """Products of strong decays become 0: an infinite state is then infinite or NaN to
    the end of its sequence, and no other sequence or channel changes."""
    p = make([50, 700, 90], 16, dtype, entry, seed=97)
    if entry == "z":
        p["z"][:] = p["z"].abs() + 2
    else:
        p["g"][:] = p["g"] - 5
    clean, _ = run(p)
    p["x"][60, 5] = float("inf")
    p["x"][70, 9] = float("nan")
    out, _ = run(p)
    y, keep = out[0].cpu().float(), torch.ones(840, 16, dtype=torch.bool)
    keep[60:750, 5] = keep[70:750, 9] = False
    assert not torch.isfinite(y[~keep]).any()
    assert torch.equal(out[0].cpu()[keep], clean[0].cpu()[keep])
    assert not torch.isfinite(out[1][1, [5, 9]]).any() and torch.isfinite(out[1][2]).all()
