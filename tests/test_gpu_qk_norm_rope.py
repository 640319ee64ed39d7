"""Norm of the query and key heads with the position rotation on the GPU
against the float64 oracle, within the oracle's bound for a float32 evaluation."""
import numpy as np
import pytest
import torch

from gated_delta_rule_98_b200 import kda
from layer_testutil import close, cuda, draw
from oracle import qk_rope

pytestmark = pytest.mark.gpu


def make(T, Hq, Hk, d, rot, dtype, weights=True, seed=0, far=100000):
    rng = np.random.default_rng(seed)
    p = dict(q=draw(seed, dtype, T, Hq, d), k=draw(seed + 1, dtype, T, Hk, d),
             dq=draw(seed + 2, dtype, T, Hq, d), dk=draw(seed + 3, dtype, T, Hk, d),
             pos=torch.from_numpy(rng.integers(-far, far, T).astype(np.int32)),
             freqs=torch.from_numpy(10000.0 ** (-2.0 * np.arange(rot // 2) / max(rot, 1))))
    p["qw"] = draw(seed + 4, "f32", d, mean=1.0, std=0.2) if weights else None
    p["kw"] = draw(seed + 5, "f32", d, mean=1.0, std=0.2) if weights else None
    return p


def call(p, q=None, k=None, **kw):
    q, k = cuda(p["q"]) if q is None else q, cuda(p["k"]) if k is None else k
    how = dict(q_weight=cuda(p["qw"]), k_weight=cuda(p["kw"]), **kw)
    out = kda.qk_norm_rope(q, k, cuda(p["pos"]), cuda(p["freqs"]), **how)
    back = kda.qk_norm_rope_backward(q, k, cuda(p["dq"]), cuda(p["dk"]), cuda(p["pos"]),
                                     cuda(p["freqs"]), **how)
    torch.cuda.synchronize()
    return out, back


def check(p, out, back, **kw):
    for i, n in enumerate("qk"):
        want, bound = qk_rope.forward(p[n], p["pos"], p["freqs"], p[n + "w"], **kw)
        close(out[i], want, bound, n)
        dv, dw, e_dv, e_dw = qk_rope.backward(p[n], p["d" + n], p["pos"], p["freqs"],
                                              p[n + "w"], **kw)
        close(back[i], dv, e_dv, "d" + n)
        if p[n + "w"] is None:
            assert back[2 + i] is None
        else:
            close(back[2 + i], dw, e_dw, "d%s_weight" % n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,d,rot", [
    (1, 1, 1, 32, 32), (5, 3, 1, 32, 8), (4, 16, 16, 128, 128), (7, 32, 8, 128, 64),
    (33, 6, 3, 64, 32), (9, 5, 2, 64, 64), (3, 8, 4, 128, 96), (2, 17, 7, 128, 0),
    (130, 2, 1, 64, 24),
])
def test_shapes(T, Hq, Hk, d, rot, interleaved, dtype):
    p = make(T, Hq, Hk, d, rot, dtype, weights=T % 2 == 1, seed=T)
    check(p, *call(p, interleaved=interleaved), interleaved=interleaved)


def test_many_tokens():
    p = make(6000, 2, 1, 32, 32, "bf16", seed=2)
    check(p, *call(p))


def test_far_positions():
    """The largest positions an int32 holds, both signs."""
    p = make(8, 2, 2, 64, 64, "f32", seed=3)
    p["pos"] = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 0, 1, -1, 123456789, 65535],
                            dtype=torch.int32)
    # an angle of 2^31 radians is known to 2^31 * 2^-52 of itself in 64 bits, on both sides
    out, back = call(p)
    slack = 2.0 ** -20
    for i, n in enumerate("qk"):
        want, bound = qk_rope.forward(p[n], p["pos"], p["freqs"], p[n + "w"])
        close(out[i], want, bound + slack * np.abs(want).max(), n)


@pytest.mark.parametrize("interleaved", [False, True])
def test_slices_of_one_projection_and_in_place(interleaved):
    T, Hq, Hk, d, rot = 21, 4, 2, 64, 32
    p = make(T, Hq, Hk, d, rot, "bf16", seed=4)
    width = (Hq + 2 * Hk) * d
    fused = torch.zeros(T, width, dtype=torch.bfloat16)
    fused[:, :Hq * d] = p["q"].reshape(T, -1)
    fused[:, Hq * d:(Hq + Hk) * d] = p["k"].reshape(T, -1)
    fused[:, (Hq + Hk) * d:] = 5
    f = fused.cuda()
    q, k = f[:, :Hq * d].view(T, Hq, d), f[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d)
    out, back = call(p, q, k, interleaved=interleaved)
    assert torch.equal(f.cpu(), fused)
    check(p, out, back, interleaved=interleaved)
    dq, dk = cuda(p["dq"]).clone(), cuda(p["dk"]).clone()
    how = dict(q_weight=cuda(p["qw"]), k_weight=cuda(p["kw"]), interleaved=interleaved)
    b = kda.qk_norm_rope_backward(q, k, dq, dk, cuda(p["pos"]), cuda(p["freqs"]), dq=dq, dk=dk,
                                  **how)
    assert b[0] is dq and torch.equal(dq, back[0]) and torch.equal(dk, back[1])
    kda.qk_norm_rope(q, k, cuda(p["pos"]), cuda(p["freqs"]), q_out=q, k_out=k, **how)
    assert torch.equal(q, out[0]) and torch.equal(k, out[1]) and (f[:, (Hq + Hk) * d:] == 5).all()


def test_zero_rows_infinities_and_nan_stay_in_their_row():
    p = make(6, 4, 2, 64, 32, "f32", seed=5)
    p["q"][1] = 0
    p["dk"][2] = 0
    check(p, *call(p))
    clean, _ = call(p)
    p["q"][3, 2, 5] = float("nan")
    p["q"][4, 1, 0] = float("inf")
    p["k"][0, 0, 1] = float("nan")
    out, _ = call(p)
    keep = torch.ones(6, 4, dtype=torch.bool)
    keep[3, 2] = keep[4, 1] = False
    assert torch.equal(out[0].cpu()[keep], clean[0].cpu()[keep])
    assert torch.equal(out[1].cpu()[1:], clean[1].cpu()[1:])
    assert torch.isnan(out[0][3, 2]).all()


def test_eps_zero_and_large():
    p = make(5, 2, 2, 32, 16, "f32", seed=6)
    for eps in (0.0, 3.0):
        check(p, *call(p, eps=eps), eps=eps)


def test_no_tokens():
    p = make(0, 4, 2, 64, 32, "bf16")
    out, back = call(p)
    assert out[0].shape == (0, 4, 64) and back[1].shape == (0, 2, 64)
    assert (back[2] == 0).all() and (back[3] == 0).all()


def test_repeated_captured_and_side_stream():
    p = make(700, 4, 2, 128, 128, "bf16", seed=7)
    g = {k: cuda(v) for k, v in p.items()}
    how = dict(q_weight=g["qw"], k_weight=g["kw"])

    def f():
        return (*kda.qk_norm_rope(g["q"], g["k"], g["pos"], g["freqs"], **how),
                *kda.qk_norm_rope_backward(g["q"], g["k"], g["dq"], g["dk"], g["pos"],
                                           g["freqs"], **how))
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
        for s, t in zip(got, want):
            assert torch.equal(s, t)


def test_rotated_queries_and_keys_through_the_operator():
    """Norm and rotation, then the KDA prefill, which scales q and k to unit length
    itself: against the oracle on the rounded rows that the pass wrote."""
    from gated_delta_rule_98_b200 import synth
    from kda_testutil import assert_close
    from oracle import ref
    T, H, d = 200, 2, 128
    inp = synth.draw(T, H, d, d, seed=11, dtype="bf16")
    c = {k: cuda(v) for k, v in inp.items()}
    pos = torch.arange(T, dtype=torch.int32)
    freqs = torch.from_numpy(10000.0 ** (-2.0 * np.arange(d // 2) / d))
    q, k = kda.qk_norm_rope(c["q"], c["k"], pos.cuda(), freqs.cuda())
    want, bound = qk_rope.forward(inp["q"], pos, freqs)
    close(q, want, bound, "q")
    o, S = kda.forward(q, k, c["v"], c["z"], c["A"], c["beta"])
    torch.cuda.synchronize()
    o_ref, S_ref = ref.forward(q.cpu(), k.cpu(), inp["v"], inp["beta"], z=inp["z"], A=inp["A"])
    assert_close(o, o_ref, torch.bfloat16, "o")
    assert_close(S, S_ref, torch.bfloat16, "S_final")


def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the last tokens, alone, give the same bits."""
    T, H, d, tail = 65600, 256, 128, 40
    q, dq = (torch.zeros(T, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q[-tail:], dq[-tail:] = draw(50, "bf16", tail, H, d).cuda(), draw(51, "bf16", tail, H, d).cuda()
    k = torch.ones(T, 1, d, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    freqs = torch.from_numpy(10000.0 ** (-2.0 * np.arange(d // 2) / d)).cuda()
    out = kda.qk_norm_rope(q, k, pos, freqs)
    back = kda.qk_norm_rope_backward(q, k, dq, k, pos, freqs)
    cut = lambda t: t[-tail:].clone()
    out1 = kda.qk_norm_rope(cut(q), cut(k), cut(pos), freqs)
    back1 = kda.qk_norm_rope_backward(cut(q), cut(k), cut(dq), cut(k), cut(pos), freqs)
    assert torch.equal(out[0][-tail:], out1[0]) and torch.equal(back[0][-tail:], back1[0])
    assert torch.equal(out[1][-tail:], out1[1]) and (out[0][:50] == 0).all()


def test_stream_argument():
    p = make(300, 4, 2, 64, 64, "bf16", seed=12)
    want, want_back = call(p)
    g = {k: cuda(v) for k, v in p.items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    how = dict(q_weight=g["qw"], k_weight=g["kw"], stream=side)
    out = kda.qk_norm_rope(g["q"], g["k"], g["pos"], g["freqs"], **how)
    back = kda.qk_norm_rope_backward(g["q"], g["k"], g["dq"], g["dk"], g["pos"], g["freqs"], **how)
    junk = [torch.full((1 << 21,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    for a, b in zip((*out, *back), (*want, *want_back)):
        assert torch.equal(a, b)
    del junk
