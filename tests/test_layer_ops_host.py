"""CPU tests of the gated scan, the prologue's gradient and the norm-and-rotation
pass: the oracles against differences and against independent forms, and the
refusals of the C ABI and of the binding (all before any CUDA call)."""
import numpy as np
import pytest
import torch

from gated_delta_rule_98_b200 import kda
from oracle import prologue, qk_rope, scan

FAKE = 0x10000  # aligned fake device address: never dereferenced by these calls
BAD, UNS = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def built():
    from gated_delta_rule_98_b200 import build
    build.build()


def _difference(f, v, i, step=1e-6):
    p, m = v.copy(), v.copy()
    p[i] += step
    m[i] -= step
    return (f(p) - f(m)) / (2 * step)


@pytest.mark.parametrize("by_z", [True, False])
def test_scan_oracle_gradients_against_differences(by_z):
    rng = np.random.default_rng(3)
    cu, C = [0, 3, 3, 4, 9], 2
    T, N = cu[-1], len(cu) - 1
    v = dict(x=rng.standard_normal((T, C)), h0=rng.standard_normal((N, C)))
    if by_z:
        v.update(z=rng.standard_normal((T, C)), A=0.3 * rng.standard_normal(C))
    else:
        v.update(g=-np.exp(rng.standard_normal((T, C))))
    dy, dh = rng.standard_normal((T, C)), rng.standard_normal((N, C))
    grads = scan.backward(v["x"], cu, dy, dh_final=dh, **{k: v[k] for k in v if k != "x"})
    for name in v:
        def loss(value):
            w = dict(v, **{name: value})
            f = scan.forward(w["x"], cu, **{k: w[k] for k in w if k != "x"})
            return (f["y"] * dy).sum() + (f["h_final"] * dh).sum()
        for i in np.ndindex(v[name].shape):
            want = _difference(loss, v[name], i)
            assert abs(grads["d" + name][i] - want) <= 1e-7 * (1 + abs(want)), (name, i)


def test_scan_oracle_is_a_convex_average_with_the_library_gate():
    """With the gate entry, h_t is the average of h0 and the inputs under the
    weights (1 - a_s) prod a, which add to 1; the gate is the operator's own."""
    rng = np.random.default_rng(4)
    T, C = 12, 3
    z, A = rng.standard_normal((T, C)), rng.standard_normal(C)
    one = scan.forward(np.ones((T, C)), [0, T], z=z, A=A, h0=np.ones((1, C)))
    assert np.abs(one["y"] - 1).max() < 1e-14
    x, h0 = rng.standard_normal((T, C)), rng.standard_normal((1, C))
    a = np.exp(-5.0 / (1.0 + np.exp(-np.exp(A) * z)))
    want = sum((1 - a[s]) * np.prod(a[s + 1:], 0) * x[s] for s in range(T)) + np.prod(a, 0) * h0[0]
    got = scan.forward(x, [0, T], z=z, A=A, h0=h0)["h_final"][0]
    assert np.abs(got - want).max() < 1e-13


def test_conv_oracle_gradient_against_differences():
    rng = np.random.default_rng(5)
    cu, C, W = [0, 1, 1, 6, 8], 2, 4
    T = cu[-1]
    x, w, dy = rng.standard_normal((T, C)), rng.standard_normal((C, W)), rng.standard_normal((T, C))
    grads = scan.conv_backward(x, w, cu, dy)
    for i in np.ndindex(x.shape):
        want = _difference(lambda v: (prologue.short_conv_swish(v, w, cu) * dy).sum(), x, i)
        assert abs(grads["dx"][i] - want) <= 1e-7 * (1 + abs(want))
    for i in np.ndindex(w.shape):
        want = _difference(lambda v: (prologue.short_conv_swish(x, v, cu) * dy).sum(), w, i)
        assert abs(grads["dw"][i] - want) <= 1e-7 * (1 + abs(want))


@pytest.mark.parametrize("interleaved", [False, True])
def test_qk_oracle_gradient_and_rotation(interleaved):
    rng = np.random.default_rng(6)
    T, H, d, rot = 3, 2, 12, 8
    v, dout = rng.standard_normal((T, H, d)), rng.standard_normal((T, H, d))
    w, pos, freqs = rng.standard_normal(d), np.array([0, 5, -3]), 10.0 ** -np.arange(rot // 2)
    how = dict(eps=1e-2, interleaved=interleaved)
    dv, dw, _, _ = qk_rope.backward(v, dout, pos, freqs, w, **how)
    for i in np.ndindex(v.shape):
        want = _difference(lambda u: (qk_rope.forward(u, pos, freqs, w, **how)[0] * dout).sum(),
                           v, i)
        assert abs(dv[i] - want) <= 1e-7 * (1 + abs(want))
    for i in range(d):
        want = _difference(lambda u: (qk_rope.forward(v, pos, freqs, u, **how)[0] * dout).sum(),
                           w, i)
        assert abs(dw[i] - want) <= 1e-7 * (1 + abs(want))
    # products of rotated rows depend on the distance of their positions alone
    a = qk_rope.forward(v, pos, freqs, **how)[0]
    b = qk_rope.forward(v, pos + 1000, freqs, **how)[0]
    assert np.abs(np.einsum("thd,shd->tsh", a, a) - np.einsum("thd,shd->tsh", b, b)).max() < 1e-10
    assert np.abs(qk_rope.forward(v, 0 * pos, freqs, **how)[0][..., rot:] - a[..., rot:]).max() == 0


def _scan(entry="z", back=False, **over):
    a = dict(x=FAKE, gate=FAKE, A=FAKE, h0=None, cu=None, N=1, T=64, L=64, C=32, dt=kda.KDA_BF16,
             out=FAKE, h=FAKE, states=FAKE, dy=FAKE, dgate=FAKE, dA=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(over)
    gate = (a["gate"], a["A"]) if entry == "z" else (a["gate"],)
    size = (a["cu"], a["N"], a["T"], a["L"], a["C"], a["dt"])
    tail = (a["ws"], a["wsb"], None)
    if not back:
        fn = kda.kda_gated_scan if entry == "z" else kda.kda_gated_scan_g
        return fn(a["x"], *gate, a["h0"], *size, a["out"], a["h"], a["states"], *tail)
    fn = kda.kda_gated_scan_backward if entry == "z" else kda.kda_gated_scan_g_backward
    grads = (a["dgate"], a["dA"]) if entry == "z" else (a["dgate"],)
    return fn(a["x"], *gate, a["states"], a["h0"], *size, a["dy"], None, a["out"], *grads, a["h"],
              *tail)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("entry", ["z", "g"])
@pytest.mark.parametrize("over,want", [
    (dict(x=None), BAD), (dict(gate=None), BAD), (dict(out=None), BAD), (dict(ws=None), BAD),
    (dict(wsb=4), BAD), (dict(x=FAKE + 8), BAD), (dict(gate=FAKE + 4), BAD),
    (dict(h0=FAKE + 4), BAD), (dict(h=FAKE + 4), BAD), (dict(states=FAKE + 8), BAD),
    (dict(cu=FAKE + 2), BAD), (dict(T=65), BAD), (dict(N=-1), BAD), (dict(N=0, L=0), BAD),
    (dict(T=-64, L=-64), BAD), (dict(C=0), UNS), (dict(C=12), UNS), (dict(C=-8), UNS),
    (dict(dt=2), UNS),
])
def test_gated_scan_rejects_bad_arguments(entry, back, over, want):
    assert _scan(entry, back, **over) == want


def test_gated_scan_rejects_missing_gradient_arguments():
    for over in (dict(states=None), dict(dy=None), dict(dgate=None), dict(dy=FAKE + 2)):
        assert _scan("z", True, **over) == BAD
        assert _scan("g", True, **over) == BAD
    assert _scan("z", True, dA=None) == BAD
    assert _scan("z", A=None) == BAD
    assert kda.kda_gated_scan_workspace_size(64, 12) == 0
    assert kda.kda_gated_scan_workspace_size(-1, 16) == 0
    assert kda.kda_gated_scan_workspace_size(0, 8) > 0
    # nothing to do: no sequences, no tokens
    assert _scan("z", N=0, T=0, L=0, x=None, gate=None, A=None, out=None) == kda.KDA_OK


def test_sizes_beyond_the_kernels_arithmetic_are_refused():
    T = 0x7fffff01
    assert _scan("z", T=T, L=T) == UNS and _scan("g", True, T=T, L=T) == UNS
    assert kda.kda_short_conv_swish_backward(FAKE, FAKE, FAKE, None, 1, T, T, 8, 4, kda.KDA_BF16,
                                             FAKE, FAKE, FAKE, 1 << 60, None) == UNS
    # (Hq + Hk) * d above 2^20
    assert kda.kda_qk_norm_rope(FAKE, 1 << 20, FAKE, 64, FAKE, FAKE, None, None, 1e-6, 1,
                                1 << 14, 1, 64, 64, 0, kda.KDA_BF16, FAKE, 1 << 20, FAKE, 64,
                                None) == UNS


def test_gradient_of_the_initial_state_is_not_written_over_the_final_states():
    st = kda.kda_gated_scan_g_backward(FAKE, FAKE, FAKE, None, None, 1, 64, 64, 32, kda.KDA_F32,
                                       FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40, None)
    assert st == BAD


def test_gated_scan_step_rejects_bad_arguments():
    def step(x=FAKE, h=FAKE, B=4, C=32, dt=kda.KDA_F32):
        return kda.kda_gated_scan_step(x, FAKE, FAKE, h, B, C, dt, FAKE, None)
    assert step(x=None) == BAD
    assert step(h=FAKE + 4) == BAD
    assert step(B=-1) == BAD
    assert step(C=20) == UNS
    assert step(dt=9) == UNS
    assert step(x=None, B=0) == kda.KDA_OK


def test_short_conv_swish_backward_rejects_bad_arguments():
    size = kda.kda_short_conv_swish_backward_workspace_size
    assert size(64, 32, 4) > 0 and size(64, 12, 4) == 0 and size(64, 32, 5) == 0

    def back(x=FAKE, w=FAKE, dy=FAKE, C=64, W=4, T=32, N=1, L=32, dt=kda.KDA_BF16, dx=FAKE,
             dw=FAKE, ws=FAKE, wsb=1 << 40):
        return kda.kda_short_conv_swish_backward(x, w, dy, None, N, T, L, C, W, dt, dx, dw, ws,
                                                 wsb, None)
    for over in (dict(x=None), dict(w=None), dict(dy=None), dict(dx=None), dict(dw=None),
                 dict(ws=None), dict(wsb=8), dict(x=FAKE + 8), dict(dy=FAKE + 8),
                 dict(w=FAKE + 2), dict(dw=FAKE + 2), dict(T=33), dict(N=-1, T=-32)):
        assert back(**over) == BAD, over
    for over in (dict(W=0), dict(W=5), dict(C=12), dict(dt=3)):
        assert back(**over) == UNS, over


@pytest.mark.parametrize("back", [False, True])
def test_qk_norm_rope_rejects_bad_arguments(back):
    def call(q=FAKE, k=FAKE, qs=256, ks=128, pos=FAKE, freqs=FAKE, qw=None, eps=1e-6, T=8, Hq=4,
             Hk=2, d=64, rot=32, dt=kda.KDA_BF16, qo=FAKE, qos=256, dout=FAKE, ws=FAKE,
             wsb=1 << 40):
        if not back:
            return kda.kda_qk_norm_rope(q, qs, k, ks, pos, freqs, qw, None, eps, T, Hq, Hk, d,
                                        rot, 0, dt, qo, qos, FAKE, 128, None)
        return kda.kda_qk_norm_rope_backward(q, qs, k, ks, dout, 256, FAKE, 128, pos, freqs, qw,
                                             None, eps, T, Hq, Hk, d, rot, 0, dt, qo, qos, FAKE,
                                             128, None, None, ws, wsb, None)
    for over in (dict(q=None), dict(k=None), dict(qo=None), dict(q=FAKE + 8), dict(qs=248),
                 dict(qs=260), dict(ks=64), dict(qos=128), dict(pos=None), dict(pos=FAKE + 2),
                 dict(freqs=None), dict(freqs=FAKE + 4), dict(qw=FAKE + 4), dict(eps=-1.0),
                 dict(eps=float("nan")), dict(eps=float("inf")), dict(T=-1), dict(Hq=-1)):
        assert call(**over) == BAD, over
    for over in (dict(d=96), dict(d=256), dict(rot=12), dict(rot=72), dict(rot=-8), dict(dt=2)):
        assert call(**over) == UNS, over
    if back:
        assert call(dout=None) == BAD and call(ws=None) == BAD and call(wsb=16) == BAD
        assert kda.kda_qk_norm_rope_backward_workspace_size(8, 96) == 0


def test_binding_rejects_wrong_tensors():
    T, C = 6, 16
    x, z = torch.zeros(T, C), torch.zeros(T, C)
    A, st = torch.zeros(C), torch.zeros(1, C)
    ok = [lambda: kda.gated_scan(x, z, A), lambda: kda.gated_scan_g(x, z),
          lambda: kda.gated_scan_step(x, z, A, torch.zeros(T, C)),
          lambda: kda.gated_scan_backward(x, z, A, st, x),
          lambda: kda.short_conv_swish_backward(x, torch.zeros(C, 4), x)]
    for f in ok:                                                # right, but on the CPU
        with pytest.raises(ValueError, match="GPU only"):
            f()
    for f in (lambda: kda.gated_scan(x, z.bfloat16(), A),
              lambda: kda.gated_scan(x, z, torch.zeros(C + 1)),
              lambda: kda.gated_scan(x.t().contiguous().t(), z, A),
              lambda: kda.gated_scan(x, z, A, h0=torch.zeros(2, C)),
              lambda: kda.gated_scan(x, z, A, cu_seqlens=torch.zeros(2, dtype=torch.int32)),
              lambda: kda.gated_scan(x, z, A, max_seqlen=6,
                                     cu_seqlens=torch.zeros(2, dtype=torch.int64)),
              lambda: kda.gated_scan_g(x, z.double()),
              lambda: kda.gated_scan_backward(x, z, A, torch.zeros(2, C), x),
              lambda: kda.gated_scan_backward(x, z, A, st, x[:5]),
              lambda: kda.gated_scan_step(x, z, A, torch.zeros(T, C, dtype=torch.bfloat16)),
              lambda: kda.short_conv_swish_backward(x, torch.zeros(C + 1, 4), x)):
        with pytest.raises(ValueError):
            f()
    q, k = torch.zeros(T, 4, 32), torch.zeros(T, 2, 32)
    pos, freqs = torch.zeros(T, dtype=torch.int32), torch.zeros(16, dtype=torch.float64)
    with pytest.raises(ValueError, match="GPU only"):
        kda.qk_norm_rope(q, k, pos, freqs)
    for f in (lambda: kda.qk_norm_rope(q, k[:5], pos, freqs),
              lambda: kda.qk_norm_rope(q, k, pos.long(), freqs),
              lambda: kda.qk_norm_rope(q, k, pos, freqs.float()),
              lambda: kda.qk_norm_rope(q, k, pos[:5], freqs),
              lambda: kda.qk_norm_rope(q, k, pos, freqs, q_weight=torch.zeros(31)),
              lambda: kda.qk_norm_rope(q.transpose(0, 1).contiguous().transpose(0, 1), k, pos,
                                       freqs),
              lambda: kda.qk_norm_rope(q, k, pos, freqs, q_out=k),
              lambda: kda.qk_norm_rope_backward(q, k, q.bfloat16(), k, pos, freqs)):
        with pytest.raises(ValueError):
            f()


def _qk_backward(T, Hq, Hk, pos, freqs, dqw=None, dkw=None, d=64, rot=32, ws=FAKE, stream=None):
    """The rotation's gradient through the C ABI on fp32 rows that do not exist."""
    nbytes = kda.kda_qk_norm_rope_backward_workspace_size(T, d)
    return kda.kda_qk_norm_rope_backward(None, 0, None, 0, None, 0, None, 0, pos, freqs, None,
                                         None, 1e-6, T, Hq, Hk, d, rot, 0, kda.KDA_F32, None, 0,
                                         None, 0, dqw, dkw, ws, nbytes, stream)


@pytest.mark.parametrize("T,Hq,Hk", [(0, 4, 2), (5, 0, 0), (0, 0, 0)])
def test_rotation_gradient_without_rows_launches_nothing(T, Hq, Hk):
    """positions and freqs are allowed to be NULL there: a kernel would read
    address 0.  Without a GPU every launch fails, so KDA_OK means that there was none."""
    assert _qk_backward(T, Hq, Hk, None, None) == kda.KDA_OK
    assert _qk_backward(T, Hq, Hk, FAKE, FAKE) == kda.KDA_OK
    assert _qk_backward(T, Hq, Hk, FAKE, None, ws=None) == BAD


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk", [(0, 4, 2), (5, 0, 0), (0, 0, 0)])
def test_rotation_gradient_without_rows_clears_the_weight_gradients(T, Hq, Hk):
    ws = torch.empty(kda.kda_qk_norm_rope_backward_workspace_size(T, 64), dtype=torch.uint8,
                     device="cuda")
    dqw, dkw = torch.full((64,), 7.0, device="cuda"), torch.full((65,), 7.0, device="cuda")
    st = _qk_backward(T, Hq, Hk, None, None, dqw.data_ptr(), dkw.data_ptr(), ws=ws.data_ptr(),
                      stream=torch.cuda.current_stream().cuda_stream)
    assert st == kda.KDA_OK
    assert (dqw == 0).all() and (dkw[:64] == 0).all() and dkw[64] == 7


def test_binding_rejects_a_stream_of_another_gpu():
    """It would be made current on its own GPU, and the call would run on another stream."""
    from types import SimpleNamespace
    stream = SimpleNamespace(device=torch.device("cuda", 1))
    x, A, st = torch.zeros(6, 16), torch.zeros(16), torch.zeros(1, 16)
    q, pos = torch.zeros(6, 2, 32), torch.zeros(6, dtype=torch.int32)
    freqs = torch.zeros(16, dtype=torch.float64)
    for f in (lambda: kda.gated_scan(x, x, A, stream=stream),
              lambda: kda.gated_scan_g(x, x, stream=stream),
              lambda: kda.gated_scan_backward(x, x, A, st, x, stream=stream),
              lambda: kda.gated_scan_g_backward(x, x, st, x, stream=stream),
              lambda: kda.gated_scan_step(x, x, A, torch.zeros(6, 16), stream=stream),
              lambda: kda.short_conv_swish_backward(x, torch.zeros(16, 4), x, stream=stream),
              lambda: kda.qk_norm_rope(q, q, pos, freqs, stream=stream),
              lambda: kda.qk_norm_rope_backward(q, q, q, q, pos, freqs, stream=stream)):
        with pytest.raises(ValueError, match="stream"):
            f()


@pytest.mark.parametrize("C", [(1 << 28) + 8, (1 << 31) - 8])
def test_channels_beyond_the_launch_arithmetic_are_refused(C):
    """Counting the blocks of 2^31 - 8 channels passes 32 bits; the sizes say 0 for
    what the calls refuse, and for the largest sizes that they take they do not."""
    big = 1 << 60
    assert kda.kda_short_conv_swish_backward(FAKE, FAKE, FAKE, None, 1, 1, 1, C, 4, kda.KDA_F32,
                                             FAKE, FAKE, FAKE, big, None) == UNS
    assert _scan("z", C=C, wsb=big) == UNS and _scan("g", True, C=C, wsb=big) == UNS
    for T, size in ((1, C), (0x7fffff01, 8)):
        assert kda.kda_short_conv_swish_backward_workspace_size(T, size, 4) == 0
        assert kda.kda_gated_scan_workspace_size(T, size) == 0
    for T, size in ((1, 1 << 28), (0x7fffff00, 8), (0x7fffff00, 1 << 28)):
        assert kda.kda_short_conv_swish_backward_workspace_size(T, size, 4) >= 16 * size
        assert kda.kda_gated_scan_workspace_size(T, size) >= 12 * size
