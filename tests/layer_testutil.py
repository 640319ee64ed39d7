"""Shared helpers of the tests of the gated scan, the prologue's gradient and
the norm-and-rotation pass: inputs and the comparison with a bounded oracle."""
import numpy as np
import torch

from gated_delta_rule_98_b200 import synth

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def draw(seed, dtype, *shape, mean=0.0, std=1.0):
    v = np.random.default_rng(seed).standard_normal(shape) * std + mean
    return torch.from_numpy(np.asarray(v)).to(DT[dtype])


def cu_of(lens):
    return synth.cu_from_lengths(lens)


def cuda(t):
    return None if t is None else t.cuda()


def close(got, want, bound, what):
    """|got - want| <= bound + half a step of got's type (a rounding to it is off
    by at most eps / 2 of the value), + the smallest normal number (results
    below it may be flushed to zero)."""
    g = got.detach().cpu().double().numpy()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    if not g.size:
        return
    info = torch.finfo(got.dtype)
    tol = bound * (1 + info.eps) + np.abs(want) * info.eps / 2 + 2 * info.tiny
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {g.size} off, first at "
                           f"{tuple(np.argwhere(bad)[0])}: got {g[bad][0]!r}, want "
                           f"{want[bad][0]!r} +- {tol[bad][0]:.3e}")
