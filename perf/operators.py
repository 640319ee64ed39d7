"""What the operators around the recurrent layer cost, in their plain form and through the library.

Three operators, all packed over sequences like the rest of the library:

* ``scan``: the gated linear recurrence of one number per channel, with its
  gradients and its step for one token a sequence.  The gate is the library's
  own, g = -5 sigmoid(e^A z), or a log-decay g given directly:

      z:  a = exp(g),  h_t = a_t h_{t-1} + (1 - a_t) x_t
      g:  a = exp(g),  h_t = a_t h_{t-1} + x_t

* ``conv``: the gradients of the input prologue, y = Swish(causal depthwise
  convolution of x), with respect to x and the taps.
* ``qk``: RMS norm of every query and key head and the position rotation in
  one pass, with its gradients.

``run`` is the plain form where ``own`` is false: elementary torch operations in
32 bits (the angles of the rotation in 64, since a far position times a frequency
does not fit 32), rounded once at the end.  ``exact`` is the definition in 64 bits.
"""
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
BASE = 10000.0      # base of the rotation's geometric frequencies


# --------------------------------------------------------------------- cases --

def listed():
    return [
        # one token for each of 256 requests (the decode workload's batch, 16 heads of 128)
        {"name": "scan step 256x2048", "op": "step", "T": 256, "C": 2048, "dtype": "bf16"},
        # one long prompt, the long prefill workload's size
        {"name": "scan prefill 65536x2048", "op": "scan", "gate": "z", "train": False, "T": 65536,
         "N": 1, "C": 2048, "dtype": "bf16", "cu": False, "state": False},
        # a training batch of packed documents, the packed workload's size (32 heads of 128)
        {"name": "scan train packed 32768x4096", "op": "scan", "gate": "z", "train": True,
         "T": 32768, "N": 10, "C": 4096, "dtype": "bf16", "cu": True, "state": True},
        # few channels over a long sequence: one rank's slice of the channels
        {"name": "scan_g train 65536x256", "op": "scan", "gate": "g", "train": True, "T": 65536,
         "N": 1, "C": 256, "dtype": "bf16", "cu": False, "state": False},
        # full precision, ragged sizes, an empty sequence among the packed ones
        {"name": "scan train f32 4099x264", "op": "scan", "gate": "z", "train": True, "T": 4099,
         "N": 6, "C": 264, "dtype": "f32", "cu": True, "state": True},
        # the prologue's gradient over q, k and v of 16 heads of 128 in one tensor
        {"name": "conv grad 32768x6144", "op": "conv", "T": 32768, "N": 10, "C": 6144, "W": 4,
         "dtype": "bf16", "cu": True},
        # a short training sequence
        {"name": "conv grad 512x2048", "op": "conv", "T": 512, "N": 1, "C": 2048, "W": 4,
         "dtype": "bf16", "cu": False},
        # many short documents, an odd number of channel vectors, three taps
        {"name": "conv grad f32 4099x1000", "op": "conv", "T": 4099, "N": 37, "C": 1000, "W": 3,
         "dtype": "f32", "cu": True},
        # one token for each of 256 requests at far positions
        {"name": "qk decode 256x16+16x128", "op": "qk", "train": False, "T": 256, "Hq": 16,
         "Hk": 16, "d": 128, "rot": 128, "pairs": False, "fused": True, "dtype": "bf16",
         "far": 1000000},
        # prefill, shared key heads, half of each head rotated
        {"name": "qk prefill 32768x32+8x128", "op": "qk", "train": False, "T": 32768, "Hq": 32,
         "Hk": 8, "d": 128, "rot": 64, "pairs": False, "fused": True, "dtype": "bf16",
         "far": 65536},
        # training, queries and keys as slices of one projection's output
        {"name": "qk train 16384x16+16x128", "op": "qk", "train": True, "T": 16384, "Hq": 16,
         "Hk": 16, "d": 128, "rot": 128, "pairs": True, "fused": True, "dtype": "bf16",
         "far": 16384},
        # full precision, odd counts of tokens and heads
        {"name": "qk train f32 1021x6+3x64", "op": "qk", "train": True, "T": 1021, "Hq": 6,
         "Hk": 3, "d": 64, "rot": 32, "pairs": False, "fused": False, "dtype": "f32",
         "far": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["step", "scan", "scan", "scan", "conv", "conv", "qk", "qk"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    half = 1 if dtype == "bf16" else 2      # keeps the bytes of the largest cases
    if op == "step":
        return {"op": op, "T": _log(rng, 1, 2048), "C": 8 * _log(rng, 4, 512), "dtype": dtype}
    if op in ("scan", "conv"):
        T = _log(rng, 1, 65536)
        C = 8 * min(_log(rng, 4, 768), max(1, (1 << 24) // (half * T)))
        N = _log(rng, 1, min(T, 512)) if rng.random() < 0.6 else 1
        case = {"op": op, "T": T, "N": N, "C": C, "dtype": dtype, "cu": N > 1 or rng.random() < 0.5}
        if op == "conv":
            return dict(case, W=rng.randint(1, 4))
        return dict(case, gate=rng.choice("zzg"), train=rng.random() < 0.7,
                    state=rng.random() < 0.6)
    d = rng.choice([32, 64, 128])
    Hk = _log(rng, 1, 32)
    Hq = Hk * rng.choice([1, 1, 2, 4]) if Hk <= 8 else Hk
    T = _log(rng, 1, min(65536, (1 << 27) // (half * (Hq + Hk) * d)))
    return {"op": op, "train": rng.random() < 0.6, "T": T, "Hq": Hq, "Hk": Hk, "d": d,
            "rot": rng.choice([d, d, d // 2]), "pairs": rng.random() < 0.4,
            "fused": rng.random() < 0.6, "dtype": dtype, "far": _log(rng, 64, 1000000)}


# -------------------------------------------------------------------- inputs --

def _lengths(T, N, seed):
    """N lengths that sum to T, cut at random places (so that some may be empty)."""
    r = random.Random(seed)
    cuts = sorted(r.randint(0, T) for _ in range(N - 1))
    ends = [0] + cuts + [T]
    return [b - a for a, b in zip(ends, ends[1:])]


def prepare(case, seed):
    dev, dt = DEVICE, DT[case["dtype"]]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, mean=0.0, std=1.0, dtype=torch.float32):
        out = torch.empty(shape, dtype=dtype, device=dev)
        return out.normal_(mean, std, generator=gen)

    s = {"case": case}
    op, T = case["op"], case["T"]
    if op in ("step", "scan"):
        C, N = case["C"], case.get("N", 1)
        s["x"] = normal(T, C, dtype=dt)
        if case.get("gate", "z") == "z":
            # sigmoid(e^A z) around 0.05: the state remembers from a few to a few hundred tokens
            s["z"] = normal(T, C, mean=-3.0, std=1.5, dtype=dt)
            s["A"] = normal(C, std=0.3)
        else:
            s["g"] = normal(T, C, mean=-3.0, std=1.5).exp_().neg_()
        if op == "step":
            s["h"] = normal(T, C)
            return s
        s["h0"] = normal(N, C) if case["state"] else None
        if case["train"]:
            s["dy"] = normal(T, C, dtype=dt)
            s["dh"] = normal(N, C) if case["state"] else None
    elif op == "conv":
        C, W = case["C"], case["W"]
        s["x"] = normal(T, C, dtype=dt)
        s["w"] = normal(C, W, std=W ** -0.5)
        s["dy"] = normal(T, C, dtype=dt)
    else:
        Hq, Hk, d, rot = case["Hq"], case["Hk"], case["d"], case["rot"]
        if case["fused"]:   # one projection's output: queries, keys, values side by side
            qkv = normal(T, (Hq + 2 * Hk) * d, dtype=dt)
            s["q"] = qkv[:, :Hq * d].view(T, Hq, d)
            s["k"] = qkv[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d)
        else:
            s["q"], s["k"] = normal(T, Hq, d, dtype=dt), normal(T, Hk, d, dtype=dt)
        s["q_weight"], s["k_weight"] = normal(d, mean=1.0, std=0.2), normal(d, mean=1.0, std=0.2)
        first = torch.randint(0, case["far"], (1,), generator=gen, device=dev)
        s["positions"] = (torch.arange(T, device=dev) * 7 + first).remainder(
            case["far"]).to(torch.int32)
        i = torch.arange(rot // 2, dtype=torch.float64, device=dev)
        s["freqs"] = BASE ** (-2.0 * i / rot)
        if case["train"]:
            s["dq"], s["dk"] = normal(T, Hq, d, dtype=dt), normal(T, Hk, d, dtype=dt)
    if op in ("scan", "conv"):
        lens = _lengths(T, case["N"], seed) if case["cu"] else [T // case["N"]] * case["N"]
        s["max_seqlen"] = max(lens)
        cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
        s["cu"] = cu.to(dev) if case["cu"] else None
        full = [n for n, length in enumerate(lens) if length]     # sequences with tokens
        at = cu.tolist()
        s["full"] = torch.tensor(full, device=dev)
        s["first"] = torch.tensor([at[n] for n in full], device=dev)
        s["last"] = torch.tensor([at[n + 1] - 1 for n in full], device=dev)
    return s


def work(case):
    e, T = SIZE[case["dtype"]], case["T"]
    if case["op"] == "step":
        n = T * case["C"]
        return {"bytes": n * (3 * e + 8), "flops": 8 * n}
    if case["op"] == "scan":
        n, N = T * case["C"], case["N"]
        gate = e if case["gate"] == "z" else 4
        states = (8 if case["state"] else 4) * N * case["C"]
        size = n * (2 * e + gate) + states
        if case["train"]:       # x, gate and dy in, dx and the gate's gradient out
            size += n * (3 * e + 2 * gate) + states
        return {"bytes": size, "flops": (30 if case["train"] else 10) * n}
    if case["op"] == "conv":
        n = T * case["C"]
        return {"bytes": 3 * e * n + 8 * case["C"] * case["W"], "flops": (6 * case["W"] + 12) * n}
    n = T * (case["Hq"] + case["Hk"]) * case["d"]
    return {"bytes": n * e * (5 if case["train"] else 2) + 4 * T,
            "flops": (25 if case["train"] else 8) * n}


# --------------------------------------------------------------- plain forms --

def _sigmoid(u):
    return 1.0 / (1.0 + torch.exp(-u))


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t from h_{-1} = 0, by doubling the distance that each element has seen."""
    s = 1
    while s < a.shape[0]:
        b = torch.cat([b[:s], b[s:] + a[s:] * b[:-s]])
        a = torch.cat([a[:s], a[s:] * a[:-s]])
        s *= 2
    return b


def _gate(s):
    """(a, 1 - a or None, sigmoid or None) in 32 bits."""
    if "z" in s:
        sig = _sigmoid(torch.exp(s["A"]) * s["z"].float())
        return torch.exp(-5.0 * sig), -torch.expm1(-5.0 * sig), sig
    return torch.exp(s["g"]), None, None


def _plain_step(s):
    a, m, _ = _gate(s)
    s["h"].copy_(a * s["h"] + m * s["x"].float())
    return {"y": s["h"].to(s["x"].dtype), "h": s["h"]}


def _plain_scan(s):
    case, dt = s["case"], s["x"].dtype
    x = s["x"].float()
    a, m, sig = _gate(s)
    b = x if m is None else m * x
    N, C = case["N"], case["C"]
    h0 = s["h0"] if s["h0"] is not None else x.new_zeros(N, C)
    first, last, full = s["first"], s["last"], s["full"]
    carried = a.clone()
    carried[first] = 0.0                    # nothing passes from one sequence to the next
    b = b.clone() if m is None else b
    b[first] += a[first] * h0[full]
    h = _scan(carried, b)
    h_final = h0.clone()
    h_final[full] = h[last]
    out = {"y": h.to(dt), "h_final": h_final}
    if not case["train"]:
        return out
    dh = s["dh"] if s["dh"] is not None else x.new_zeros(N, C)
    prev = torch.cat([h[:1], h[:-1]])       # the state before each token
    prev[first] = h0[full]
    lam = s["dy"].float().clone()           # .float() of 32 bits is the input itself
    lam[last] += dh[full]
    passed = torch.cat([a[1:], a[:1]])      # what token t+1 passes back to t
    passed[last] = 0.0
    lam = _scan(passed.flip(0), lam.flip(0)).flip(0)
    dh0 = dh.clone()
    dh0[full] = a[first] * lam[first]
    if m is None:
        out.update(dx=lam.to(dt), dg=lam * a * prev)
    else:
        slope = -5.0 * sig * (1.0 - sig) * torch.exp(s["A"])
        dz = lam * a * (prev - x) * slope
        out.update(dx=(lam * m).to(dt), dz=dz.to(dt), dA=(dz * s["z"].float()).sum(0))
    if case["state"]:
        out["dh0"] = dh0
    return out


def _shifted(v, j, seq):
    """v of j tokens later in the same sequence (j < 0: earlier), zero outside it."""
    if j == 0:
        return v
    out = torch.zeros_like(v)
    if abs(j) >= v.shape[0]:
        return out
    to, of = (slice(None, -j), slice(j, None)) if j > 0 else (slice(-j, None), slice(None, j))
    same = (seq[to] == seq[of]).to(v.dtype)
    out[to] = v[of] * same[:, None]
    return out


def _plain_conv(s):
    W = s["case"]["W"]
    x, w, dy = s["x"].float(), s["w"], s["dy"].float()
    seq = x.new_zeros(x.shape[0], dtype=torch.int32)
    seq[s["first"]] = 1
    seq = seq.cumsum(0)
    u = sum(w[:, W - 1 - j] * _shifted(x, -j, seq) for j in range(W))
    sig = _sigmoid(u)
    du = dy * sig * (1.0 + u * (1.0 - sig))
    dx = sum(w[:, W - 1 - j] * _shifted(du, j, seq) for j in range(W))
    dw = torch.stack([(du * _shifted(x, -j, seq)).sum(0) for j in reversed(range(W))], 1)
    return {"dx": dx.to(s["x"].dtype), "dw": dw}


def _rotate(v, cos, sin, rot, pairs):
    """The pairs of v's first `rot` channels turned by the angles (sin negated: turned back)."""
    r, rest = v[..., :rot], v[..., rot:]
    if pairs:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, rest], -1)


EPS = 1e-6


def _plain_qk(s):
    case = s["case"]
    rot, pairs = case["rot"], case["pairs"]
    angle = s["positions"].double()[:, None] * s["freqs"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    out = {}
    for n in "qk":
        x, w = s[n].float(), s[n + "_weight"]
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        out[n] = _rotate(x * r * w, cos, sin, rot, pairs).to(s[n].dtype)
        if case["train"]:
            back = _rotate(s["d" + n].float(), cos, -sin, rot, pairs)
            out["d%s_weight" % n] = (back * x * r).sum((0, 1))
            back = back * w
            out["d" + n] = (r * (back - x * r * r * (back * x).mean(-1, keepdim=True))).to(
                s[n].dtype)
    return out


# ---------------------------------------------------------- the library's calls --

def _own(s):
    from gated_delta_rule_98_b200 import kda
    case = s["case"]
    if case["op"] == "step":
        return {"y": kda.gated_scan_step(s["x"], s["z"], s["A"], s["h"]), "h": s["h"]}
    if case["op"] == "conv":
        dx, dw = kda.short_conv_swish_backward(s["x"], s["w"], s["dy"], cu_seqlens=s["cu"],
                                               num_seqs=case["N"], max_seqlen=s["max_seqlen"])
        return {"dx": dx, "dw": dw}
    if case["op"] == "qk":
        how = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                   interleaved=case["pairs"])
        q, k = kda.qk_norm_rope(s["q"], s["k"], s["positions"], s["freqs"], **how)
        out = {"q": q, "k": k}
        if case["train"]:
            out["dq"], out["dk"], out["dq_weight"], out["dk_weight"] = kda.qk_norm_rope_backward(
                s["q"], s["k"], s["dq"], s["dk"], s["positions"], s["freqs"], **how)
        return out
    how = dict(cu_seqlens=s["cu"], num_seqs=case["N"], max_seqlen=s["max_seqlen"])
    gate = (s["z"], s["A"]) if case["gate"] == "z" else (s["g"],)
    forward, backward = ((kda.gated_scan, kda.gated_scan_backward) if case["gate"] == "z" else
                         (kda.gated_scan_g, kda.gated_scan_g_backward))
    if not case["train"]:
        y, h_final = forward(s["x"], *gate, h0=s["h0"], **how)
        return {"y": y, "h_final": h_final}
    y, h_final, states = forward(s["x"], *gate, h0=s["h0"], save_states=True, **how)
    grads = backward(s["x"], *gate, states, s["dy"], h0=s["h0"], dh_final=s["dh"], **how)
    names = ("dx", "dz", "dA", "dh0") if case["gate"] == "z" else ("dx", "dg", "dh0")
    out = dict(zip(names, grads), y=y, h_final=h_final)
    if not case["state"]:
        del out["dh0"]
    return out


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    plain = {"step": _plain_step, "scan": _plain_scan, "conv": _plain_conv, "qk": _plain_qk}
    return plain[op](state)


# -------------------------------------------------------------------- 64 bits --

def _exact_scan(s, case):
    x = s["x"].double()
    N, C, T = case["N"], case["C"], case["T"]
    by_z = case["gate"] == "z"
    if by_z:
        sig = torch.sigmoid(torch.exp(s["A"].double()) * s["z"].double())
        g = -5.0 * sig
        m = -torch.expm1(g)
    else:
        g = s["g"].double()
    a = torch.exp(g)
    b = m * x if by_z else x
    cu = s["cu"].tolist() if s["cu"] is not None else [n * (T // N) for n in range(N + 1)]
    zero = torch.zeros(N, C, dtype=torch.float64, device=x.device)
    h0 = s["h0"].double() if s["h0"] is not None else zero
    h_final = h0.clone()
    y, prev = torch.empty_like(x), torch.empty_like(x)
    for n in range(N):
        h = h0[n]
        for t in range(cu[n], cu[n + 1]):
            prev[t] = h
            h = torch.addcmul(b[t], a[t], h, out=y[t])
        h_final[n] = h
    out = {"y": y, "h_final": h_final}
    if not case["train"]:
        return out
    dh = s["dh"].double() if s["dh"] is not None else zero
    dy = s["dy"].double()
    lam, dh0 = torch.empty_like(x), dh.clone()
    for n in range(N):
        back = dh[n]
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            torch.add(dy[t], back, out=lam[t])
            back = a[t] * lam[t]
        dh0[n] = back
    if by_z:
        dz = lam * a * (prev - x) * (-5.0) * sig * (1.0 - sig) * torch.exp(s["A"].double())
        out.update(dx=lam * m, dz=dz, dA=(dz * s["z"].double()).sum(0))
    else:
        out.update(dx=lam, dg=lam * a * prev)
    if case["state"]:
        out["dh0"] = dh0
    return out


def _exact_conv(s, case):
    W, T = case["W"], case["T"]
    N = case["N"]
    cu = s["cu"].tolist() if s["cu"] is not None else [n * (T // N) for n in range(N + 1)]
    w = s["w"].double()
    dx = torch.empty(T, case["C"], dtype=torch.float64, device=w.device)
    dw = torch.zeros_like(w)
    for n in range(N):
        lo, hi = cu[n], cu[n + 1]
        if lo == hi:
            continue
        # the sequence with W - 1 zero rows before it; window i holds the inputs under tap i
        x = torch.nn.functional.pad(s["x"][lo:hi].double(), (0, 0, W - 1, 0))
        view = [x[i:i + hi - lo] for i in range(W)]
        u = sum(w[:, i] * view[i] for i in range(W))
        p = torch.sigmoid(u)
        du = s["dy"][lo:hi].double() * (p + u * p * (1.0 - p))
        dw += torch.stack([(du * view[i]).sum(0) for i in range(W)], 1)
        g = torch.nn.functional.pad(du, (0, 0, 0, W - 1))
        dx[lo:hi] = sum(w[:, W - 1 - j] * g[j:j + hi - lo] for j in range(W))
    return {"dx": dx, "dw": dw}


def _exact_qk(s, case):
    rot, d = case["rot"], case["d"]
    turn = s["positions"].double()[:, None] * s["freqs"].double()
    unit = torch.polar(torch.ones_like(turn), turn)[:, None]        # e^{i angle}
    half = torch.arange(rot // 2, device=turn.device)
    one, two = (2 * half, 2 * half + 1) if case["pairs"] else (half, half + rot // 2)
    out = {}

    def turned(v, by):
        c = torch.complex(v[..., one], v[..., two]) * by
        v = v.clone()
        v[..., one], v[..., two] = c.real, c.imag
        return v

    for n in "qk":
        x, w = s[n].double(), s[n + "_weight"].double()
        rms = (x.square().sum(-1, keepdim=True) / d + EPS).sqrt()
        unit_x = x / rms
        out[n] = turned(unit_x * w, unit)
        if case["train"]:
            back = turned(s["d" + n].double(), unit.conj())
            out["d%s_weight" % n] = (back * unit_x).sum((0, 1))
            g = back * w
            out["d" + n] = (g - unit_x * (g * unit_x).sum(-1, keepdim=True) / d) / rms
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "step":
        g = -5.0 * torch.sigmoid(torch.exp(s["A"].double()) * s["z"].double())
        h = torch.exp(g) * s["h"].double() - torch.expm1(g) * s["x"].double()
        return {"y": h, "h": h}
    return {"scan": _exact_scan, "conv": _exact_conv, "qk": _exact_qk}[case["op"]](s, case)
