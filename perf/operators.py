"""What is measured of the token operators: rotary positions and linear
attention with a decay for each head.

* rotary: q and k of a projection ``[B, N, heads, d]`` turned by their token's
  position and laid out as ``[B, H, N, d]`` for the attention, and the
  gradients' way back;
* prompt: causal linear attention with a decay for each head over a whole
  sequence, ``S_t = decay S_{t-1} + k_t v_t^T``, ``out_t = scale q_t S_t``;
* train: its gradients;
* step: one token per sequence, the state updated in place.

Each case runs in a plain form of elementary torch operations in 32 bits, or,
with ``own``, through the library's public calls.
"""

import math

import numpy as np
import torch

own = False

CHUNK = 128  # tokens that the plain form takes together


def listed():
    return [
        # q and k of the 1.3B video DiT: three axes, pairs of neighbours, moved
        # into tiles of 2 x 4 x 8 tokens on the way
        dict(name="rotary_video", op="rotary", way="forward", B=1, H=12, F=21, R=30, C=52, d=128, dtype="bf16",
             rot=128, layout="interleaved", axes=3, tiled=True, scaling="plain", factor=1.0, far=0),
        # the gradients of the same step, fp32 from the attention's backward,
        # back to the projection's layout and type
        dict(name="rotary_video_grad", op="rotary", way="backward", B=1, H=12, F=21, R=30, C=52, d=128, dtype="bf16",
             rot=128, layout="interleaved", axes=3, tiled=True, scaling="plain", factor=1.0, far=0),
        # one token of each of 24 sequences, far behind the trained length,
        # half of each head turned
        dict(name="rotary_token", op="rotary", way="forward", B=24, H=12, F=1, R=1, C=1, d=128, dtype="bf16",
             rot=64, layout="half", axes=1, tiled=False, scaling="yarn", factor=16.0, far=500000),
        # a full-precision run of odd length, 42 of 64 channels turned
        dict(name="rotary_odd_f32", op="rotary", way="forward", B=2, H=6, F=1, R=1, C=4099, d=64, dtype="f32",
             rot=42, layout="half", axes=1, tiled=False, scaling="ntk", factor=4.0, far=100000),
        # the 1.3B DiT's clip as one causal sequence
        dict(name="prompt_video", op="prompt", B=1, H=12, N=32760, d=128, dtype="bf16", ragged=False, state=False),
        # the 14B DiT's clip: the largest
        dict(name="prompt_14b", op="prompt", B=1, H=40, N=75600, d=128, dtype="bf16", ragged=False, state=False),
        # a batch of short prompts of unequal lengths that go on from a state
        dict(name="prompt_ragged", op="prompt", B=6, H=8, N=1003, d=64, dtype="bf16", ragged=True, state=True),
        # a full-precision check run at the tiny workload's shape
        dict(name="prompt_f32", op="prompt", B=1, H=2, N=1024, d=64, dtype="f32", ragged=False, state=True),
        # fine-tuning at the 1.3B DiT's shape
        dict(name="train_video", op="train", B=1, H=12, N=32760, d=128, dtype="bf16", ragged=False, state=False),
        # a ragged batch in training, with gradients through the states
        dict(name="train_ragged", op="train", B=3, H=6, N=2029, d=128, dtype="bf16", ragged=True, state=True),
        # one token of one sequence: latency
        dict(name="step_one", op="step", B=1, H=12, N=1, d=128, dtype="bf16", ragged=False, state=True),
        # one token of each of 48 sequences: the states' traffic
        dict(name="step_batch", op="step", B=48, H=40, N=1, d=128, dtype="bf16", ragged=False, state=True),
    ]


def draw(rng):
    """One more case of the listed ones' ranges."""
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rotary", "rotary", "prompt", "prompt", "train", "step"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    H = rng.choice([1, 2, 3, 5, 6, 8, 12, 16, 24, 40])
    if op == "rotary":
        axes = rng.choice([1, 1, 3])
        grid = (spread(1, 21), spread(4, 45), spread(4, 80)) if axes == 3 else (1, 1, spread(1, 32768))
        B = 1 if axes == 3 else spread(1, 8)
        while B * H * grid[0] * grid[1] * grid[2] * d > 12 * 32760 * 128:
            grid = (max(1, grid[0] // 2), grid[1], grid[2]) if grid[0] > 1 else (1, max(1, grid[1] // 2), max(1, grid[2] * 2 // 3))
        layout = rng.choice(["half", "interleaved"])
        rot = d if axes == 3 else rng.choice([d, d // 2, 2 * rng.randint(2, d // 2)])
        return dict(op="rotary", way=rng.choice(["forward", "backward"]), B=B, H=H, F=grid[0], R=grid[1], C=grid[2], d=d,
                    dtype=dtype, rot=rot, layout=layout, axes=axes, tiled=axes == 3 and rng.random() < 0.5,
                    scaling=rng.choice(["plain", "linear", "ntk", "yarn"]), factor=rng.choice([2.0, 4.0, 16.0]),
                    far=0 if axes == 3 else rng.choice([0, spread(1, 1000000)]))
    if op == "step":
        return dict(op="step", B=spread(1, 48), H=H, N=1, d=d, dtype=dtype, ragged=False, state=True)
    most = 12 * 32760 if op == "train" else 40 * 75600
    if dtype == "f32":
        most //= 16
    B = rng.choice([1, 1, 2, 4, 7])
    N = spread(1, max(2, min(75600, most // (B * H))))
    return dict(op=op, B=B, H=H, N=N, d=d, dtype=dtype, ragged=B > 1 and rng.random() < 0.7, state=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _tile_order(F, R, C, tf, tr, tc):
    """Raster indices of a grid's tokens, walked tile by tile."""
    f, r, c = np.meshgrid(np.arange(F), np.arange(R), np.arange(C), indexing="ij")
    keys = [x.ravel() for x in (c % tc, r % tr, f % tf, c // tc, r // tr, f // tf)]
    return np.lexsort(keys).astype(np.int32)


def _axis_pairs(case):
    """Pairs that turn with each axis: a third each of the head's, the rest with the first."""
    pairs = case["rot"] // 2
    if case["axes"] == 1:
        return [pairs]
    third = pairs // 3
    return [pairs - 2 * third, third, third]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    t = _dtype(case)
    B, H, d = case["B"], case["H"], case["d"]

    def normal(*shape, dtype=t):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    if case["op"] == "rotary":
        grid = (case["F"], case["R"], case["C"])
        N = grid[0] * grid[1] * grid[2]
        s = dict(case=case, positions=None, perm=None)
        if case["axes"] == 1:
            # where each sequence stands: a stretch of consecutive positions
            first = torch.randint(0, case["far"] + 1, (B, 1, 1), generator=g, device=dev, dtype=torch.int32)
            s["positions"] = first + torch.arange(N, device=dev, dtype=torch.int32)
        if case["tiled"]:
            s["perm"] = torch.from_numpy(_tile_order(*grid, 2, 4, 8)).to(dev)
        if case["way"] == "forward":
            # one projection's output holds q and k side by side
            qk = normal(B, N, 2, H, d)
            s["q"], s["k"] = qk[:, :, 0].transpose(1, 2), qk[:, :, 1].transpose(1, 2)
        else:
            s["q"], s["k"] = (normal(B, H, N, d, dtype=torch.float32) for _ in range(2))
        return s

    N = case["N"]
    s = dict(case=case, lens=None, state=None)
    s["q"], s["k"], s["v"] = (normal(B, H, N, d) for _ in range(3))
    # decays 1 - 2^-5 ... 1 - 2^-12 over the heads, as logarithms
    power = torch.linspace(5, 12, H, dtype=torch.float64) if H > 1 else torch.tensor([6.0], dtype=torch.float64)
    s["log_decay"] = torch.log1p(-torch.exp2(-power)).float().to(dev)
    if case["ragged"]:
        lens = torch.randint(0, N + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        lens[0] = N
        s["lens"] = lens
    if case["state"]:
        s["state"] = normal(B, H, d, d, dtype=torch.float32) * 4
    if case["op"] == "train":
        s["dout"] = normal(B, H, N, d)
        s["dstate"] = normal(B, H, d, d, dtype=torch.float32) if case["state"] else None
    return s


# ------------------------------------------------------------------ plain form


def _frequencies(case):
    """Radians per position for each pair, in 64 bits, and the amplitude of the turned pairs."""
    base, f = 10000.0, case["factor"]
    out = []
    for pairs in _axis_pairs(case):
        i = torch.arange(pairs, dtype=torch.float64)
        b = base * f ** (pairs / (pairs - 1.0)) if case["scaling"] == "ntk" and pairs > 1 else base
        w = b ** (-i / max(pairs, 1))
        if case["scaling"] == "linear":
            w = w / f
        if case["scaling"] == "yarn":
            # long waves are stretched by the factor, short ones stay, a ramp between
            turns = 4096.0 / (2 * math.pi)

            def at(beta):
                return 2 * pairs * math.log(turns / beta) / (2 * math.log(base))

            lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), 2 * pairs - 1)
            ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
            w = w / f * ramp + w * (1 - ramp)
        out.append(w)
    return torch.cat(out), (0.1 * math.log(f) + 1.0 if case["scaling"] == "yarn" else 1.0)


def _positions(state):
    """[B or 1, axes, N] positions of the tokens in raster order."""
    case = state["case"]
    if state["positions"] is not None:
        return state["positions"]
    t = torch.arange(case["F"] * case["R"] * case["C"], device="cuda")
    return torch.stack([t // (case["R"] * case["C"]), t // case["C"] % case["R"], t % case["C"]])[None]


def _angles(state):
    """[B or 1, 1, N, pairs] angles in 64 bits, and the amplitude."""
    case = state["case"]
    w, amplitude = _frequencies(case)
    axis = torch.repeat_interleave(torch.arange(case["axes"]), torch.tensor(_axis_pairs(case)))
    pos = _positions(state)[:, axis.to("cuda")].double()  # [B, pairs, N]
    return (pos.transpose(1, 2) * w.to("cuda"))[:, None], amplitude


def _turn(x, cos, sin, rot, layout):
    """The first `rot` channels of x turned pair by pair."""
    y, rest = x[..., :rot], x[..., rot:]
    if layout == "half":
        a, b = y[..., : rot // 2], y[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, rest], -1)


def _plain_rotary(state):
    case = state["case"]
    angle, amplitude = _angles(state)
    cos, sin = (torch.cos(angle) * amplitude).float(), (torch.sin(angle) * amplitude).float()
    perm = state["perm"].long() if state["perm"] is not None else None
    out = []
    for x in (state["q"], state["k"]):
        if case["way"] == "forward":
            y = _turn(x.float(), cos, sin, case["rot"], case["layout"]).to(x.dtype)
            out.append(y.contiguous() if perm is None else y[:, :, perm])
        else:
            if perm is not None:
                x = torch.empty_like(x).index_copy_(2, perm, x)
            y = _turn(x, cos, -sin, case["rot"], case["layout"])
            out.append(y.transpose(1, 2).to(_dtype(case)).contiguous().transpose(1, 2))
    return out


def _powers(log_decay, n):
    """decay^n per head for whole n >= 0: [H, *n.shape], formed in 64 bits."""
    g = log_decay.double().reshape(-1, *[1] * n.dim())
    return torch.exp(g * n.double()).float()


def _decayed(a, b, c, log_decay, s0, first):
    """out_t = sum_{s <= t} decay^(t-s) (a_t . b_s) c_s + decay^(t+first) a_t s0, chunk by chunk."""
    B, H, N, d = a.shape
    n = -(-N // CHUNK)
    pad = [0, 0, 0, n * CHUNK - N]
    a, b, c = (torch.nn.functional.pad(x, pad).view(B, H, n, CHUNK, d) for x in (a, b, c))
    i = torch.arange(CHUNK, device=a.device)
    gap = i[:, None] - i
    inside = _powers(log_decay, gap.clamp(min=0)) * (gap >= 0)
    out = (a @ b.transpose(-1, -2) * inside[:, None]) @ c
    if n > 1:
        added = (b * _powers(log_decay, CHUNK - 1 - i)[:, None, :, None]).transpose(-1, -2) @ c
        j = torch.arange(n, device=a.device)
        gap = j[:, None] - 1 - j
        over = _powers(log_decay, gap.clamp(min=0) * CHUNK) * (gap >= 0)
        start = (over @ added.view(B, H, n, d * d)).view(B, H, n, d, d)
        out = out + (a * _powers(log_decay, i + 1)[:, None, :, None]) @ start
    out = out.view(B, H, n * CHUNK, d)[:, :, :N]
    if s0 is not None:
        t = torch.arange(N, device=a.device)
        out = out + (a.view(B, H, n * CHUNK, d)[:, :, :N] @ s0) * _powers(log_decay, t + first)[..., None]
    return out


def _lens(state):
    """[B, 1, 1, 1] lengths."""
    case = state["case"]
    lens = state["lens"] if state["lens"] is not None else torch.full((case["B"],), case["N"], device="cuda")
    return lens.long().view(-1, 1, 1, 1)


def _after(b, c, log_decay, s0, lens, first):
    """decay^len s0 + sum_s decay^(first + (len-1-s, or s)) b_s c_s^T over a sequence's tokens."""
    N = b.shape[2]
    s = torch.arange(N, device=b.device)
    left = (s + 1 if first else lens.view(-1, 1) - 1 - s).clamp(min=0).expand(b.shape[0], N)
    w = _powers(log_decay, left).transpose(0, 1)  # [B, H, N]
    out = (b * w[..., None]).transpose(-1, -2) @ c
    return out if s0 is None else out + s0 * _powers(log_decay, lens.view(-1)).transpose(0, 1)[..., None, None]


def _plain_prompt(state):
    case, scale = state["case"], state["case"]["d"] ** -0.5
    lens = _lens(state)
    real = torch.arange(case["N"], device="cuda").view(1, 1, -1, 1) < lens
    q, k, v = (torch.where(real, state[x].float(), 0.0) for x in "qkv")
    out = _decayed(q, k, v, state["log_decay"], state["state"], 1) * scale
    return out.to(_dtype(case)), _after(k, v, state["log_decay"], state["state"], lens, 0)


def _plain_train(state):
    case, scale = state["case"], state["case"]["d"] ** -0.5
    lens, g, s0, ds = _lens(state), state["log_decay"], state["state"], state["dstate"]
    t = torch.arange(case["N"], device="cuda").view(1, 1, -1, 1)
    real = t < lens
    q, k, v, do = (torch.where(real, state[x].float(), 0.0) for x in ("q", "k", "v", "dout"))
    q = q * scale

    def back(x):  # each sequence's own tokens from its last to its first
        return torch.where(real, x.gather(2, (lens - 1 - t).clamp(min=0).expand(x.shape)), 0.0)

    def turned(x):
        return None if x is None else x.transpose(-1, -2)

    dq = _decayed(do, v, k, g, turned(s0), 1) * scale
    qb, kb, vb, dob = back(q), back(k), back(v), back(do)
    dv = back(_decayed(kb, qb, dob, g, ds, 0))
    dk = back(_decayed(vb, dob, qb, g, turned(ds), 0))
    out = [x.to(_dtype(case)) for x in (torch.where(real, dq, 0.0), dk, dv)]
    return out + ([_after(q, do, g, ds, lens, 1)] if s0 is not None else [])


def _plain_step(state):
    case = state["case"]
    q, k, v = (state[x].float() for x in "qkv")
    s = state["state"]
    s.mul_(_powers(state["log_decay"], torch.ones(1, device="cuda"))[..., None])
    s.add_(k.transpose(-1, -2) * v)
    out = (q * case["d"] ** -0.5).transpose(-1, -2) * s
    return out.sum(-2, keepdim=True).to(_dtype(case)), s


# ------------------------------------------------------------------ the library's calls


def _own(state):
    from block_sparse_linear_mean_b200 import sla
    case = state["case"]
    op = case["op"]
    if op == "rotary":
        N = case["F"] * case["R"] * case["C"]
        if "handle" not in state:  # a model's constants
            state["handle"] = (sla.token_params(case["B"], case["H"], N, case["d"], _dtype(case)),
                               sla.rotary(case["rot"], layout=case["layout"], axis_pairs=_axis_pairs(case),
                                          grid=(case["F"], case["R"], case["C"]) if case["axes"] == 3 else None,
                                          scaling=case["scaling"], factor=case["factor"], base=10000.0,
                                          trained_length=4096))
        p, r = state["handle"]
        if case["way"] == "forward":
            return sla.apply_rotary(p, r, state["q"], state["k"], positions=state["positions"], perm=state["perm"])
        return sla.apply_rotary_backward(p, r, state["q"], state["k"], positions=state["positions"], perm=state["perm"])
    if "handle" not in state:  # constants and scratch that a program keeps
        p = sla.token_params(case["B"], case["H"], case["N"], case["d"], _dtype(case))
        state["handle"] = (p, sla.workspace(p, sla.SLA_OP_DECAY_BACKWARD if op == "train" else sla.SLA_OP_DECAY, "cuda")
                           if op != "step" else None)
    p, ws = state["handle"]
    if op == "prompt":
        f = sla.decay_attention(p, state["q"], state["k"], state["v"], state["log_decay"], lens=state["lens"],
                                state=state["state"], ws=ws)
        return f["out"], f["state"]
    if op == "train":
        g = sla.decay_attention_backward(p, state["q"], state["k"], state["v"], state["log_decay"], state["dout"],
                                         lens=state["lens"], state=state["state"], dstate=state["dstate"], ws=ws)
        return [g["dq"], g["dk"], g["dv"]] + ([g["dstate"]] if state["state"] is not None else [])
    out = sla.decay_attention_step(p, state["q"], state["k"], state["v"], state["log_decay"], state["state"])
    return out, state["state"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "rotary":
        return _plain_rotary(state)
    if op == "prompt":
        return _plain_prompt(state)
    if op == "train":
        return _plain_train(state)
    return _plain_step(state)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    B, H, d = case["B"], case["H"], case["d"]
    if case["op"] == "rotary":
        N = case["F"] * case["R"] * case["C"]
        values = 2 * B * H * N * d
        read = 4 if case["way"] == "backward" else e
        return dict(bytes=values * (read + e) + (4 * B * N if case["axes"] == 1 else 0) + (4 * N if case["tiled"] else 0),
                    flops=3 * values * case["rot"] / d)
    tokens, states = B * H * case["N"], 4 * B * H * d * d
    if case["op"] == "train":
        # S and its use, R and its two uses: five products of d x d per token
        return dict(bytes=7 * e * tokens * d + (3 * states if case["state"] else 0), flops=10 * tokens * d * d)
    return dict(bytes=4 * e * tokens * d + states * (2 if case["state"] else 1), flops=(4 if case["op"] == "prompt" else 5) * tokens * d * d)


# ------------------------------------------------------------------ the definition in 64 bits


def _exact_rotary(state):
    case = state["case"]
    B, H, d, rot = case["B"], case["H"], case["d"], case["rot"]
    N = case["F"] * case["R"] * case["C"]
    sign = 1.0 if case["way"] == "forward" else -1.0
    n = np.arange(N)
    if case["axes"] == 1:
        at = [state["positions"].cpu().numpy()[:, 0].astype(np.float64)]
    else:
        at = [x[None].astype(np.float64) for x in np.unravel_index(n, (case["F"], case["R"], case["C"]))]
    # one matrix of cosines and sines, axis by axis and pair by pair
    cos, sin = np.empty((at[0].shape[0], N, rot // 2)), np.empty((at[0].shape[0], N, rot // 2))
    first, f, amp = 0, case["factor"], 1.0
    for axis, pairs in enumerate(_axis_pairs(case)):
        for i in range(pairs):
            dim = 2 * pairs
            w = 10000.0 ** (-2.0 * i / dim)
            if case["scaling"] == "linear":
                w /= f
            elif case["scaling"] == "ntk" and dim > 2:
                w = (10000.0 * f ** (dim / (dim - 2.0))) ** (-2.0 * i / dim)
            elif case["scaling"] == "yarn":
                def corner(rotations):
                    return dim * math.log(4096.0 / (rotations * 2 * math.pi)) / (2 * math.log(10000.0))
                low, high = max(math.floor(corner(32.0)), 0), min(math.ceil(corner(1.0)), dim - 1)
                keep = 1.0 - min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
                w = (w / f) * (1.0 - keep) + w * keep
                amp = 0.1 * math.log(f) + 1.0
            cos[:, :, first + i] = np.cos(at[axis] * w)
            sin[:, :, first + i] = np.sin(at[axis] * w) * sign
        first += pairs
    cos, sin = (torch.from_numpy(x * amp).to("cuda")[:, None] for x in (cos, sin))
    order = np.arange(N) if state["perm"] is None else state["perm"].cpu().numpy()
    order = torch.from_numpy(order.astype(np.int64)).to("cuda")
    if case["layout"] == "half":
        one, two = torch.arange(rot // 2, device="cuda"), torch.arange(rot // 2, rot, device="cuda")
    else:
        one, two = torch.arange(0, rot, 2, device="cuda"), torch.arange(1, rot, 2, device="cuda")
    out = []
    for x in (state["q"], state["k"]):
        x = x.double()
        if case["way"] == "backward":
            y = torch.empty_like(x)
            y[:, :, order] = x
            x = y
        y = x.clone()
        y[..., one] = x[..., one] * cos - x[..., two] * sin
        y[..., two] = x[..., one] * sin + x[..., two] * cos
        out.append(y[:, :, order] if case["way"] == "forward" else y)
    return out


def _exact_row(a, b, c, g, start):
    """One sequence of one head: out_t = sum_{s<=t} e^{g(t-s)} (a_t.b_s) c_s, plus e^{g(t+1)} a_t start."""
    n = a.shape[0]
    out = torch.zeros_like(a)
    step = 1024
    for t0 in range(0, n, step):
        t1 = min(n, t0 + step)
        t = torch.arange(t0, t1, device=a.device, dtype=torch.float64)
        gap = t[:, None] - t
        w = torch.where(gap >= 0, torch.exp(g * gap.clamp(min=0)), 0.0)
        out[t0:t1] = (a[t0:t1] @ b[t0:t1].T * w) @ c[t0:t1]
        if t0:
            s = torch.arange(t0, device=a.device, dtype=torch.float64)
            before = (b[:t0] * torch.exp(g * (t0 - s))[:, None]).T
            out[t0:t1] += torch.exp(g * (t - t0))[:, None] * ((a[t0:t1] @ before) @ c[:t0])
        if start is not None:
            out[t0:t1] += torch.exp(g * (t + 1))[:, None] * (a[t0:t1] @ start)
    return out


def _exact_decay(state):
    case = state["case"]
    B, H, N, d = case["B"], case["H"], case["N"], case["d"]
    scale = 1.0 / math.sqrt(d)
    lens = [N] * B if state["lens"] is None else state["lens"].tolist()
    g = state["log_decay"].double()
    train = case["op"] == "train"
    new = [torch.zeros(B, H, N, d, dtype=torch.float64, device="cuda") for _ in range(3 if train else 1)]
    after = torch.zeros(B, H, d, d, dtype=torch.float64, device="cuda")
    for i in range(B):
        for h in range(H):
            n = lens[i]
            q, k, v = (state[x][i, h, :n].double() for x in "qkv")
            s0 = None if state["state"] is None else state["state"][i, h].double()
            t = torch.arange(n, device="cuda", dtype=torch.float64)
            if not train:
                new[0][i, h, :n] = scale * _exact_row(q, k, v, g[h], s0)
                after[i, h] = (k * torch.exp(g[h] * (n - 1 - t))[:, None]).T @ v
                if s0 is not None:
                    after[i, h] += torch.exp(g[h] * n) * s0
                continue
            do = state["dout"][i, h, :n].double() * scale
            new[0][i, h, :n] = _exact_row(do, v, k, g[h], None if s0 is None else s0.T)
            # the sums over later tokens, by the same function on reversed rows; the
            # state's gradient comes in behind the last token
            kr, vr, qr, dor = (x.flip(0) for x in (k, v, q, do))
            dv, dk = _exact_row(kr, qr, dor, g[h], None).flip(0), _exact_row(vr, dor, qr, g[h], None).flip(0)
            after[i, h] = (q * torch.exp(g[h] * (t + 1))[:, None]).T @ do
            if state["dstate"] is not None:
                ds = state["dstate"][i, h].double()
                left = torch.exp(g[h] * (n - 1 - t))[:, None]
                dv, dk = dv + left * (k @ ds), dk + left * (v @ ds.T)
                after[i, h] += torch.exp(g[h] * n) * ds
            new[1][i, h, :n], new[2][i, h, :n] = dk, dv
    if train:
        return new + ([after] if state["state"] is not None else [])
    return new[0], after


def exact(case, seed):
    state = prepare(case, seed)
    return _exact_rotary(state) if case["op"] == "rotary" else _exact_decay(state)
