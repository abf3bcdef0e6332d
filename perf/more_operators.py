"""Workloads of the selective state space scan, of the short causal convolution before it and of the
slots their states live in.

The scan is the recurrent sibling of linear attention whose decay and write strength come from the
token: with delta_t = softplus(dt_t + bias) and a_t = e^(delta_t A), one number per (token, head),
    S_t = a_t S_{t-1} + delta_t B_t x_t^T,   y_t = S_t^T C_t + D x_t,
B and C shared by the H / G heads of a group.  The convolution gives every channel of x, B and C the
weighted sum of its last W inputs (and a SiLU).  The slots are pools of states and convolution windows:
finished sequences release theirs, the used ones are moved together, sequences fork.

Each case runs in a plain form (elementary torch operations in fp32, decays summed in fp64) or, with
`own` set, through the library.  `exact` gives the same outputs from the definitions, token by token
in fp64.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
PLAIN_CHUNK = 64

# The largest drawn calls: elements of a convolution, products B x^T of a scan and of its gradients,
# elements of a batch's states, elements of a pool.
MOST_CONV = 16384 * 4352
MOST_FWD = 65536 * 32 * 128 * 64
MOST_BWD = 4 * 4096 * 32 * 128 * 64
MOST_STATES = 256 * 32 * 128 * 64
MOST_POOL = 1024 * 32 * 128 * 64


# ------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # A few short prompts in fp32, channels and lengths that divide nothing: launch latency counts.
        dict(name="conv_f32_packed_odd", op="conv", dtype="f32", lens="1 2 130 0 67", C=332, W=3, packed=True,
             state=True, bias=True, silu=False),
        # x, B and C of a batch of prompts, 64 heads of 64 channels and one group of 128.
        dict(name="conv_bf16_4x4096x4352", op="conv", dtype="bf16", lens="4096 4096 4096 4096", C=4352, W=4,
             packed=False, state=False, bias=True, silu=True),
        # Gradients of a packed training batch of short documents.
        dict(name="conv_bwd_bf16_packed_ragged", op="conv_bwd", dtype="bf16", lens="517 33 1029 200 1", C=2304,
             W=4, packed=True, state=False, bias=True, silu=True),
        # Gradients of an ordinary training batch.
        dict(name="conv_bwd_bf16_4x4096x4352", op="conv_bwd", dtype="bf16", lens="4096 4096 4096 4096", C=4352,
             W=4, packed=False, state=False, bias=True, silu=True),
        # A packed batch of ragged prompts, one of a single token and one empty, in groups of four heads.
        dict(name="ssm_bf16_packed_ragged", op="ssm", dtype="bf16", lens="1 700 0 4099 63 2050 1333 8209", H=8,
             G=2, dk=128, dv=64, packed=True, state=True, skip=True),
        # One long prompt: the parallelism has to come from within the sequence.
        dict(name="ssm_bf16_1x65536x32", op="ssm", dtype="bf16", lens="65536", H=32, G=1, dk=128, dv=64,
             packed=False, state=True, skip=True),
        # Gradients of a small fp32 batch, every head with its own B and C: a model's first experiments.
        dict(name="ssm_bwd_f32_3x250x4_d64", op="ssm_bwd", dtype="f32", lens="250 250 250", H=4, G=4, dk=64,
             dv=64, packed=False, state=True, skip=False),
        # Gradients of an ordinary training batch, one group.
        dict(name="ssm_bwd_bf16_4x4096x32", op="ssm_bwd", dtype="bf16", lens="4096 4096 4096 4096", H=32, G=1,
             dk=128, dv=64, packed=False, state=False, skip=True),
        # One sequence's decode step, convolution and scan: launch latency counts.
        dict(name="step_bf16_1x32", op="step", dtype="bf16", N=1, H=32, G=1, dk=128, dv=64, W=4, slots=8),
        # A full decode batch.
        dict(name="step_bf16_256x32", op="step", dtype="bf16", N=256, H=32, G=1, dk=128, dv=64, W=4,
             slots=300),
        # One request ends, one is moved into its slot, one forks: launch latency counts.
        dict(name="slots_16x8_d64", op="slots", slots=16, used=11, freed=1, moves=1, forks=1, H=8, G=1, dk=64,
             dv=64, W=4),
        # A busy server's pool: a quarter of the requests ends, the rest is moved together, beams fork.
        dict(name="slots_1024x32", op="slots", slots=1024, used=600, freed=200, moves=150, forks=256, H=32,
             G=1, dk=128, dv=64, W=4),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_lens(rng, most):
    total = _log_int(rng, 1, min(65536, most))
    n = _log_int(rng, 1, min(16, total))
    packed = rng.random() < 0.5
    if packed:
        cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    else:
        lens = [total // n] * n
    return dict(lens=" ".join(map(str, lens)), packed=packed)


def draw(rng):
    op = rng.choice(["conv", "conv_bwd", "ssm", "ssm", "ssm_bwd", "ssm_bwd", "step", "slots"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("conv", "conv_bwd"):
        C, W = 4 * _log_int(rng, 1, 1088), rng.choice([2, 3, 4])
        return dict(op=op, dtype=dtype, C=C, W=W, state=rng.random() < 0.5, bias=rng.random() < 0.7,
                    silu=rng.random() < 0.7, **_draw_lens(rng, MOST_CONV // C // (2 if dtype == "f32" else 1)))
    G = _log_int(rng, 1, 8)
    H = G * _log_int(rng, 1, 32 // G)
    dk, dv = rng.choice([64, 128]), rng.choice([64, 128])
    sizes = dict(H=H, G=G, dk=dk, dv=dv)
    if op in ("ssm", "ssm_bwd"):
        most = (MOST_FWD if op == "ssm" else MOST_BWD) // (H * dk * dv)
        return dict(op=op, dtype=dtype, state=rng.random() < 0.7, skip=rng.random() < 0.7, **sizes,
                    **_draw_lens(rng, max(1, most // (4 if dtype == "f32" else 1))))
    W = rng.choice([2, 3, 4])
    if op == "step":
        N = _log_int(rng, 1, max(1, min(256, MOST_STATES // (H * dk * dv))))
        return dict(op=op, dtype=dtype, N=N, W=W, slots=N + _log_int(rng, 1, 64), **sizes)
    slots = _log_int(rng, 8, max(8, min(1024, MOST_POOL // (H * dk * dv))))
    used = rng.randint(2, slots // 2)
    freed = rng.randint(1, used - 1)
    left = used - freed                       # in use when the pool is moved together
    forks = rng.randint(1, max(1, slots // 4))
    moves = rng.randint(0, min(left, slots - left - forks))
    return dict(op=op, slots=slots, used=used, freed=freed, moves=moves, forks=forks, W=W, **sizes)


def _lens(case):
    return [int(n) for n in case["lens"].split()]


def _channels(case):
    return case["H"] * case["dv"] + 2 * case["G"] * case["dk"]


def work(case):
    op = case["op"]
    es = 4 if case.get("dtype") == "f32" else 2
    if op in ("conv", "conv_bwd"):
        tok, C, W, N = sum(_lens(case)), case["C"], case["W"], len(_lens(case))
        window = N * (W - 1) * C * es * (2 if case["state"] else 1)       # the last inputs out, earlier ones in
        if op == "conv":
            return {"bytes": tok * C * 2 * es + window + C * (W + 1) * 4, "flops": tok * C * (2 * W + 4)}
        return {"bytes": tok * C * 3 * es + window + C * (W + 1) * 8, "flops": tok * C * (6 * W + 10)}
    H, G, dk, dv = case["H"], case["G"], case["dk"], case["dv"]
    if op in ("ssm", "ssm_bwd"):
        tok = sum(_lens(case))
        states = len(_lens(case)) * H * dk * dv * 4
        if op == "ssm":
            return {"bytes": tok * (2 * H * dv + 2 * G * dk + H) * es + states * (2 if case["state"] else 1),
                    "flops": tok * H * (4 * dk * dv + 2 * dv)}
        # x, dy, B, C, dt in; dx, dB, dC, ddt out; initial state and its final state's gradient in, the
        # initial state's gradient out
        return {"bytes": tok * (3 * H * dv + 4 * G * dk + 2 * H) * es + (states * 3 if case["state"] else 0),
                "flops": tok * H * (12 * dk * dv + 6 * dv)}
    row = _channels(case)
    if op == "step":
        units = case["N"] * H
        return {"bytes": units * 2 * dk * dv * 4 + case["N"] * es * (row * 2 + row * 2 * (case["W"] - 1) + row
                                                                     + H * (dv + 1)) + row * case["W"] * 4,
                "flops": units * 5 * dk * dv + case["N"] * row * (2 * case["W"] + 4)}
    slot = H * dk * dv * 4 + (case["W"] - 1) * row * 2
    return {"bytes": 2 * (case["moves"] + case["forks"]) * slot + 16 * case["slots"], "flops": 0}


# ------------------------------------------------------------------------------------ the inputs

def _gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def _normal(shape, gen, std=1.0, dtype=torch.float32):
    """Normal values, made in slices so that fp32 copies stay small."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 26):
        n = min(1 << 26, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=gen, device=DEV) * std
    return out


def _conv_weights(C, W, gen):
    return _normal((C, W), gen, 1.0 / math.sqrt(W)), _normal((C,), gen, 0.1)


def _scan_weights(H, gen):
    """A in (-16, -1), and biases that put softplus(bias) between 1e-3 and 0.1, as models start."""
    A = -(1.0 + 15.0 * torch.rand((H,), generator=gen, device=DEV))
    step = torch.exp(math.log(1e-3) + torch.rand((H,), generator=gen, device=DEV) * math.log(100.0))
    return A, torch.log(torch.expm1(step)), _normal((H,), gen)


def _split(s, row):
    """x, B and C as the convolution leaves them: parts of one row."""
    H, G, dk, dv = (s["case"][k] for k in ("H", "G", "dk", "dv"))
    lead = row.shape[:-1]
    s["x"] = row[..., :H * dv].view(lead + (H, dv))
    s["B"] = row[..., H * dv:H * dv + G * dk].view(lead + (G, dk))
    s["C"] = row[..., H * dv + G * dk:].view(lead + (G, dk))


def prepare(case, seed):
    gen = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("conv", "conv_bwd", "ssm", "ssm_bwd"):
        lens, dt = _lens(case), DTYPES[case["dtype"]]
        N = len(lens)
        B, T = (1, sum(lens)) if case["packed"] else (N, lens[0])
        s["cu"] = None
        if case["packed"]:
            cuts = [0]
            for n in lens:
                cuts.append(cuts[-1] + n)
            s["cu"] = torch.tensor(cuts, dtype=torch.int32, device=DEV)
        if op in ("conv", "conv_bwd"):
            C, W = case["C"], case["W"]
            s["x"] = _normal((B, T, C), gen, dtype=dt)
            s["w"], bias = _conv_weights(C, W, gen)
            s["b"] = bias if case["bias"] else None
            s["h0"] = _normal((N, W - 1, C), gen, dtype=dt) if case["state"] else None
            if op == "conv_bwd":
                s["dy"] = _normal((B, T, C), gen, dtype=dt)
                s["dhT"] = _normal((N, W - 1, C), gen, dtype=dt) if case["state"] else None
            return s
        H, dk, dv = case["H"], case["dk"], case["dv"]
        _split(s, torch.nn.functional.silu(_normal((B, T, _channels(case)), gen, dtype=dt)))
        s["dt"] = _normal((B, T, H), gen, dtype=dt)
        s["A"], s["bias"], D = _scan_weights(H, gen)
        s["D"] = D if case["skip"] else None
        s["h0"] = _normal((N, H, dk, dv), gen, 0.1) if case["state"] else None
        if op == "ssm_bwd":
            s["dy"] = _normal((B, T, H, dv), gen, dtype=dt)
            s["dhT"] = _normal((N, H, dk, dv), gen, 0.1) if case["state"] else None
        return s
    H, dk, dv, W, row = case["H"], case["dk"], case["dv"], case["W"], _channels(case)
    n_slots = case["slots"]
    if op == "step":
        N, dt = case["N"], DTYPES[case["dtype"]]
        s["in"] = _normal((N, row), gen, dtype=dt)
        s["w"], s["b"] = _conv_weights(row, W, gen)
        _split(s, torch.nn.functional.silu(_normal((N, row), gen, dtype=dt)))
        s["dt"] = _normal((N, H), gen, dtype=dt)
        s["A"], s["bias"], s["D"] = _scan_weights(H, gen)
        s["windows"] = _normal((n_slots, W - 1, row), gen, dtype=dt)
        s["states"] = _normal((n_slots, H, dk, dv), gen)
        s["slots"] = torch.randperm(n_slots, generator=gen, device=DEV)[:N].to(torch.int32)
        return s
    # A pool after some time of service: `left` sequences stay, `moves` of them in high slots.
    used, freed, moves, forks = case["used"], case["freed"], case["moves"], case["forks"]
    left = used - freed
    s["pool"] = [_normal((n_slots, H, dk, dv), gen),
                 _normal((n_slots, W - 1, row), gen, dtype=torch.bfloat16)]
    low = torch.randperm(left, generator=gen, device=DEV)
    high = left + forks + torch.randperm(n_slots - left - forks, generator=gen, device=DEV)[:moves]
    stay = torch.cat([low[:left - moves], high])
    stay = stay[torch.randperm(left, generator=gen, device=DEV)]
    taken = torch.zeros(n_slots, dtype=torch.bool, device=DEV)
    taken[stay] = True
    free = torch.nonzero(~taken)[:, 0]
    gone = free[torch.randperm(free.numel(), generator=gen, device=DEV)[:freed]]
    s["refs0"] = torch.zeros(n_slots, dtype=torch.int32, device=DEV)
    s["refs0"][stay] = 1 + (torch.rand(left, generator=gen, device=DEV) < 0.2).to(torch.int32)
    s["refs0"][gone] = 1
    s["finished"] = gone.to(torch.int32)
    s["table0"] = stay.to(torch.int32)
    s["parents"] = torch.randint(0, left, (forks,), generator=gen, device=DEV)
    s["refs"], s["table"] = s["refs0"].clone(), s["table0"].clone()
    return s


# ------------------------------------------------------------------------------------ one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from gated_delta_rule_60_amd import kda as K
    c = s["case"]
    op = c["op"]
    if op == "conv":
        return K.kda_conv_fwd(s["x"], s["w"], s["b"], initial_state=s["h0"], cu_seqlens=s["cu"],
                              silu=c["silu"], output_final_state=True)
    if op == "conv_bwd":
        out = K.kda_conv_bwd(s["x"], s["w"], s["dy"], s["b"], initial_state=s["h0"], d_final_state=s["dhT"],
                             cu_seqlens=s["cu"], silu=c["silu"])
        return [g for g in out if g is not None]
    if op == "ssm":
        return K.kda_ssm_chunk_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], dt_bias=s["bias"],
                                   initial_state=s["h0"], cu_seqlens=s["cu"])
    if op == "ssm_bwd":
        out = K.kda_ssm_chunk_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["dy"], D=s["D"],
                                  dt_bias=s["bias"], initial_state=s["h0"], d_final_state=s["dhT"],
                                  cu_seqlens=s["cu"])
        return [g for g in out if g is not None]
    if op == "step":
        u = K.kda_conv_step(s["in"], s["w"], s["windows"], s["b"], slots=s["slots"])
        y = K.kda_ssm_decode_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["states"], D=s["D"],
                                  dt_bias=s["bias"], slots=s["slots"])
        return u, y, s["windows"], s["states"]
    s["refs"].copy_(s["refs0"])
    s["table"].copy_(s["table0"])
    K.kda_slots_release(s["refs"], s["finished"])
    used = K.kda_slots_compact(s["pool"], s["refs"], s["table"])
    children = K.kda_slots_fork(s["pool"], s["refs"], s["table"][s["parents"]])
    return [*s["pool"], s["refs"], s["table"], used, children]


def _run_plain(s):
    op = s["case"]["op"]
    return dict(conv=_plain_conv, conv_bwd=_plain_conv_bwd, ssm=_plain_ssm, ssm_bwd=_plain_ssm_bwd,
                step=_plain_step, slots=_plain_slots)[op](s)


def _runs(s):
    """(sequence numbers, their tokens) of the batch: all of them at once where they have one length."""
    x = s["x"]
    if s["cu"] is None:
        return [(slice(0, x.shape[0]), slice(0, x.shape[0]), slice(None))]
    out, at = [], 0
    for n, length in enumerate(_lens(s["case"])):
        out.append((slice(n, n + 1), slice(0, 1), slice(at, at + length)))
        at += length
    return out


# ---- convolution

def _silu(u):
    return u / (1.0 + torch.exp(-u))


def _with_window(s, n, b, t):
    """Inputs of a run in fp32, the W - 1 before it in front."""
    c, x = s["case"], s["x"][b, t].float()
    h0 = x.new_zeros((x.shape[0], c["W"] - 1, c["C"])) if s["h0"] is None else s["h0"][n].float()
    return torch.cat([h0, x], 1)


def _taps(s, xp):
    W = s["case"]["W"]
    T = xp.shape[1] - (W - 1)
    u = 0.0 if s["b"] is None else s["b"]
    for i in range(W):
        u = u + s["w"][:, i] * xp[:, i:i + T]
    return u


def _plain_conv(s):
    c = s["case"]
    y = torch.empty_like(s["x"])
    hT = torch.empty((len(_lens(c)), c["W"] - 1, c["C"]), dtype=y.dtype, device=DEV)
    for n, b, t in _runs(s):
        xp = _with_window(s, n, b, t)
        u = _taps(s, xp)
        y[b, t] = (_silu(u) if c["silu"] else u).to(y.dtype)
        hT[n] = xp[:, xp.shape[1] - (c["W"] - 1):].to(y.dtype)
    return y, hT


def _plain_conv_bwd(s):
    c, W = s["case"], s["case"]["W"]
    dx = torch.empty_like(s["x"])
    dw, db = torch.zeros_like(s["w"]), torch.zeros((c["C"],), device=DEV)
    dh0 = None if s["h0"] is None else torch.empty_like(s["h0"])
    for n, b, t in _runs(s):
        xp = _with_window(s, n, b, t)
        T = xp.shape[1] - (W - 1)
        du = s["dy"][b, t].float()
        if c["silu"]:
            u = _taps(s, xp)
            sig = 1.0 / (1.0 + torch.exp(-u))
            du = du * (sig * (1.0 + u * (1.0 - sig)))
        dxp = torch.zeros_like(xp)
        if s["dhT"] is not None:
            dxp[:, T:] += s["dhT"][n].float()
        for i in range(W):
            dxp[:, i:i + T] += s["w"][:, i] * du
            dw[:, i] += (du * xp[:, i:i + T]).sum((0, 1))
        db += du.sum((0, 1))
        dx[b, t] = dxp[:, W - 1:].to(dx.dtype)
        if dh0 is not None:
            dh0[n] = dxp[:, :W - 1].to(dh0.dtype)
    out = [dx, dw]
    if s["b"] is not None:
        out.append(db)
    if dh0 is not None:
        out.append(dh0)
    return out


# ---- scan

def _softplus(x):
    return torch.where(x > 30.0, x, torch.log1p(torch.exp(x.clamp(max=30.0))))


def _pieces(x, pad):
    """[N, T, H, ...] -> fp32 or fp64 [N, H, chunks, PLAIN_CHUNK, ...], zeros behind the last token."""
    if pad:
        x = torch.cat([x, x.new_zeros((x.shape[0], pad) + tuple(x.shape[2:]))], 1)
    x = x.transpose(1, 2)
    return x.reshape(x.shape[:2] + (-1, PLAIN_CHUNK) + tuple(x.shape[3:]))


def _joined(x, T):
    """The other way round."""
    x = x.reshape(x.shape[:2] + (-1,) + tuple(x.shape[4:])).transpose(1, 2)
    return x[:, :T]


class _Run:
    """Chunks of one run of tokens: heads' B, C and x in fp32, write strengths, summed log-decays."""

    def __init__(self, s, b, t):
        c = s["case"]
        self.T = s["x"][b, t].shape[1]
        pad = -self.T % PLAIN_CHUNK
        self.pad = pad
        rep = c["H"] // c["G"]
        self.x = _pieces(s["x"][b, t].float(), pad)
        self.B, self.C = (_pieces(s[k][b, t].float().repeat_interleave(rep, 2), pad) for k in "BC")
        self.pre = s["dt"][b, t].double() + s["bias"].double()
        self.delta64 = _pieces(_softplus(self.pre), pad)
        self.delta = self.delta64.float()
        self.cum = (self.delta64 * s["A"].double()[:, None, None]).cumsum(-1)
        pos = torch.arange(PLAIN_CHUNK, device=DEV)
        self.seen = pos[:, None] >= pos[None, :]

    def decays(self):
        """From after token j to after token i of a chunk, zero where j comes later."""
        d = self.cum[..., :, None] - self.cum[..., None, :]
        return torch.where(self.seen, torch.exp(d.clamp(max=0.0)), 0.0).float()

    def into(self):
        return torch.exp(self.cum).float()[..., None]

    def out_of(self):
        return torch.exp(self.cum[..., -1:] - self.cum).float()[..., None]

    def over(self):
        return torch.exp(self.cum[..., -1]).float()[..., None, None]

    def starts(self, S):
        """States before every chunk, and the last one."""
        local = torch.matmul((self.B * (self.out_of() * self.delta[..., None])).transpose(-1, -2).contiguous(), self.x)
        over, out = self.over(), torch.empty_like(local)
        for i in range(local.shape[2]):
            out[:, :, i] = S
            S = S * over[:, :, i] + local[:, :, i]
        return out, S


def _zeros(s):
    c = s["case"]
    return torch.zeros((len(_lens(c)), c["H"], c["dk"], c["dv"]), device=DEV)


def _plain_ssm(s):
    y, hT = torch.empty_like(s["x"]), _zeros(s)
    for n, b, t in _runs(s):
        S = _zeros(s)[n] if s["h0"] is None else s["h0"][n]
        r = _Run(s, b, t)
        if r.T:
            starts, S = r.starts(S)
            o = torch.matmul(r.C * r.into(), starts)
            del starts
            w = torch.matmul(r.C, r.B.transpose(-1, -2).contiguous()) * r.decays() * r.delta[..., None, :]
            o += torch.matmul(w, r.x)
            del w
            if s["D"] is not None:
                o += s["D"][:, None, None, None] * r.x
            y[b, t] = _joined(o, r.T).to(y.dtype)
        hT[n] = S
    return y, hT


def _plain_ssm_bwd(s):
    c = s["case"]
    rep = c["H"] // c["G"]
    dx, ddt = torch.empty_like(s["x"]), torch.empty_like(s["dt"])
    dB, dC = torch.empty_like(s["B"]), torch.empty_like(s["C"])
    dA, dD, dbias = (torch.zeros((c["H"],), dtype=torch.float64, device=DEV) for _ in range(3))
    dh0 = None if s["h0"] is None else torch.empty_like(s["h0"])
    for n, b, t in _runs(s):
        X = _zeros(s)[n] if s["dhT"] is None else s["dhT"][n]      # gradient of the state after the chunk
        r = _Run(s, b, t)
        if r.T:
            dy = _pieces(s["dy"][b, t].float(), r.pad)
            starts, _ = r.starts(_zeros(s)[n] if s["h0"] is None else s["h0"][n])
            local = torch.matmul((r.C * r.into()).transpose(-1, -2).contiguous(), dy)
            ends, over = torch.empty_like(local), r.over()
            for i in reversed(range(local.shape[2])):
                ends[:, :, i] = X
                X = X * over[:, :, i] + local[:, :, i]
            del local
            decays = r.decays()
            cb = torch.matmul(r.C, r.B.transpose(-1, -2).contiguous())
            xy = torch.matmul(dy, r.x.transpose(-1, -2).contiguous())
            w = decays * r.delta[..., None, :] * xy
            into, out_of = r.into(), r.out_of() * r.delta[..., None]
            dC_state = torch.matmul(dy * into, starts.transpose(-1, -2).contiguous())
            dB_state = torch.matmul(r.x * out_of, ends.transpose(-1, -2).contiguous())
            gC = dC_state + torch.matmul(w, r.B)
            gB = dB_state + torch.matmul(w.transpose(-1, -2).contiguous(), r.C)
            u = torch.matmul((cb * decays).transpose(-1, -2).contiguous(), dy) + torch.matmul(r.B * r.out_of(), ends)
            dx_run = r.delta[..., None] * u
            if s["D"] is not None:
                dx_run += s["D"][:, None, None, None] * dy
            # the gradient of a token's log-decay: every way from a token before it (or the chunk's first
            # state) to an output from it on (or the chunk's last state)
            z = (w * cb).double()
            rows, cols = z.sum(-1), z.sum(-2)
            late = (dC_state * r.C).double().sum(-1)
            early = (dB_state * r.B).double().sum(-1)
            through = (starts * ends * over).double().sum((-1, -2))[..., None]
            dg = (rows - cols + late).flip(-1).cumsum(-1).flip(-1) + (early.cumsum(-1) - early) + through
            dg, r64 = _joined(dg, r.T), _joined(r.delta64, r.T)
            d_delta = _joined((u * r.x).double().sum(-1), r.T) + dg * s["A"].double()
            d_pre = d_delta / (1.0 + torch.exp(-r.pre))
            dA += (r64 * dg).sum((0, 1))
            dbias += d_pre.sum((0, 1))
            dD += (dy * r.x).double().sum((0, 2, 3, 4))
            dx[b, t], ddt[b, t] = _joined(dx_run, r.T).to(dx.dtype), d_pre.to(ddt.dtype)
            dB[b, t] = _joined(gB, r.T).unflatten(2, (-1, rep)).sum(3).to(dB.dtype)
            dC[b, t] = _joined(gC, r.T).unflatten(2, (-1, rep)).sum(3).to(dC.dtype)
        if dh0 is not None:
            dh0[n] = X
    return _gradients(s, dx, ddt, dA.float(), dB, dC, dD.float(), dbias.float(), dh0)


def _gradients(s, dx, ddt, dA, dB, dC, dD, dbias, dh0):
    out = [dx, ddt, dA, dB, dC]
    if s["D"] is not None:
        out.append(dD)
    out.append(dbias)
    if s["h0"] is not None:
        out.append(dh0)
    return out


# ---- decode step and slots

def _plain_step(s):
    c = s["case"]
    at, W, rep = s["slots"].long(), c["W"], c["H"] // c["G"]
    xp = torch.cat([s["windows"][at].float(), s["in"].float()[:, None]], 1)
    u = s["b"] + (s["w"].t() * xp).sum(1)
    s["windows"][at] = xp[:, 1:].to(s["windows"].dtype)
    delta = _softplus(s["dt"].double() + s["bias"].double())
    a, delta = torch.exp(delta * s["A"].double()).float(), delta.float()
    x = s["x"].float()
    B, C = (s[k].float().repeat_interleave(rep, 1) for k in "BC")
    S = s["states"][at] * a[..., None, None] + (delta[..., None] * B)[..., :, None] * x[..., None, :]
    s["states"][at] = S
    y = (S * C[..., :, None]).sum(-2) + s["D"][:, None] * x
    return _silu(u).to(s["in"].dtype), y.to(s["x"].dtype), s["windows"], s["states"]


def _plain_slots(s):
    c, refs, table, pool = s["case"], s["refs"], s["table"], s["pool"]
    n = c["slots"]
    refs.copy_(s["refs0"])
    table.copy_(s["table0"])
    refs.index_add_(0, s["finished"].long(), torch.full_like(s["finished"], -1))
    # the used slots behind the number of used ones go to the free slots before it, both in order
    taken = refs > 0
    used = taken.sum().to(torch.int32).reshape(1)
    place = torch.arange(n, device=DEV)
    src = torch.nonzero(taken & (place >= used))[:, 0]
    dst = torch.nonzero(~taken & (place < used))[:, 0]
    to = place.clone()
    to[src] = dst
    for plane in pool:
        plane[dst] = plane[src]
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(to[table.long()].to(torch.int32))
    children = torch.nonzero(refs == 0)[:c["forks"], 0]
    parents = table[s["parents"]].long()
    for plane in pool:
        plane[children] = plane[parents]
    refs[children] = 1
    return [*pool, refs, table, used, children.to(torch.int32)]


# ------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    op = case["op"]
    if op in ("ssm", "ssm_bwd"):
        steps = sum(_lens(case)) if case["packed"] else _lens(case)[0]
        if steps > (70000 if op == "ssm" else 16000):      # one token after the other
            return None
    s = prepare(case, seed)
    return dict(conv=_exact_conv, conv_bwd=_exact_conv_bwd, ssm=_exact_ssm, ssm_bwd=_exact_ssm_bwd,
                step=_exact_step, slots=_exact_slots)[op](s)


def _spans(s):
    """(states, batch rows, first token, one past the last) of runs that advance together."""
    if s["cu"] is None:
        N, T = s["x"].shape[:2]
        return [(slice(0, N), slice(0, N), 0, T)]
    cu = s["cu"].tolist()
    return [(slice(n, n + 1), slice(0, 1), cu[n], cu[n + 1]) for n in range(len(cu) - 1)]


def _input_at(s, n, b, lo, t):
    """The convolution's input at token t of a run that starts at token lo (t - lo may be negative)."""
    if t >= lo:
        return s["x"][b, t].double()
    back = s["case"]["W"] - 1 + (t - lo)
    return torch.zeros_like(s["x"][b, 0:1].double()[:, 0]) if s["h0"] is None else s["h0"][n, back].double()


def _exact_pre(s, n, b, lo, hi):
    """Weighted sums of a run [N, T, C], its inputs by taps alongside."""
    c = s["case"]
    W, T = c["W"], hi - lo
    taps = []
    for i in range(W):
        back = W - 1 - i
        head = [_input_at(s, n, b, lo, lo + k - back) for k in range(min(back, T))]
        tail = s["x"][b, lo:hi - len(head)].double() if back else s["x"][b, lo:hi].double()
        if back and T <= back:
            tail = tail[:, :0]
        taps.append(torch.cat([torch.stack(head, 1), tail], 1) if head else tail)
    u = sum(taps[i] * s["w"][:, i].double() for i in range(W))
    return (u if s["b"] is None else u + s["b"].double()), taps


def _exact_conv(s):
    c = s["case"]
    W = c["W"]
    y = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEV)
    hT = torch.zeros((len(_lens(c)), W - 1, c["C"]), dtype=torch.float64, device=DEV)
    for n, b, lo, hi in _spans(s):
        if hi > lo:
            u, _ = _exact_pre(s, n, b, lo, hi)
            y[b, lo:hi] = u * torch.sigmoid(u) if c["silu"] else u
        for i in range(W - 1):
            if s["x"].shape[1]:
                hT[n, i] = _input_at(s, n, b, lo, hi - (W - 1) + i)
            elif s["h0"] is not None:
                hT[n, i] = s["h0"][n, i].double()
    return y, hT


def _exact_conv_bwd(s):
    c = s["case"]
    W = c["W"]
    dx = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEV)
    dw = torch.zeros(s["w"].shape, dtype=torch.float64, device=DEV)
    db = torch.zeros((c["C"],), dtype=torch.float64, device=DEV)
    dh0 = None if s["h0"] is None else torch.zeros(s["h0"].shape, dtype=torch.float64, device=DEV)
    for n, b, lo, hi in _spans(s):
        T = hi - lo
        grad = torch.zeros((n.stop - n.start, T + W - 1, c["C"]), dtype=torch.float64, device=DEV)
        if T:
            u, taps = _exact_pre(s, n, b, lo, hi)
            du = s["dy"][b, lo:hi].double()
            if c["silu"]:
                sig = torch.sigmoid(u)
                du = du * (sig + u * sig * torch.sigmoid(-u))
            for i in range(W):
                grad[:, i:i + T] += du * s["w"][:, i].double()
                dw[:, i] += torch.einsum("ntc,ntc->c", du, taps[i])
            db += torch.einsum("ntc->c", du)
        if s["dhT"] is not None:
            grad[:, T:] += s["dhT"][n].double()
        dx[b, lo:hi] = grad[:, W - 1:]
        if dh0 is not None:
            dh0[n] = grad[:, :W - 1]
    out = [dx, dw]
    if s["b"] is not None:
        out.append(db)
    if dh0 is not None:
        out.append(dh0)
    return out


def _strengths(s):
    """delta and a of every token, and the derivative of delta."""
    pre = s["dt"].double() + s["bias"].double()
    delta = torch.clamp(pre, min=0) + torch.log1p(torch.exp(-pre.abs()))
    return delta, torch.exp(delta * s["A"].double()), torch.sigmoid(pre)


def _heads(s, x, b, t):
    """Token t's row of B or C for every head, fp64."""
    c = s["case"]
    return x[b, t].double().repeat_interleave(c["H"] // c["G"], 1)


def _exact_ssm(s):
    delta, a, _ = _strengths(s)
    y = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEV)
    hT = _zeros(s).double()
    D = None if s["D"] is None else s["D"].double()[:, None]
    for n, b, lo, hi in _spans(s):
        S = hT[n] if s["h0"] is None else s["h0"][n].double()
        for t in range(lo, hi):
            x = s["x"][b, t].double()
            S = torch.addcmul(S * a[b, t][..., None, None], _heads(s, s["B"], b, t)[..., None],
                              (x * delta[b, t][..., None])[..., None, :])
            o = torch.matmul(_heads(s, s["C"], b, t)[..., None, :], S)[..., 0, :]
            y[b, t] = o if D is None else o + D * x
        hT[n] = S
    return y, hT


def _exact_ssm_bwd(s):
    c = s["case"]
    rep = c["H"] // c["G"]
    delta, a, slope = _strengths(s)
    A = s["A"].double()
    dx, ddt, dB, dC = (torch.zeros(s[k].shape, dtype=torch.float64, device=DEV) for k in ("x", "dt", "B", "C"))
    dA, dD, dbias = (torch.zeros((c["H"],), dtype=torch.float64, device=DEV) for _ in range(3))
    dh0 = _zeros(s).double()
    D = None if s["D"] is None else s["D"].double()[:, None]

    def step(S, b, t):
        return torch.addcmul(S * a[b, t][..., None, None], _heads(s, s["B"], b, t)[..., None],
                             (s["x"][b, t].double() * delta[b, t][..., None])[..., None, :])

    for n, b, lo, hi in _spans(s):
        S = dh0[n] if s["h0"] is None else s["h0"][n].double()
        kept = []                                    # the state before every 64th token
        for t in range(lo, hi):
            if (t - lo) % 64 == 0:
                kept.append(S)
            S = step(S, b, t)
        G = _zeros(s)[n].double() if s["dhT"] is None else s["dhT"][n].double()
        for first in reversed(range(lo, hi, 64)):
            states = [kept.pop()]                    # before each token of the stretch, and after the last
            for t in range(first, min(first + 64, hi)):
                states.append(step(states[-1], b, t))
            for t in reversed(range(first, min(first + 64, hi))):
                x, dy = s["x"][b, t].double(), s["dy"][b, t].double()
                Bt, Ct = _heads(s, s["B"], b, t), _heads(s, s["C"], b, t)
                G = torch.addcmul(G, Ct[..., None], dy[..., None, :])
                dC[b, t] = torch.matmul(states[t - first + 1], dy[..., None])[..., 0].unflatten(1, (-1, rep)).sum(2)
                Gx = torch.matmul(G, x[..., None])[..., 0]
                dB[b, t] = (Gx * delta[b, t][..., None]).unflatten(1, (-1, rep)).sum(2)
                GB = torch.matmul(Bt[..., None, :], G)[..., 0, :]
                dx[b, t] = GB * delta[b, t][..., None] if D is None else GB * delta[b, t][..., None] + D * dy
                d_log = (G * states[t - first]).sum((-1, -2)) * a[b, t]
                d_pre = ((Gx * Bt).sum(-1) + d_log * A) * slope[b, t]
                ddt[b, t] = d_pre
                dA += (d_log * delta[b, t]).sum(0)
                dbias += d_pre.sum(0)
                dD += (dy * x).sum((0, 2))
                G = G * a[b, t][..., None, None]
        dh0[n] = G
    return _gradients(s, dx, ddt, dA, dB, dC, dD, dbias, dh0)


def _exact_step(s):
    c = s["case"]
    delta, a, _ = _strengths(s)
    win, states = s["windows"].double(), s["states"].double()
    out, y = [], []
    W = c["W"]
    for n, slot in enumerate(s["slots"].tolist()):
        new = s["in"][n].double()
        u = s["b"].double() + s["w"][:, W - 1].double() * new
        for i in range(W - 1):
            u = u + s["w"][:, i].double() * win[slot, i]
        out.append(u * torch.sigmoid(u))
        win[slot] = torch.cat([win[slot, 1:], new[None]])
        x = s["x"][n].double()
        b, cc = (s[k][n].double().repeat_interleave(c["H"] // c["G"], 0) for k in "BC")
        S = states[slot] * a[n][:, None, None] + torch.einsum("hc,he->hce", b, x) * delta[n][:, None, None]
        states[slot] = S
        y.append(torch.einsum("hce,hc->he", S, cc) + s["D"].double()[:, None] * x)
    return torch.stack(out), torch.stack(y), win, states


def _exact_slots(s):
    """Slot by slot on the host."""
    c = s["case"]
    refs, table = s["refs0"].tolist(), s["table0"].tolist()
    holds = list(range(c["slots"]))                  # whose contents a slot has
    for slot in s["finished"].tolist():
        refs[slot] -= 1
    used = sum(r > 0 for r in refs)
    to, low = {}, 0
    for slot in range(used, c["slots"]):
        if refs[slot] > 0:
            while refs[low] > 0:
                low += 1
            holds[low], refs[low], refs[slot], to[slot] = holds[slot], refs[slot], 0, low
    table = [to.get(slot, slot) for slot in table]
    children = []
    for parent in s["parents"].tolist():
        child = refs.index(0)
        holds[child], refs[child] = holds[table[parent]], 1
        children.append(child)
    holds = torch.tensor(holds, device=DEV)
    whole = [torch.tensor(v, dtype=torch.int32, device=DEV) for v in (refs, table, [used], children)]
    return [plane[holds].double() for plane in s["pool"]] + whole
