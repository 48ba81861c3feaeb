"""Cases of the rotary and decay-attention operators, with plain forms.

Five operators, named in a case by ``"op"``:

* ``rotary``       positions rotated into queries and keys
* ``rotary_back``  its gradient
* ``decay``        linear attention with a decay per head over whole sequences
* ``decay_step``   the same for one token per sequence, on a carried state
* ``decay_back``   its gradients

``run`` with ``own`` false computes them with elementary torch operations in
32 bits (angles of positions in 64), rounded once at the end; with ``own`` true
it makes the library calls a user makes.  ``exact`` evaluates the definitions
in 64 bits: the rotation as a complex product, the attention token by token.
"""

import math

import torch

own = False

INTERLEAVED, HALF = 0, 1
PLAIN, LINEAR, BASE, RAMP = 0, 1, 2, 3
RAMP_FAST, RAMP_SLOW = 32.0, 1.0


# --------------------------------------------------------------------- cases

def _rotary(name, op, B, L, Hq, Hk, D, bands, layout, scaling=PLAIN, factor=1.0, context=0, dtype="bf16", far=0,
            magnitude=1.0):
    return dict(name=name, op=op, B=B, L=L, Hq=Hq, Hk=Hk, D=D, band0=bands[0], band1=bands[1], band2=bands[2],
                layout=layout, scaling=scaling, factor=factor, context=context, dtype=dtype, far=far,
                magnitude=magnitude)


def _decay(name, op, B, L, H, D, state=False, ragged=False):
    return dict(name=name, op=op, B=B, L=L, H=H, D=D, state=state, ragged=ragged)


def listed():
    return [
        # one new token's queries and keys, three-axis positions: latency
        _rotary("rotary_token", "rotary", 1, 1, 12, 12, 128, (44, 42, 42), INTERLEAVED, far=1 << 12),
        # one streamed chunk of 2 x 24 x 32 latent patches
        _rotary("rotary_chunk", "rotary", 1, 1536, 12, 12, 128, (44, 42, 42), INTERLEAVED),
        # long-context prompts far from the origin: shared keys, half of the
        # head rotated, frequencies stretched by parts, an odd length
        _rotary("rotary_far", "rotary", 4, 8191, 24, 8, 128, (64, 0, 0), HALF, RAMP, 16.0, 32768, far=1 << 21,
                magnitude=1.2772588722239782),
        # gradients of whole training sequences
        _rotary("rotary_back_train", "rotary_back", 2, 30720, 12, 12, 128, (44, 42, 42), INTERLEAVED),
        # gradients kept in 32 bits, small heads, shared keys, odd length
        _rotary("rotary_back_f32", "rotary_back", 3, 1023, 24, 4, 64, (64, 0, 0), HALF, LINEAR, 4.0, dtype="f32"),
        # one streamed chunk with the state of the chunks before it
        _decay("decay_chunk", "decay", 1, 1536, 12, 128, state=True),
        # a padded batch of prompts of unequal lengths, one of them empty
        _decay("decay_ragged", "decay", 8, 2047, 24, 64, state=True, ragged=True),
        # whole training sequences
        _decay("decay_train", "decay", 2, 30720, 12, 128),
        # one token of one stream: latency
        _decay("decay_step_one", "decay_step", 1, 1, 12, 128, state=True),
        # one token of each sequence of a padded serving batch
        _decay("decay_step_batch", "decay_step", 256, 1, 24, 128, state=True, ragged=True),
        # gradients of one chunk with the state carried in and out
        _decay("decay_back_chunk", "decay_back", 1, 1536, 12, 128, state=True),
        # gradients of whole training sequences
        _decay("decay_back_train", "decay_back", 2, 30720, 12, 128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary_back", "decay", "decay", "decay_step", "decay_back", "decay_back"])
    if op in ("rotary", "rotary_back"):
        D = rng.choice([64, 80, 128, 128, 256])
        Hq = rng.randint(1, 24)
        Hk = rng.choice([h for h in range(1, Hq + 1) if Hq % h == 0])
        B = rng.randint(1, 4)
        room = (2 * 30720 * 24 * 128) // (B * (Hq + Hk) * D * 2)
        L = _log_int(rng, 1, min(30720, room))
        if rng.random() < 0.4:
            b1 = 2 * (D // 6)
            bands = (D - 2 * b1, b1, b1)
        else:
            bands = (rng.choice([D, D // 2, 2 * rng.randint(1, D // 2)]), 0, 0)
        scaling = rng.choice([PLAIN, LINEAR, BASE, RAMP]) if bands[0] > 2 and min(bands) != 2 else PLAIN
        return dict(_rotary("", op, B, L, Hq, Hk, D, bands, rng.choice([INTERLEAVED, HALF]), scaling,
                            1.0 if scaling == PLAIN else rng.choice([2.0, 4.0, 16.0, 40.0]),
                            rng.choice([4096, 32768]) if scaling == RAMP else 0, rng.choice(["bf16", "bf16", "f32"]),
                            rng.choice([0, 0, 1 << 12, 1 << 22]), rng.choice([1.0, 1.25])))
    D = rng.choice([64, 128])
    H = rng.randint(1, 24)
    if op == "decay_step":
        return _decay("", op, _log_int(rng, 1, 256), 1, H, D, state=True, ragged=rng.random() < 0.5)
    B = _log_int(rng, 1, 8)
    L = _log_int(rng, 1, min(30720, (2 * 30720 * 12 * 128) // (B * H * D)))
    return _decay("", op, B, L, H, D, state=rng.random() < 0.6, ragged=rng.random() < 0.4)


def work(case):
    c = case
    if c["op"] in ("rotary", "rotary_back"):
        es = 2 if c["dtype"] == "bf16" else 4
        rows = c["B"] * c["L"] * (c["Hq"] + c["Hk"])
        dims = c["band0"] + c["band1"] + c["band2"]
        pos = 8 * c["B"] * c["L"] * (3 if c["band1"] else 1)
        return {"bytes": 2 * rows * c["D"] * es + pos, "flops": 3 * rows * dims}
    B, L, H, D = c["B"], c["L"], c["H"], c["D"]
    # lengths of the ragged batches average half of L (sequences) or 7/8 (active tokens)
    live = B * L * H * (1.0 if not c["ragged"] else (0.5 if c["op"] != "decay_step" else 0.875))
    st = B * H * D * D * 4 if c["state"] else 0
    if c["op"] == "decay_back":
        return {"bytes": int(4 * live * D * 2 + 3 * B * L * H * D * 2 + 3 * st), "flops": int(10 * D * D * live)}
    return {"bytes": int(3 * live * D * 2 + B * L * H * D * 2 + 2 * st), "flops": int(4 * D * D * live)}


# -------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def prepare(case, seed):
    c, g = case, _gen(seed)
    B, L, D = c["B"], c["L"], c["D"]
    if c["op"] in ("rotary", "rotary_back"):
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s = dict(case=c, q=_randn(g, B, L, c["Hq"], D, dtype=dt), k=_randn(g, B, L, c["Hk"], D, dtype=dt))
        t = torch.arange(L, device="cuda", dtype=torch.int64)
        start = torch.randint(c["far"] + 1, (B, 1), generator=g, device="cuda", dtype=torch.int64)
        if c["band1"]:  # frame, row and column of a grid of 24 x 32 patches
            axes = [start + t // 768, (t // 32 % 24).expand(B, L), (t % 32).expand(B, L)]
        else:
            axes = [start + t]
        s["pos"] = torch.stack([a.expand(B, L) for a in axes]).contiguous()
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        if not own:
            s["freq"], s["axis"] = _frequencies(c)
        else:
            import streaming_attention_block_gb300 as sab

            s["plan"] = sab.rotary_plan(
                (c["band0"], c["band1"], c["band2"]) if c["band1"] else (c["band0"],),
                layout=c["layout"], base=10000.0, scaling=c["scaling"], factor=c["factor"],
                original_context=c["context"], ramp_fast=RAMP_FAST, ramp_slow=RAMP_SLOW, magnitude=c["magnitude"])
        return s
    H = c["H"]
    # decays from 0.7 to almost 1, and (last head of several) none at all
    ld = [math.log1p(-(2.0 ** -(1.7 + 9.0 * h / max(1, H - 1)))) for h in range(H)]
    if H > 1:
        ld[-1] = 0.0
    s = dict(case=c, ld=torch.tensor(ld, dtype=torch.float32, device="cuda"), scale=D ** -0.5)
    shape = (B, H, D) if c["op"] == "decay_step" else (B, L, H, D)
    for n in ("q", "k", "v"):
        s[n] = _randn(g, *shape)
    s["state"] = _randn(g, B, H, D, D, dtype=torch.float32) * 4 if c["state"] else None
    s["lens"] = None
    if c["ragged"]:
        if c["op"] == "decay_step":
            s["lens"] = (torch.rand(B, generator=g, device="cuda") < 0.875).to(torch.int32)
        else:
            s["lens"] = torch.randint(L + 1, (B,), generator=g, device="cuda").to(torch.int32)
            if B > 1:
                s["lens"][-1] = 0
    s["o"] = torch.empty_like(s["q"])
    s["state_out"] = torch.empty(B, H, D, D, dtype=torch.float32, device="cuda") if c["state"] else None
    if c["op"] == "decay_back":
        s["do"] = _randn(g, *shape)
        s["dstate"] = _randn(g, B, H, D, D, dtype=torch.float32) if c["state"] else None
        s["dq"], s["dk"], s["dv"] = (torch.empty_like(s["q"]) for _ in range(3))
    if own and c["op"] in ("decay", "decay_back"):
        import streaming_attention_block_gb300 as sab

        size = sab.decay_attention_workspace if c["op"] == "decay" else sab.decay_attention_backward_workspace
        s["ws"] = torch.empty(max(size(B, L, H, D), 256), dtype=torch.uint8, device="cuda")
    return s


# ----------------------------------------------------------- rotary, plainly

def _frequencies(c):
    """[dims / 2] radians per position and the position axis of each pair."""
    out, axis = [], []
    for a, n in enumerate((c["band0"], c["band1"], c["band2"])):
        if n == 0:
            continue
        base, s = 10000.0, c["factor"]
        if c["scaling"] == BASE:
            base = base * s ** (n / (n - 2.0))
        f = base ** (-2.0 * torch.arange(n // 2, dtype=torch.float64, device="cuda") / n)
        if c["scaling"] == LINEAR:
            f = f / s
        if c["scaling"] == RAMP:
            turns = c["context"] * f / (2.0 * math.pi)
            keep = ((turns - RAMP_SLOW) / (RAMP_FAST - RAMP_SLOW)).clamp(0.0, 1.0)
            f = f * (keep + (1.0 - keep) / s)
        out.append(f)
        axis += [a] * (n // 2)
    return torch.cat(out), torch.tensor(axis, device="cuda")


def _rotary_plain(s, back):
    c, freq = s["case"], s["freq"]
    ang = s["pos"][s["axis"]].permute(1, 2, 0).double() * freq  # [B, L, dims / 2]
    cos = (torch.cos(ang) * c["magnitude"]).float()[:, :, None, :]
    sin = (torch.sin(ang) * c["magnitude"]).float()[:, :, None, :]
    if back:
        sin = -sin
    n = 2 * freq.numel()

    def turn(x):
        y = x.float()
        if c["layout"] == INTERLEAVED:
            a, b = y[..., 0:n:2], y[..., 1:n:2]
            rot = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
        else:
            a, b = y[..., :n // 2], y[..., n // 2:n]
            rot = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
        return torch.cat([rot, y[..., n:]], dim=-1).to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def _rotary_exact(s, back):
    """The rotation of each pair as a product of complex numbers."""
    c = s["case"]
    cols = []
    for a, n in enumerate((c["band0"], c["band1"], c["band2"])):
        for i in range(n // 2):
            e = -2.0 * i / n
            f = 10000.0 ** e
            if c["scaling"] == LINEAR:
                f /= c["factor"]
            elif c["scaling"] == BASE:
                f *= c["factor"] ** (e * n / (n - 2.0))
            elif c["scaling"] == RAMP:
                turns = c["context"] * f / (2.0 * math.pi)
                w = min(1.0, max(0.0, (turns - RAMP_SLOW) / (RAMP_FAST - RAMP_SLOW)))
                f = (1.0 - w) * f / c["factor"] + w * f
            cols.append(s["pos"][a].double() * f)
    ang = torch.stack(cols, dim=-1)
    z = torch.polar(torch.full_like(ang, c["magnitude"]), -ang if back else ang)[:, :, None]
    m = len(cols)

    def turn(x):
        y = x.double()
        if c["layout"] == INTERLEAVED:
            w = torch.view_as_complex(y[..., :2 * m].unflatten(-1, (m, 2)).contiguous()) * z
            y[..., :2 * m] = torch.view_as_real(w).flatten(-2)
        else:
            w = torch.complex(y[..., :m], y[..., m:2 * m]) * z
            y[..., :m], y[..., m:2 * m] = w.real, w.imag
        return y

    return turn(s["q"].clone()), turn(s["k"].clone())


# ------------------------------------------------- decay attention, in chunks

CHUNK = 128


class _Chunks:
    """[B, H, n, CHUNK, D] views of padded 32-bit inputs and their decays."""

    def __init__(self, s):
        q = s["q"]
        self.B, self.L, self.H, self.D = q.shape
        self.n = (self.L + CHUNK - 1) // CHUNK
        pad = self.n * CHUNK
        lens = s["lens"] if s["lens"] is not None else torch.full((self.B,), self.L, device=q.device)
        self.live = torch.arange(pad, device=q.device) < lens[:, None]
        done = self.live.view(self.B, self.n, CHUNK).float().cumsum(-1)[:, None]  # live tokens so far in the chunk
        ld = s["ld"].view(1, -1, 1, 1)
        last = done[..., -1:]
        self.to_row = torch.exp(ld * done)           # start of the chunk .. row
        self.to_end = torch.exp(ld * (last - done))  # row .. end of the chunk
        self.whole = torch.exp(ld * last)[..., None]
        gap = done[..., :, None] - done[..., None, :]
        tri = torch.ones(CHUNK, CHUNK, device=q.device, dtype=torch.bool).tril()
        self.between = torch.where(tri, torch.exp(ld[..., None] * gap.clamp(min=0.0)), torch.zeros((), device=q.device))

    def split(self, x):
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, self.n * CHUNK - self.L))
        x = torch.where(self.live[:, :, None, None], x, torch.zeros((), device=x.device))
        return x.view(self.B, self.n, CHUNK, self.H, self.D).permute(0, 3, 1, 2, 4)

    def join(self, x):
        x = x.permute(0, 2, 3, 1, 4).reshape(self.B, self.n * CHUNK, self.H, self.D)[:, :self.L]
        return torch.where(self.live[:, :self.L, None, None], x, torch.zeros((), device=x.device)).bfloat16()

    def start(self, state):
        if state is not None:
            return state
        return torch.zeros(self.B, self.H, self.D, self.D, device=self.live.device)

    def carry(self, parts, state, order):
        """States before each chunk (in ``order``) and after the last."""
        seen = torch.empty_like(parts)
        for i in order:
            seen[:, :, i] = state
            state = state * self.whole[:, :, i] + parts[:, :, i]
        return seen, state


def _decay_plain(s):
    h = _Chunks(s)
    q, k, v = h.split(s["q"]), h.split(s["k"]), h.split(s["v"])
    parts = (k * h.to_end[..., None]).transpose(-1, -2) @ v
    seen, last = h.carry(parts, h.start(s["state"]), range(h.n))
    o = ((q @ k.transpose(-1, -2)) * h.between) @ v + (q @ seen) * h.to_row[..., None]
    out = [h.join(o * s["scale"])]
    return out + [last] if s["state"] is not None else out


def _decay_back_plain(s):
    h = _Chunks(s)
    q, k, v, do = h.split(s["q"]) * s["scale"], h.split(s["k"]), h.split(s["v"]), h.split(s["do"])
    seen, _ = h.carry((k * h.to_end[..., None]).transpose(-1, -2) @ v, h.start(s["state"]), range(h.n))
    dp = (do @ v.transpose(-1, -2)) * h.between
    dq = (dp @ k + (do @ seen.transpose(-1, -2)) * h.to_row[..., None]) * s["scale"]
    back, dstate = h.carry((q * h.to_row[..., None]).transpose(-1, -2) @ do, h.start(s["dstate"]),
                           range(h.n - 1, -1, -1))
    dk = dp.transpose(-1, -2) @ q + (v @ back.transpose(-1, -2)) * h.to_end[..., None]
    p = (q @ k.transpose(-1, -2)) * h.between
    dv = p.transpose(-1, -2) @ do + (k @ back) * h.to_end[..., None]
    out = [h.join(dq), h.join(dk), h.join(dv)]
    return out + [dstate] if s["state"] is not None else out


def _decay_step_plain(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    state = s["state"] * torch.exp(s["ld"])[:, None, None] + k[..., :, None] * v[..., None, :]
    o = (q[..., None, :] @ state)[..., 0, :] * s["scale"]
    if s["lens"] is not None:
        on = (s["lens"] != 0)[:, None, None]
        o = torch.where(on, o, torch.zeros((), device=o.device))
        state = torch.where(on[..., None], state, s["state"])
    return [o.bfloat16(), state]


def _decay_exact(s, c):
    """The recurrence, one token at a time, in 64 bits."""
    step, back = c["op"] == "decay_step", c["op"] == "decay_back"
    rows = [s[n].double() for n in (("q", "k", "v", "do") if back else ("q", "k", "v"))]
    if step:
        rows = [x[:, None] for x in rows]
    q, k, v = rows[:3]
    B, L, H, D = q.shape
    lens = s["lens"] if s["lens"] is not None else torch.full((B,), L, device=q.device)
    on = (torch.arange(L, device=q.device)[:, None] < lens).double()[:, :, None, None]  # [L, B, 1, 1]
    ld = s["ld"].double().view(1, H, 1)
    g = torch.exp(ld * on)[..., None]  # padding neither decays nor adds
    q, k, v = (x.transpose(0, 1) * on for x in (q, k, v))  # [L, B, H, D]
    S = s["state"].double().clone() if s["state"] is not None else torch.zeros(B, H, D, D, device=q.device).double()
    if not back:
        o = torch.empty_like(q)
        for t in range(L):
            S.mul_(g[t]).addcmul_(k[t].unsqueeze(-1), v[t].unsqueeze(-2))
            torch.matmul(q[t].unsqueeze(-2), S, out=o[t].unsqueeze(-2))
        o = (o * s["scale"]).transpose(0, 1)
        out = [o[:, 0] if step else o]
        return out + [S] if s["state"] is not None else out
    do = rows[3].transpose(0, 1) * on
    dq, dk, dv = (torch.empty_like(q) for _ in range(3))
    for t in range(L):
        S.mul_(g[t]).addcmul_(k[t].unsqueeze(-1), v[t].unsqueeze(-2))
        torch.matmul(S, do[t].unsqueeze(-1), out=dq[t].unsqueeze(-1))
    dq = (dq * s["scale"] * on).transpose(0, 1)
    R = s["dstate"].double().clone() if s["state"] is not None else torch.zeros_like(S)
    q = q * s["scale"]
    for t in range(L - 1, -1, -1):
        R.addcmul_(q[t].unsqueeze(-1), do[t].unsqueeze(-2))
        torch.matmul(R, v[t].unsqueeze(-1), out=dk[t].unsqueeze(-1))
        torch.matmul(k[t].unsqueeze(-2), R, out=dv[t].unsqueeze(-2))
        R.mul_(g[t])
    out = [dq, (dk * on).transpose(0, 1), (dv * on).transpose(0, 1)]
    return out + [R] if s["state"] is not None else out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rotary", "rotary_back"):
        return _rotary_exact(s, case["op"] == "rotary_back")
    return _decay_exact(s, case)


# ----------------------------------------------------------------------- run

def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        if op in ("rotary", "rotary_back"):
            return _rotary_plain(s, op == "rotary_back")
        return {"decay": _decay_plain, "decay_step": _decay_step_plain, "decay_back": _decay_back_plain}[op](s)
    import streaming_attention_block_gb300 as sab

    if op == "rotary":
        sab.rotary(s["plan"], s["q"], s["k"], s["q_out"], s["k_out"], positions=s["pos"])
        return s["q_out"], s["k_out"]
    if op == "rotary_back":
        sab.rotary_backward(s["plan"], s["q"], s["k"], s["q_out"], s["k_out"], positions=s["pos"])
        return s["q_out"], s["k_out"]
    if op == "decay":
        sab.decay_attention(s["q"], s["k"], s["v"], s["ld"], s["scale"], s["o"], state_in=s["state"],
                            state_out=s["state_out"], seq_len=s["lens"], workspace=s["ws"])
        out = [s["o"]]
    elif op == "decay_step":
        sab.decay_attention_step(s["q"], s["k"], s["v"], s["ld"], s["scale"], s["state"], s["state_out"], s["o"],
                                 active=s["lens"])
        out = [s["o"]]
    else:
        sab.decay_attention_backward(s["q"], s["k"], s["v"], s["do"], s["ld"], s["scale"], s["dq"], s["dk"], s["dv"],
                                     state_in=s["state"], d_state_out=s["dstate"], d_state_in=s["state_out"],
                                     seq_len=s["lens"], workspace=s["ws"])
        out = [s["dq"], s["dk"], s["dv"]]
    return out + [s["state_out"]] if s["state"] is not None else out
