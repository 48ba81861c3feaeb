"""Cases of the cross-attention and layer-norm operators, with plain forms.

Four operators, named in a case by ``"op"``:

* ``cross``       attention of one sequence's queries to an encoder's states of another length
* ``cross_back``  its gradients
* ``norm``        layer norm, its weight and bias shared by groups of rows
* ``norm_back``   its gradients, the sums over the rows of a group among them

``run`` with ``own`` false computes them with elementary torch operations in
32 bits, rounded once at the end; with ``own`` true it makes the library calls
a user makes.  ``exact`` evaluates the definitions in 64 bits: the attention
head by head, the norm from moments about the mean.
"""

import math

import torch

own = False

EPS = 1e-6


# --------------------------------------------------------------------- cases

def _cross(name, op, B, Lq, Lk, H, Hk, D, kv_batch=0, q_ragged=False, kv_ragged=False, fused=False):
    return dict(name=name, op=op, B=B, Lq=Lq, Lk=Lk, H=H, Hk=Hk, D=D, kv_batch=kv_batch or B, q_ragged=q_ragged,
                kv_ragged=kv_ragged, fused=fused)


def _norm(name, op, rows, C, group=0, dtype="bf16", offset=0.0):
    return dict(name=name, op=op, rows=rows, C=C, group=group or rows, dtype=dtype, offset=offset)


def listed():
    return [
        # one token of one stream against a short prompt: latency
        _cross("cross_token", "cross", 1, 1, 77, 12, 12, 128),
        # one streamed chunk of 2 x 24 x 32 latent patches against a text prompt
        _cross("cross_chunk", "cross", 1, 1536, 512, 12, 12, 128),
        # one token of each sequence of a padded serving batch against long
        # encoder states with shared heads
        _cross("cross_decode", "cross", 64, 1, 4095, 24, 8, 128, kv_ragged=True, fused=True),
        # a padded batch of both lengths, one sequence and one prompt empty,
        # keys and values as one projection writes them
        _cross("cross_ragged", "cross", 8, 1023, 777, 24, 4, 64, q_ragged=True, kv_ragged=True, fused=True),
        # whole training sequences against text prompts
        _cross("cross_train", "cross", 2, 30720, 512, 12, 12, 128),
        # gradients of one chunk
        _cross("cross_back_chunk", "cross_back", 1, 1536, 512, 12, 12, 128),
        # gradients of a padded batch that shares one prompt, heads shared too
        _cross("cross_back_shared", "cross_back", 4, 2047, 333, 24, 8, 64, kv_batch=1, q_ragged=True, fused=True),
        # gradients of whole training sequences
        _cross("cross_back_train", "cross_back", 2, 30720, 512, 12, 12, 128),
        # the tokens of one streamed chunk
        _norm("norm_chunk", "norm", 1536, 1536),
        # whole training sequences, scale and shift of each chunk's own noise level
        _norm("norm_train", "norm", 61440, 1536, group=1536, offset=1.0),
        # its gradients
        _norm("norm_back_train", "norm_back", 61440, 1536, group=1536, offset=1.0),
        # gradients kept in 32 bits, odd counts of rows and channels
        _norm("norm_back_odd", "norm_back", 4095, 1001, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["cross", "cross", "cross", "cross_back", "cross_back", "norm", "norm_back"])
    if op in ("norm", "norm_back"):
        C = rng.choice([8 * _log_int(rng, 8, 640), _log_int(rng, 64, 5120)])
        rows = _log_int(rng, 1, min(61440, 61440 * 1536 // (2 * C)))
        group = rng.choice([0, 0, _log_int(rng, max(1, rows // 64), rows)])
        return _norm("", op, rows, C, group, rng.choice(["bf16", "bf16", "f32"]), rng.choice([0.0, 1.0]))
    D = rng.choice([64, 128])
    H = rng.randint(1, 24)
    Hk = rng.choice([h for h in range(1, H + 1) if H % h == 0])
    B = _log_int(rng, 1, 64)
    room = 2 * 30720 * 12 * 128
    Lk = _log_int(rng, 1, min(8192, max(1, room // (B * Hk * D))))
    Lq = 1 if op == "cross" and rng.random() < 0.3 else _log_int(rng, 1, 30720)
    Lq = max(1, min(Lq, room // (B * H * D), room * 512 // (B * H * D * Lk)))
    return _cross("", op, B, Lq, Lk, H, Hk, D, rng.choice([0, 0, 0, 1]), rng.random() < 0.3, rng.random() < 0.5,
                  rng.random() < 0.5)


def work(case):
    c = case
    if c["op"] in ("norm", "norm_back"):
        es = 2 if c["dtype"] == "bf16" else 4
        n, groups = c["rows"] * c["C"], -(-c["rows"] // c["group"])
        if c["op"] == "norm":
            return {"bytes": 2 * n * es + 8 * groups * c["C"] + 8 * c["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * es + 12 * groups * c["C"] + 8 * c["rows"], "flops": 14 * n}
    # lengths of the ragged batches average half of the padded ones
    q = c["B"] * c["H"] * c["Lq"] * (0.5 if c["q_ragged"] else 1.0)
    kv = c["kv_batch"] * c["Hk"] * c["Lk"] * (0.5 if c["kv_ragged"] else 1.0)
    all_q, all_kv = c["B"] * c["H"] * c["Lq"], c["kv_batch"] * c["Hk"] * c["Lk"]
    pairs = q * c["Lk"] * (0.5 if c["kv_ragged"] else 1.0)
    D = c["D"]
    if c["op"] == "cross":
        return {"bytes": int(2 * D * (q + all_q + 2 * kv) + 4 * all_q), "flops": int(4 * D * pairs)}
    return {"bytes": int(2 * D * (3 * q + all_q + 2 * kv + 2 * all_kv) + 4 * q), "flops": int(10 * D * pairs)}


# -------------------------------------------------------------------- inputs

def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _lengths(g, n, most):
    """Lengths 0 .. most, the last of several empty."""
    lens = torch.randint(most + 1, (n,), generator=g, device="cuda").to(torch.int32)
    if n > 1:
        lens[-1] = 0
    return lens


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    if c["op"] in ("norm", "norm_back"):
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        rows, C = c["rows"], c["C"]
        groups = -(-rows // c["group"])
        # a residual stream: uneven channels, a few of them large, off centre
        spread = 0.5 + torch.rand(C, generator=g, device="cuda")
        spread = torch.where(torch.rand(C, generator=g, device="cuda") < 0.01, 20.0 * spread, spread)
        s = dict(case=c, x=(_randn(g, rows, C, dtype=torch.float32) * spread + 0.3).to(dt),
                 weight=(1.0 - c["offset"]) + 0.2 * _randn(g, groups, C, dtype=torch.float32),
                 bias=0.2 * _randn(g, groups, C, dtype=torch.float32))
        s["y"] = torch.empty_like(s["x"])
        s["mean"], s["rstd"] = (torch.empty(rows, device="cuda") for _ in range(2))
        if c["op"] == "norm_back":
            s["dy"] = _randn(g, rows, C, dtype=dt)
            s["mean"], s["rstd"] = _moments(s["x"])
            s["dweight"], s["dbias"] = torch.empty_like(s["weight"]), torch.empty_like(s["bias"])
            if own:
                import streaming_attention_block_gb300 as sab

                n = sab.layer_norm_backward_workspace(rows, C, c["group"])
                s["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        return s
    B, Lq, Lk, H, Hk, D, Bk = (c[n] for n in ("B", "Lq", "Lk", "H", "Hk", "D", "kv_batch"))
    s = dict(case=c, scale=D ** -0.5, q=_randn(g, B, Lq, H, D))
    if c["fused"]:
        s["k"], s["v"] = _randn(g, Bk, Lk, 2, Hk, D).unbind(2)
    else:
        s["k"], s["v"] = _randn(g, Bk, Lk, Hk, D), _randn(g, Bk, Lk, Hk, D)
    s["q_len"] = _lengths(g, B, Lq) if c["q_ragged"] else None
    s["kv_len"] = _lengths(g, Bk, Lk) if c["kv_ragged"] else None
    if c["op"] == "cross":
        s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty(B, H, Lq, device="cuda")
    else:
        s["o"], s["lse"] = _cross_plain(s)  # the forward pass is behind the caller
        s["do"] = _randn(g, B, Lq, H, D)
        s["dq"] = torch.empty_like(s["q"])
        if c["fused"]:
            s["dk"], s["dv"] = torch.empty(Bk, Lk, 2, Hk, D, dtype=torch.bfloat16, device="cuda").unbind(2)
        else:
            s["dk"], s["dv"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        if own:
            import streaming_attention_block_gb300 as sab

            n = sab.cross_attention_backward_workspace(B, Lq, Lk, H, Hk, D, Bk)
            s["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    return s


# -------------------------------------------------- cross attention, plainly

def _heads(x, Hk):
    """[B, Lq, H, D] -> [B, Hk, (H / Hk) Lq, D] in 32 bits: the query rows of each key head."""
    B, L, H, D = x.shape
    return x.float().view(B, L, Hk, H // Hk, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, D)


def _tokens(x, H):
    """The way back: [B, Hk, (H / Hk) Lq, D] -> [B, Lq, H, D]."""
    B, Hk, R, D = x.shape
    return x.view(B, Hk, H // Hk, -1, D).permute(0, 3, 1, 2, 4).reshape(B, -1, H, D)


def _scores(s):
    """Scores [B, Hk, rows, Lk] in 32 bits, -inf where a query or key is padding; k and v by head."""
    c = s["case"]
    q = _heads(s["q"], c["Hk"])
    k, v = s["k"].float().transpose(1, 2), s["v"].float().transpose(1, 2)
    x = (q @ k.transpose(-1, -2)) * s["scale"]
    if s["kv_len"] is not None:
        dead = torch.arange(c["Lk"], device=x.device) >= s["kv_len"][:, None]
        x = x.masked_fill(dead[:, None, None, :], -math.inf)
        v = v.masked_fill(dead[:, None, :, None], 0.0)
        k = k.masked_fill(dead[:, None, :, None], 0.0)
    if s["q_len"] is not None:
        dead = torch.arange(c["Lq"], device=x.device) >= s["q_len"][:, None]
        x = x.masked_fill(dead.repeat(1, c["H"] // c["Hk"])[:, None, :, None], -math.inf)
    return x, q, k, v


def _softmax(x):
    """(exp(x - max), their sum, max), a row without a key 0, 0, -inf."""
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    return e, e.sum(-1, keepdim=True), top


def _cross_plain(s):
    c = s["case"]
    x, _, _, v = _scores(s)
    e, total, top = _softmax(x)
    o = (e @ v) / torch.where(total > 0, total, torch.ones_like(total))
    return [_tokens(o, c["H"]).bfloat16(), (top + torch.log(total)).view(c["B"], c["H"], c["Lq"])]


def _cross_back_plain(s):
    c = s["case"]
    x, q, k, v = _scores(s)
    e, total, _ = _softmax(x)
    p = e / torch.where(total > 0, total, torch.ones_like(total))
    do = _heads(s["do"], c["Hk"])
    if s["q_len"] is not None:
        dead = torch.arange(c["Lq"], device=x.device) >= s["q_len"][:, None]
        dead = dead.repeat(1, c["H"] // c["Hk"])[:, None, :, None]
        do, q = do.masked_fill(dead, 0.0), q.masked_fill(dead, 0.0)
    dv = p.transpose(-1, -2) @ do
    dp = do @ v.transpose(-1, -2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * s["scale"]
    dq, dk = ds @ k, ds.transpose(-1, -2) @ q
    if c["kv_batch"] != c["B"]:
        dk, dv = dk.sum(0, keepdim=True), dv.sum(0, keepdim=True)
    return [_tokens(dq, c["H"]).bfloat16(), dk.transpose(1, 2).bfloat16(), dv.transpose(1, 2).bfloat16()]


# ------------------------------------------------------- layer norm, plainly

def _moments(x):
    x = x.float()
    mean = x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((x - mean).square().mean(-1, keepdim=True) + EPS)
    return mean[:, 0], rstd[:, 0]


def _by_row(s, t):
    """[groups, C] -> [rows, C], or [1, C] where one row serves all."""
    c = s["case"]
    return t if t.shape[0] == 1 else t.repeat_interleave(c["group"], 0)[:c["rows"]]


def _norm_plain(s):
    x = s["x"].float()
    mean, rstd = _moments(s["x"])
    y = (x - mean[:, None]) * rstd[:, None] * (s["case"]["offset"] + _by_row(s, s["weight"])) + _by_row(s, s["bias"])
    return [y.to(s["x"].dtype), mean, rstd]


def _group_sums(s, x):
    c = s["case"]
    groups = s["weight"].shape[0]
    x = torch.nn.functional.pad(x, (0, 0, 0, groups * c["group"] - c["rows"]))
    return x.view(groups, c["group"], c["C"]).sum(1)


def _norm_back_plain(s):
    dy = s["dy"].float()
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * (s["case"]["offset"] + _by_row(s, s["weight"]))
    dx = (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True)) * s["rstd"][:, None]
    return [dx.to(s["x"].dtype), _group_sums(s, dy * xhat), _group_sums(s, dy)]


# ----------------------------------------------------- definitions in 64 bits

def _cross_exact(s):
    c = s["case"]
    back = c["op"] == "cross_back"
    B, Lq, Lk, H, D = c["B"], c["Lq"], c["Lk"], c["H"], c["D"]
    dev = s["q"].device
    o, dq = (torch.zeros(B, Lq, H, D, dtype=torch.float64, device=dev) for _ in range(2))
    lse = torch.full((B, H, Lq), -math.inf, dtype=torch.float64, device=dev)
    dk, dv = (torch.zeros(c["kv_batch"], Lk, c["Hk"], D, dtype=torch.float64, device=dev) for _ in range(2))
    q_len = [Lq] * B if s["q_len"] is None else s["q_len"].tolist()
    kv_len = [Lk] * c["kv_batch"] if s["kv_len"] is None else s["kv_len"].tolist()
    for b in range(B):
        e = b if c["kv_batch"] == B else 0
        m, n = q_len[b], kv_len[e]
        if m == 0 or n == 0:
            continue
        for h in range(H):
            j = h * c["Hk"] // H
            q, k, v = s["q"][b, :m, h].double(), s["k"][e, :n, j].double(), s["v"][e, :n, j].double()
            x = q.mul(s["scale"]) @ k.T
            z = torch.logsumexp(x, dim=1)
            p = torch.exp(x - z[:, None])
            out = p @ v
            if not back:
                o[b, :m, h], lse[b, h, :m] = out, z
                continue
            do = s["do"][b, :m, h].double()
            dx = p * (do @ v.T - (do * out).sum(1, keepdim=True))
            dv[e, :n, j] += p.T @ do
            dk[e, :n, j] += dx.T @ q * s["scale"]
            dq[b, :m, h] = dx @ k * s["scale"]
    return [dq, dk, dv] if back else [o, lse]


def _norm_exact(s):
    c = s["case"]
    x = s["x"].double()
    mean = x.sum(1) / c["C"]
    d = x - mean[:, None]
    rstd = ((d * d).sum(1) / c["C"] + EPS) ** -0.5
    at = torch.arange(c["rows"], device=x.device) // c["group"]
    w = c["offset"] + s["weight"].double()[at]
    if c["op"] == "norm":
        return [d * rstd[:, None] * w + s["bias"].double()[at], mean, rstd]
    dy = s["dy"].double()
    u = d * rstd[:, None]
    dw, db = (torch.zeros(s["weight"].shape, dtype=torch.float64, device=x.device) for _ in range(2))
    dw.index_add_(0, at, dy * u)
    db.index_add_(0, at, dy)
    t = dy * w
    inner = (t * u).sum(1, keepdim=True) / c["C"]
    return [rstd[:, None] * (t - t.sum(1, keepdim=True) / c["C"] - u * inner), dw, db]


def exact(case, seed):
    s = prepare(case, seed)
    return _norm_exact(s) if case["op"] in ("norm", "norm_back") else _cross_exact(s)


# ----------------------------------------------------------------------- run

def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"cross": _cross_plain, "cross_back": _cross_back_plain, "norm": _norm_plain,
                "norm_back": _norm_back_plain}[op](s)
    import streaming_attention_block_gb300 as sab

    if op == "cross":
        sab.cross_attention(s["q"], s["k"], s["v"], s["scale"], s["o"], s["lse"], q_len=s["q_len"],
                            kv_len=s["kv_len"])
        return [s["o"], s["lse"]]
    if op == "cross_back":
        sab.cross_attention_backward(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], s["scale"], s["dq"], s["dk"],
                                     s["dv"], q_len=s["q_len"], kv_len=s["kv_len"], workspace=s["ws"])
        return [s["dq"], s["dk"], s["dv"]]
    c = s["case"]
    if op == "norm":
        sab.layer_norm(s["x"], s["weight"], s["bias"], EPS, s["y"], s["mean"], s["rstd"], group_rows=c["group"],
                       weight_offset=c["offset"])
        return [s["y"], s["mean"], s["rstd"]]
    sab.layer_norm_backward(s["x"], s["dy"], s["weight"], s["mean"], s["rstd"], s["y"], s["dweight"], s["dbias"],
                            group_rows=c["group"], weight_offset=c["offset"], workspace=s["ws"])
    return [s["y"], s["dweight"], s["dbias"]]
