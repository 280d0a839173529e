"""Cases, plain forms and 64-bit definitions of the sequence-mixing operators
next to the S4 layer: the gated delta rule (chunked forward and backward,
recurrent step) and layer norm (forward and backward, token rows and the
channel layout of the S4Block).

Gated delta rule, per head, state S [Dk, Dv]:
    S_t = a_t S_{t-1} + k_t u_t^T,   a_t = exp(g_t),
    u_t = beta_t (v_t - a_t S_{t-1}^T k_t),   o_t = scale * S_t^T q_t.
q, k [.., Hk, Dk] are shared by Hv / Hk value heads each; v, o [.., Hv, Dv].
"""
import math
import random

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
CHUNK = 64


def _delta(name, way, dtype, batch, tokens, hk, hv, dk, dv, packed=False, state=False):
    """way: forward, train or step. packed: `batch` sequences of unequal
    lengths, `tokens` in all; otherwise `tokens` in each. state: an initial
    state is given (and, in training, a gradient of the final one)."""
    c = {"op": "gated_delta", "way": way, "dtype": dtype, "batch": batch, "tokens": tokens, "hk": hk, "hv": hv,
         "dk": dk, "dv": dv, "packed": packed, "state": state}
    return dict(c, name=name) if name else c


def _norm(name, layout, dtype, rows, width, length=0):
    """layout rows: x [rows, width]. layout channels: x [rows, width, length],
    the norm over `width` at each (row, position)."""
    c = {"op": "layernorm", "layout": layout, "dtype": dtype, "rows": rows, "width": width, "length": length}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one short prompt through a small layer (256 channels as 4 heads of 64): launches and latency
        _delta("prompt_77", "forward", "bfloat16", 1, 77, 4, 4, 64, 64),
        # a server's prefill: 13 prompts of unequal lengths packed one after the other, continued from given states
        _delta("prefill_packed_16k", "forward", "bfloat16", 13, 16384, 8, 16, 128, 128, packed=True, state=True),
        # one very long document, few heads: the longest chain of chunks
        _delta("prefill_64k_8_heads", "forward", "bfloat16", 1, 65536, 4, 8, 128, 128),
        # a training step of the 256-channel layer in the framework's own float32
        _delta("train_f32_256ch", "train", "float32", 8, 2048, 4, 4, 64, 64),
        # a training step of a wide layer, four times 4096 tokens
        _delta("train_4k_32_heads", "train", "bfloat16", 4, 4096, 16, 32, 128, 128),
        # ragged everything: odd lengths, shared key heads, unequal head sizes, gradients of the carried state
        _delta("train_ragged_f16", "train", "float16", 5, 3001, 2, 6, 96, 80, packed=True, state=True),
        # decoding one sequence, one token: latency
        _delta("step_1", "step", "bfloat16", 1, 1, 8, 16, 128, 128, state=True),
        # decoding a full batch, one token each: every state read and written
        _delta("step_256", "step", "bfloat16", 256, 1, 16, 32, 128, 128, state=True),
        # pre-norm of a training step, 8 times 4096 tokens of 1024 channels
        _norm("norm_bf16_32k_1024", "rows", "bfloat16", 32768, 1024),
        # pre-norm of a few odd rows in float32
        _norm("norm_f32_997_250", "rows", "float32", 997, 250),
        # the S4Block's pre-norm, backward, at 256 channels of 16384 steps and batch 8
        _norm("channels_256_16k", "channels", "float32", 8, 256, 16384),
        # the same in a small block
        _norm("channels_100_64", "channels", "float32", 3, 100, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["forward", "forward", "train", "train", "step", "step", "rows", "channels"])
    if kind == "rows":
        width = _log(rng, 32, 8192)
        return _norm("", "rows", rng.choice(sorted(DTYPES)), _log(rng, 8, max(9, 33000000 // width)), width)
    if kind == "channels":
        width, length = _log(rng, 8, 1024), 1 << rng.randint(4, 14)
        return _norm("", "channels", "float32", rng.randint(1, max(1, min(8, 33000000 // (width * length)))), width,
                     length)
    dtype = rng.choice(sorted(DTYPES))
    hk = rng.choice([1, 2, 3, 4, 8])
    hv = hk * rng.choice([1, 1, 2, 3, 4])
    dk, dv = 8 * rng.randint(4, 16), 8 * rng.randint(4, 16)
    if kind == "step":
        return _delta("", "step", dtype, _log(rng, 1, 256), rng.choice([1, 1, 1, 2, 5]), hk, hv, dk, dv, state=True)
    batch = rng.randint(1, 9)
    most = 65536 * 8 // hv if kind == "forward" else 4096 * 4 * 32 // hv
    most = min(most, 65536 if kind == "forward" else 16384)
    packed = rng.random() < 0.5
    tokens = _log(rng, 16, most)
    if not packed:
        tokens = max(1, tokens // batch)
    return _delta("", kind, dtype, batch, tokens, hk, hv, dk, dv, packed=packed, state=rng.random() < 0.5)


def _lengths(case):
    """The packed sequences' lengths: cuts at random places; from five
    sequences on, the second has one token and the third none."""
    n, total = case["batch"], case["tokens"]
    rng = random.Random(1000003 * n + total)
    if n < 5:
        cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
        edges = [0] + cuts + [total]
        return [b - a for a, b in zip(edges, edges[1:])]
    cuts = sorted(rng.randint(0, total - 1) for _ in range(n - 3))
    edges = [0] + cuts + [total - 1]
    rest = [b - a for a, b in zip(edges, edges[1:])]
    return rest[:1] + [1, 0] + rest[1:]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=gen)

    dt = DTYPES[case["dtype"]]
    if case["op"] == "layernorm":
        rows, width = case["rows"], case["width"]
        shape = (rows, width) if case["layout"] == "rows" else (rows, width, case["length"])
        x = normal(*shape).mul_(1.7).add_(0.3)
        return {"case": case, "x": x.to(dt), "dz": normal(*shape).to(dt), "gamma": 1 + 0.2 * normal(width),
                "beta": 0.1 * normal(width), "eps": 1e-5}
    b, t, hk, hv, dk, dv = (case[x] for x in ("batch", "tokens", "hk", "hv", "dk", "dv"))
    lead = (1, t) if case["packed"] else (b, t)
    # what a gated delta layer feeds its mixer: keys and queries of norm one, a
    # decay exp(-A softplus(.)) with A per head between 1 and 16 and steps of
    # about 0.001 to 0.1, a writing strength in (0, 1)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k = (unit(normal(*lead, hk, dk)).to(dt) for _ in range(2))
    v = normal(*lead, hv, dv).to(dt)
    a = torch.exp(uniform(hv) * math.log(16.0))
    step = torch.exp(math.log(1e-3) + uniform(hv) * math.log(100.0))
    bias = torch.log(torch.expm1(step))
    g = -a * torch.nn.functional.softplus(0.5 * normal(*lead, hv) + bias)
    beta = torch.sigmoid(normal(*lead, hv))
    s = {"case": case, "q": q, "k": k, "v": v, "g": g, "beta": beta, "scale": dk ** -0.5, "state": None, "cu": None,
         "lengths": _lengths(case) if case["packed"] else [t] * b}
    if case["state"]:
        s["state"] = 0.5 * normal(b, hv, dk, dv)
    if case["packed"]:
        edges = [0]
        for n in s["lengths"]:
            edges.append(edges[-1] + n)
        s["cu"] = torch.tensor(edges, dtype=torch.int32, device="cuda")
    if case["way"] == "train":
        s["do"] = normal(*lead, hv, dv).to(dt)
        s["dstate"] = normal(b, hv, dk, dv) if case["state"] else None
    if case["way"] == "step" and t == 1:
        for n in ("q", "k", "v", "g", "beta"):
            s[n] = s[n].squeeze(1)
    return s


# ------------------------------------------------------------------ runs ---
def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    if case["op"] == "layernorm":
        return _plain_norm(s)
    if case["way"] == "step":
        return _plain_step(s)
    if case["way"] == "forward":
        o, last = _plain_delta(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s)
        return o, last
    leaves = [s[n].detach().requires_grad_() for n in ("q", "k", "v", "g", "beta")]
    if s["state"] is not None:
        leaves.append(s["state"].detach().requires_grad_())
    with torch.enable_grad():
        o, last = _plain_delta(*leaves[:5], leaves[5] if len(leaves) > 5 else None, s)
        outs, grads = [o], [s["do"]]
        if s["dstate"] is not None:
            outs.append(last)
            grads.append(s["dstate"])
        grads = torch.autograd.grad(outs, leaves, grads)
    names = ("q", "k", "v", "g", "beta", "initial_state")
    return o.detach(), last.detach(), dict(zip(names, grads))


def _run_own(s):
    import structured_state_space_dplr_b200 as s4
    case = s["case"]
    if case["op"] == "layernorm":
        if case["layout"] == "channels":
            return s4.layernorm_channels_backward(s["dz"], s["x"], s["gamma"], s["eps"])
        z, mean, rstd = s4.layernorm(s["x"], s["gamma"], s["beta"], s["eps"])
        return (z, *s4.layernorm_backward(s["dz"], s["x"], s["gamma"], mean, rstd))
    args = (s["q"], s["k"], s["v"], s["g"], s["beta"])
    if case["way"] == "step":
        call = s4.gated_delta_step if case["tokens"] == 1 else s4.gated_delta_scan
        return call(*args, s["state"], scale=s["scale"]), s["state"]
    train = case["way"] == "train"
    o, last, work = s4.gated_delta_forward(*args, scale=s["scale"], initial_state=s["state"], cu_seqlens=s["cu"],
                                           keep=train)
    if not train:
        return o, last
    grads = s4.gated_delta_backward(*args, s["do"], work, scale=s["scale"], dfinal_state=s["dstate"],
                                    cu_seqlens=s["cu"])
    if s["state"] is None:
        grads.pop("initial_state", None)
    return o, last, grads


# ----------------------------------------------------------- plain forms ---
def _plain_norm(s):
    case = s["case"]
    rows = case["layout"] == "rows"
    axis = -1 if rows else 1
    shape = (-1,) if rows else (-1, 1)
    x, dz = s["x"].float(), s["dz"].float()
    gamma, beta = s["gamma"].reshape(shape), s["beta"].reshape(shape)
    centred = x - x.mean(axis, keepdim=True)
    rstd = torch.rsqrt((centred * centred).mean(axis, keepdim=True) + s["eps"])
    xhat = centred * rstd
    others = [d for d in range(x.dim()) if d != axis % x.dim()]
    h = dz * gamma
    dx = rstd * (h - h.mean(axis, keepdim=True) - xhat * (h * xhat).mean(axis, keepdim=True))
    grads = (dx.to(s["x"].dtype), (dz * xhat).sum(others), dz.sum(others))
    return ((xhat * gamma + beta).to(s["x"].dtype), *grads) if rows else grads


def _plain_step(s):
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    g, beta, dt = s["g"], s["beta"], s["v"].dtype
    single = q.dim() == 3
    if single:
        q, k, v, g, beta = (x.unsqueeze(1) for x in (q, k, v, g, beta))
    r = v.shape[2] // q.shape[2]
    q, k = q.repeat_interleave(r, 2), k.repeat_interleave(r, 2)
    state, os = s["state"], []
    for t in range(q.shape[1]):
        state.mul_(torch.exp(g[:, t])[..., None, None])
        u = beta[:, t, :, None] * (v[:, t] - (k[:, t, :, None] @ state)[:, :, 0])
        state.add_(k[:, t, :, :, None] * u[:, :, None])
        os.append(s["scale"] * (q[:, t, :, None] @ state)[:, :, 0])
    o = torch.stack(os, 1).to(dt)
    return (o[:, 0] if single else o), state


def _padded(s):
    """[n, longest] token numbers and which of them are real."""
    n = torch.tensor(s["lengths"], device="cuda")
    longest = -(-max(max(s["lengths"]), 1) // CHUNK) * CHUNK
    first = torch.cumsum(n, 0) - n
    at = torch.arange(longest, device="cuda")
    real = at < n[:, None]
    return torch.where(real, first[:, None] + at, 0), real


def _unit_lower_inverse(a):
    """(I + a)^-1 for strictly lower triangular a [.., C, C]: inverses of the
    diagonal blocks of size 1, 2, 4, ... each from two of half the size."""
    c = a.shape[-1]
    inv = torch.ones(*a.shape[:-2], c, 1, 1, device=a.device, dtype=a.dtype)
    size = 1
    while size < c:
        blocks = a.unflatten(-1, (c // size, size)).unflatten(-3, (c // size, size)).transpose(-3, -2)
        low = torch.arange(0, c // size, 2, device=a.device)
        a21 = blocks[..., low + 1, low, :, :]
        x11, x22 = inv[..., 0::2, :, :], inv[..., 1::2, :, :]
        x21 = -(x22 @ a21 @ x11)
        top = torch.cat([x11, torch.zeros_like(x11)], -1)
        inv = torch.cat([top, torch.cat([x21, x22], -1)], -2)
        size *= 2
    return inv[..., 0, :, :]


def _plain_delta(q, k, v, g, beta, state, s):
    """The chunked form: within a chunk (G the running sum of g)
        A_ij = beta_i exp(G_i - G_j) k_i.k_j (j < i),  T = (I + A)^-1,
        R = T (beta v) - T (beta exp(G) k) S,
        o = scale (exp(G) q S + (q k^T exp(G_i - G_j))_{j <= i} R),
        S' = exp(G_C) S + (exp(G_C - G) k)^T R."""
    dt, shape = v.dtype, v.shape
    rows, real = _padded(s)
    n, c = rows.shape[0], rows.shape[1] // CHUNK

    def chunks(x, heads):  # [n, heads, c, CHUNK, ..], zeros behind the end
        x = x.flatten(0, 1)[rows].float()
        x = x * real.reshape(real.shape + (1,) * (x.dim() - 2))
        x = x.repeat_interleave(heads // x.shape[2], 2)
        return x.transpose(1, 2).unflatten(2, (c, CHUNK))

    hv = v.shape[2]
    q, k, v, g, beta = (chunks(x, hv) for x in (q, k, v, g, beta))
    run_g = torch.cumsum(g.double(), -1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril()
    decay = torch.exp((run_g[..., :, None] - run_g[..., None, :]).masked_fill(~low, -math.inf)).float()
    into = torch.exp(run_g).float()[..., None]
    left = torch.exp(run_g[..., -1:] - run_g).float()[..., None]
    total = torch.exp(run_g[..., -1]).float()[..., None, None]
    kt = k.transpose(-1, -2)
    inv = _unit_lower_inverse((beta[..., None] * decay * (k @ kt)).tril(-1))
    b = beta[..., None]
    u, w = inv @ (b * v), inv @ (b * into * k)
    kl = (left * k).transpose(-1, -2)
    if state is None:
        state = torch.zeros(n, hv, k.shape[-1], v.shape[-1], device="cuda")
    states, news = [], []
    for i in range(c):
        states.append(state)
        new = u[:, :, i] - w[:, :, i] @ state
        news.append(new)
        state = total[:, :, i] * state + kl[:, :, i] @ new
    states, news = torch.stack(states, 2), torch.stack(news, 2)
    o = s["scale"] * (into * (q @ states) + ((q @ kt) * decay) @ news)
    o = o.flatten(2, 3).transpose(1, 2)[real].to(dt)
    return o.reshape(shape), state


# ------------------------------------------------------ 64-bit definition ---
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "layernorm":
        return _exact_norm(s)
    steps = max(s["lengths"]) if s["lengths"] else 0
    cells = case["batch"] * case["hv"] * case["dk"] * case["dv"]
    # steps of about 100 us (forward) and 500 us (train) of launches, and some
    # passes over the 64-bit state
    passes = 12 if case["way"] == "train" else 4
    if steps * ((500e-6 if passes > 4 else 100e-6) + passes * cells * 16 / 3e12) > 15:
        return None
    return _exact_delta(s)


def _exact_norm(s):
    case = s["case"]
    x, dz, gamma, beta = (s[n].double() for n in ("x", "dz", "gamma", "beta"))
    if case["layout"] == "channels":
        x, dz = x.movedim(1, -1), dz.movedim(1, -1)
    d = x.shape[-1]
    mu = x.sum(-1, keepdim=True) / d
    var = ((x - mu) ** 2).sum(-1, keepdim=True) / d
    y = (x - mu) / torch.sqrt(var + s["eps"])
    flat = lambda a: a.reshape(-1, d)  # noqa: E731
    dgamma, dbeta = flat(dz * y).sum(0), flat(dz).sum(0)
    dy = dz * gamma
    dx = (dy - dy.sum(-1, keepdim=True) / d - y * (dy * y).sum(-1, keepdim=True) / d) / torch.sqrt(var + s["eps"])
    if case["layout"] == "channels":
        return dx.movedim(-1, 1).contiguous(), dgamma, dbeta
    return y * gamma + beta, dx, dgamma, dbeta


def _exact_delta(s):
    """The recurrence token by token, and its adjoint token by token (states
    recomputed from checkpoints every 64 tokens)."""
    case = s["case"]
    lengths, n, hv = s["lengths"], case["batch"], case["hv"]
    dk, dv, r, scale = case["dk"], case["dv"], case["hv"] // case["hk"], s["scale"]
    single = s["q"].dim() == 3
    steps = max(lengths)
    edges = [sum(lengths[:i]) for i in range(n)]
    flat = {m: (s[m] if single else s[m].flatten(0, 1)).double() for m in ("q", "k", "v", "g", "beta")}
    if "do" in s:
        flat["do"] = s["do"].flatten(0, 1).double()
    seq = {}
    for m, x in flat.items():  # [steps, n * hv, ..]; behind a sequence's end nothing decays and nothing is written
        wide = torch.zeros(n, steps, *x.shape[1:], dtype=torch.float64, device="cuda")
        for i, (e, l) in enumerate(zip(edges, lengths)):
            wide[i, :l] = x[e:e + l]
        if m in "qk":
            wide = wide.repeat_interleave(r, 2)
        seq[m] = wide.transpose(0, 1).flatten(1, 2).contiguous()
    q, k, v, beta = (seq[m] for m in ("q", "k", "v", "beta"))
    alpha = torch.exp(seq["g"])
    start = torch.zeros(n, hv, dk, dv, dtype=torch.float64, device="cuda") if s["state"] is None else s["state"].double()
    state = start.reshape(n * hv, dk, dv).clone()

    def forward(state, t):
        decayed = state * alpha[t][:, None, None]
        miss = v[t] - torch.bmm(k[t][:, None], decayed)[:, 0]
        u = miss * beta[t][:, None]
        return decayed, miss, u, torch.baddbmm(decayed, k[t][:, :, None], u[:, None])

    o = torch.empty_like(v)
    marks = []
    for t in range(steps):
        if case["way"] == "train" and t % 64 == 0:
            marks.append(state)
        state = forward(state, t)[3]
        o[t] = scale * torch.bmm(q[t][:, None], state)[:, 0]

    def packed(x):  # [steps, n * hv, ..] -> the layout of the inputs
        x = x.unflatten(1, (n, hv)).transpose(0, 1)
        return torch.cat([x[i, :l] for i, l in enumerate(lengths)])

    like = lambda x, heads: packed(x).reshape(*s["v"].shape[:-2], heads, *x.shape[2:])  # noqa: E731
    last = state.reshape(n, hv, dk, dv)
    if case["way"] != "train":
        return like(o, hv), last
    do = seq["do"]
    d = torch.zeros_like(state) if s["dstate"] is None else s["dstate"].double().reshape(n * hv, dk, dv)
    dq, dkk, dvv, dg, db = (torch.empty_like(x) for x in (q, k, v, beta, beta))
    for c in range(len(marks) - 1, -1, -1):
        kept, x = [], marks[c]
        for t in range(64 * c, min(steps, 64 * c + 64)):
            kept.append(forward(x, t))
            x = kept[-1][3]
        for t in range(min(steps, 64 * c + 64) - 1, 64 * c - 1, -1):
            decayed, miss, u, after = kept[t - 64 * c]
            dq[t] = scale * torch.bmm(after, do[t][:, :, None])[:, :, 0]
            d = torch.baddbmm(d, q[t][:, :, None], do[t][:, None], alpha=scale)
            du = torch.bmm(k[t][:, None], d)[:, 0]
            db[t] = (du * miss).sum(-1)
            dm = du * beta[t][:, None]
            dvv[t] = dm
            dkk[t] = torch.bmm(d, u[:, :, None])[:, :, 0] - torch.bmm(decayed, dm[:, :, None])[:, :, 0]
            d = torch.baddbmm(d, k[t][:, :, None], dm[:, None], alpha=-1)
            dg[t] = (d * decayed).sum((-1, -2))
            d = d * alpha[t][:, None, None]
    shared = lambda x: like(x, hv).unflatten(-2, (hv // r, r)).sum(-2)  # noqa: E731
    grads = {"q": shared(dq), "k": shared(dkk), "v": like(dvv, hv), "g": like(dg, hv), "beta": like(db, hv)}
    if s["state"] is not None:
        grads["initial_state"] = d.reshape(n, hv, dk, dv)
    return like(o, hv), last, grads


# ------------------------------------------------------------------ work ---
def work(case):
    size = DTYPES[case["dtype"]].itemsize
    if case["op"] == "layernorm":
        n = case["rows"] * case["width"] * max(1, case["length"])
        if case["layout"] == "rows":  # forward: read x, write z; backward: read dz and x, write dx
            return {"bytes": 5 * n * size + 16 * case["width"], "flops": 20 * n}
        return {"bytes": 3 * n * size + 12 * case["width"], "flops": 14 * n}
    tokens = case["tokens"] * (1 if case["packed"] else case["batch"])
    hk, hv, dk, dv = (case[x] for x in ("hk", "hv", "dk", "dv"))
    states = case["batch"] * hv * dk * dv * 4
    qk, vo, gates = 2 * tokens * hk * dk * size, tokens * hv * dv * size, 2 * tokens * hv * 4
    once = 6 * tokens * hv * dk * dv  # S^T k, k u^T and S^T q of every token
    if case["way"] != "train":
        return {"bytes": qk + 2 * vo + gates + states * (2 if case["state"] else 1), "flops": once}
    back = 14 * tokens * hv * dk * dv  # the state again, its adjoint, and the products for dq, dk, dv
    read, wrote = qk + vo + gates, vo + states + qk + vo + gates  # o, last; dq, dk, dv, dg, dbeta
    more = states * 3 if case["state"] else 0  # the initial state and the last one's gradient in, the first one's out
    return {"bytes": read + vo + wrote + more, "flops": once + back}
