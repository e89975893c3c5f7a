"""Cases of the linear-attention and linear-layer operators, for measuring them.

Three operators:

  prompt   linear attention with one decay per head over a whole prompt,
             S_t = g_h S_{t-1} + k_t v_t^T,   o_t = scale q_t^T S_t,
           tensors [n][B][H][dim], a length for each sequence, the state carried
           in and out in 32 bits;
  step     the same recurrence for one new token of every sequence, the state
           updated in place;
  linear   y = act(x W^T + bias) + residual over n rows.

`run` computes each in a plain form from elementary torch operations, or, where
`own` is true, by the library's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64          # positions per chunk of the plain form


def listed():
    return [
        # One long prompt of a 2048-channel stack, 16 heads of 128: a single
        # user's context is read, so few heads have to fill the whole GPU.
        dict(name="prompt-16x128-L16K-bf16-B1", op="prompt", n=16384, batch=1, heads=16, dk=128, dv=128, dtype="bf16",
             ragged=False, carried=False, fused=False),
        # A batch of prompts of the same stack: the largest prefill, all q, k, v
        # views of one fused projection's output.
        dict(name="prompt-16x128-L2K-bf16-B32", op="prompt", n=2048, batch=32, heads=16, dk=128, dv=128, dtype="bf16",
             ragged=False, carried=False, fused=True),
        # The 864-channel stack as 9 heads of 96, four sequences of different
        # lengths in one padded batch that continue from an earlier state.
        dict(name="prompt-9x96-1777-ragged-bf16-B4", op="prompt", n=1777, batch=4, heads=9, dk=96, dv=96, dtype="bf16",
             ragged=True, carried=True, fused=True),
        # The 768-channel stack in 32 bits, 12 heads of 64, an 8K prompt.
        dict(name="prompt-12x64-L8K-f32-B1", op="prompt", n=8192, batch=1, heads=12, dk=64, dv=64, dtype="f32",
             ragged=False, carried=False, fused=False),
        # One token of one sequence of the 768-channel stack: latency alone.
        dict(name="step-12x64-f32-B1", op="step", batch=1, heads=12, dk=64, dv=64, dtype="f32"),
        # One token for each of 64 sequences of the 2048-channel stack: the
        # ordinary serving step, bound by reading and writing the state.
        dict(name="step-16x128-bf16-B64", op="step", batch=64, heads=16, dk=128, dv=128, dtype="bf16"),
        # Odd head sizes and an odd batch, as after sequences have left it.
        dict(name="step-9x(56,104)-bf16-B37", op="step", batch=37, heads=9, dk=56, dv=104, dtype="bf16"),
        # The channel-mixing block's first product for one token: the weights'
        # bytes are all that counts.
        dict(name="linear-1x2048x8192-bf16-gelu", op="linear", n=1, nin=2048, nout=8192, dtype="bf16", act="gelu",
             bias=True, residual=False),
        # A mixer's output projection with its residual for a batch of 64.
        dict(name="linear-64x2048x2048-bf16-res", op="linear", n=64, nin=2048, nout=2048, dtype="bf16", act="none",
             bias=True, residual=True),
        # The 768-channel stack's block in 32 bits over an 8K prompt.
        dict(name="linear-8192x768x768-f32-gelu", op="linear", n=8192, nin=768, nout=768, dtype="f32", act="gelu",
             bias=True, residual=False),
        # The block's first product over a 16K prompt of the 2048-channel stack.
        dict(name="linear-16384x2048x8192-bf16-gelu", op="linear", n=16384, nin=2048, nout=8192, dtype="bf16",
             act="gelu", bias=True, residual=False),
        # Odd sizes throughout: rows that start at no 16-byte boundary.
        dict(name="linear-1777x865x1727-bf16-tanh-res", op="linear", n=1777, nin=865, nout=1727, dtype="bf16",
             act="tanh", bias=True, residual=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _head_dim(rng):
    d = _log_int(rng, 16, 128)
    return d if rng.random() < 0.4 else min(128, (d + 15) // 16 * 16)


def draw(rng):
    """One more case of the same ranges: prompts of 1 to 16K positions, batches of 1
    to 64, heads of 16 to 128 dimensions, products from one row up to the largest
    listed one, both types, odd sizes among them."""
    op = rng.choice(["prompt", "prompt", "step", "linear", "linear"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "linear":
        most = 16384 * 2048 * 8192 // (8 if dtype == "f32" else 1)
        while True:
            n, nin, nout = _log_int(rng, 1, 16384), _log_int(rng, 64, 8192), _log_int(rng, 64, 8192)
            if rng.random() < 0.6:
                nin, nout = (nin + 31) // 32 * 32, (nout + 31) // 32 * 32
            if n * nin * nout <= most:
                break
        return dict(op=op, n=n, nin=nin, nout=nout, dtype=dtype, act=rng.choice(["none", "gelu", "silu", "relu", "tanh"]),
                    bias=rng.random() < 0.7, residual=rng.random() < 0.5)
    heads = rng.randint(1, 18)
    dk = _head_dim(rng)
    dv = dk if rng.random() < 0.7 else _head_dim(rng)
    if op == "step":
        return dict(op=op, batch=_log_int(rng, 1, 64), heads=min(heads, 16), dk=dk, dv=dv, dtype=dtype)
    while True:
        n, batch = _log_int(rng, 1, 16384), _log_int(rng, 1, 32)
        if n * batch * heads * max(dk, dv) <= (2048 * 32 * 16 * 128) // (4 if dtype == "f32" else 1):
            break
    return dict(op=op, n=n, batch=batch, heads=heads, dk=dk, dv=dv, dtype=dtype, ragged=rng.random() < 0.5,
                carried=rng.random() < 0.5, fused=rng.random() < 0.5)


def _lengths(case):
    """Each sequence's length: the whole prompt, or a spread down to an empty one."""
    n, b = case["n"], case["batch"]
    if not case["ragged"]:
        return [n] * b
    return [n - (i * n) // b - (i > 0 and i == b - 1) * ((n - (i * n) // b) // 2) for i in range(b)]


def _activation(u, act):
    if act == "gelu":
        return 0.5 * u * (1.0 + torch.erf(u * math.sqrt(0.5)))
    if act == "silu":
        return u / (1.0 + torch.exp(-u))
    if act == "relu":
        return torch.where(u > 0, u, torch.zeros_like(u))
    if act == "tanh":
        return torch.tanh(u)
    return u


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    st = {"case": case}
    if case["op"] == "linear":
        n, nin, nout = case["n"], case["nin"], case["nout"]
        st["x"] = normal(n, nin)
        st["w"] = normal(nout, nin, scale=nin ** -0.5)
        st["bias"] = normal(nout, scale=0.1) if case["bias"] else None
        st["residual"] = normal(n, nout) if case["residual"] else None
        st["y"] = torch.zeros(n, nout, dtype=dt, device="cuda")
        return st
    b, h, dk, dv = case["batch"], case["heads"], case["dk"], case["dv"]
    # decays from about 1 - 2^-4 to 1 - 2^-11, one for each head
    e = 4.0 + 7.0 * torch.arange(h, dtype=torch.float64, device="cuda") / max(1, h - 1)
    e = e + 0.25 * torch.rand(h, generator=g, dtype=torch.float64, device="cuda")
    st["log_decay"] = torch.log1p(-torch.exp2(-e)).float()
    st["scale"] = dk ** -0.5
    if case["op"] == "step":
        st["q"], st["k"], st["v"] = normal(b, h, dk), normal(b, h, dk, scale=dk ** -0.25), normal(b, h, dv)
        st["state"] = normal(b, h, dk, dv, dtype=torch.float32)
        st["o"] = torch.zeros(b, h, dv, dtype=dt, device="cuda")
        return st
    n = case["n"]
    if case["fused"]:
        qkv = normal(n, b, h * (2 * dk + dv))
        st["q"], st["k"], st["v"] = (t.unflatten(-1, (h, -1)) for t in qkv.split([h * dk, h * dk, h * dv], dim=-1))
    else:
        st["q"], st["k"], st["v"] = normal(n, b, h, dk), normal(n, b, h, dk), normal(n, b, h, dv)
    lens = _lengths(case)
    st["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda") if case["ragged"] else None
    st["state_in"] = normal(b, h, dk, dv, dtype=torch.float32) if case["carried"] else None
    st["state_out"] = torch.zeros(b, h, dk, dv, dtype=torch.float32, device="cuda")
    st["o"] = torch.zeros(n, b, h, dv, dtype=dt, device="cuda")
    return st


def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    if case["op"] == "linear":
        return _plain_linear(st, case)
    return _plain_step(st) if case["op"] == "step" else _plain_prompt(st, case)


def _run_own(st, case):
    from long_convolution_sequence_online_b200 import fi
    if case["op"] == "linear":
        fi.linear(st["x"], st["w"], st["y"], bias=st["bias"], residual=st["residual"], act=case["act"])
        return st["y"]
    if case["op"] == "step":
        fi.linattn_step(st["q"], st["k"], st["v"], st["log_decay"], st["state"], st["o"], scale=st["scale"])
        return {"o": st["o"], "state": st["state"]}
    fi.linattn_prefill(st["q"], st["k"], st["v"], st["log_decay"], st["o"], state_in=st["state_in"],
                       state_out=st["state_out"], lengths=st["lengths"], scale=st["scale"])
    return {"o": st["o"], "state": st["state_out"]}


def _plain_linear(st, case):
    u = st["x"].float() @ st["w"].float().t()
    if st["bias"] is not None:
        u = u + st["bias"].float()
    u = _activation(u, case["act"])
    if st["residual"] is not None:
        u = u + st["residual"].float()
    st["y"].copy_(u)
    return st["y"]


def _plain_step(st):
    decay = torch.exp(st["log_decay"].double()).float()[:, None, None]
    s = decay * st["state"] + st["k"].float()[..., :, None] * st["v"].float()[..., None, :]
    st["state"].copy_(s)
    st["o"].copy_(st["scale"] * (st["q"].float()[..., None, :] @ s)[..., 0, :])
    return {"o": st["o"], "state": st["state"]}


def _plain_prompt(st, case):
    """Chunks of 64 positions: the masked, decayed scores inside a chunk, and the
    states before the chunks as one decayed sum over the chunks before."""
    n, b, h, dk, dv = (case[k] for k in ("n", "batch", "heads", "dk", "dv"))
    dev, ld = st["q"].device, st["log_decay"].double()
    q, k, v = (t.float().permute(1, 2, 0, 3) for t in (st["q"], st["k"], st["v"]))     # [b][h][n][d]
    t = torch.arange(n, device=dev)
    lens = st["lengths"].long() if st["lengths"] is not None else torch.full((b,), n, device=dev)
    live = t < lens[:, None]                                                             # [b][n]
    zero = torch.zeros((), device=dev)
    k, v = (torch.where(live[:, None, :, None], x, zero) for x in (k, v))
    s0 = st["state_in"] if st["state_in"] is not None else torch.zeros(b, h, dk, dv, device=dev)
    # the state after each sequence's last position
    age = torch.where(live, lens[:, None] - 1 - t, torch.zeros_like(t)).double()         # [b][n]
    w = torch.exp(age[:, None, :] * ld[:, None]).float()                                 # [b][h][n]
    s_out = torch.exp(lens.double()[:, None] * ld).float()[..., None, None] * s0 + (k * w[..., None]).transpose(-1, -2) @ v
    # outputs
    c = CHUNK
    m = -(-n // c)
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, m * c - n)).unflatten(2, (m, c)) for x in (q, k, v))
    i = torch.arange(c, device=dev, dtype=torch.float64)
    lag = i[:, None] - i[None, :]
    inside = torch.where(lag >= 0, torch.exp(lag.clamp(min=0) * ld[:, None, None]), torch.zeros_like(lag)).float()
    o = ((q @ k.transpose(-1, -2)) * inside[:, None]) @ v
    left = torch.exp((c - 1 - i) * ld[:, None]).float()[:, None, :, None]
    parts = torch.cat([s0[:, :, None], (k * left).transpose(-1, -2) @ v], dim=2)[:, :, :m]
    j = torch.arange(m, device=dev, dtype=torch.float64)
    gap = (j[:, None] - j[None, :]) * c
    across = torch.where(gap >= 0, torch.exp(gap.clamp(min=0) * ld[:, None, None]), torch.zeros_like(gap)).float()
    before = (across @ parts.flatten(3)).unflatten(3, (dk, dv))                          # [b][h][m][dk][dv]
    o = o + (q * torch.exp((i + 1) * ld[:, None]).float()[:, None, :, None]) @ before
    o = (st["scale"] * o).flatten(2, 3)[:, :, :n].permute(2, 0, 1, 3).to(st["o"].dtype)  # [n][b][h][dv]
    st["o"].copy_(torch.where(live.t()[:, :, None, None], o, st["o"]))
    st["state_out"].copy_(s_out)
    return {"o": st["o"], "state": st["state_out"]}


def exact(case, seed):
    """The definitions in 64 bits: the recurrence position by position, and the product."""
    st = prepare(case, seed)
    if case["op"] == "linear":
        u = torch.einsum("ni,oi->no", st["x"].double(), st["w"].double())
        if st["bias"] is not None:
            u += st["bias"].double()
        if case["act"] == "gelu":
            u = u * torch.special.ndtr(u)
        elif case["act"] == "silu":
            u = u * torch.sigmoid(u)
        elif case["act"] == "relu":
            u = u.clamp(min=0)
        elif case["act"] == "tanh":
            u = torch.tanh(u)
        if st["residual"] is not None:
            u = u + st["residual"].double()
        return u
    decay = st["log_decay"].double().exp().view(1, -1, 1, 1)
    if case["op"] == "step":
        s = st["state"].double() * decay
        s += torch.einsum("bhd,bhe->bhde", st["k"].double(), st["v"].double())
        return {"o": st["scale"] * torch.einsum("bhd,bhde->bhe", st["q"].double(), s), "state": s}
    n, b, h, dk, dv = (case[k] for k in ("n", "batch", "heads", "dk", "dv"))
    lens = _lengths(case)
    s = st["state_in"].double() if case["carried"] else torch.zeros(b, h, dk, dv, dtype=torch.float64, device="cuda")
    o = torch.zeros(n, b, h, dv, dtype=torch.float64, device="cuda")
    q, k, v = st["q"].double(), st["k"].double(), st["v"].double()
    # sequences in order of falling length, so that those still running are a prefix
    order = sorted(range(b), key=lambda r: -lens[r])
    at = torch.tensor(order, device="cuda")
    s, q, k, v = s[at].contiguous(), q[:, at].contiguous(), k[:, at].contiguous(), v[:, at].contiguous()
    alive = b
    for t in range(n):
        while alive and lens[order[alive - 1]] <= t:
            alive -= 1
        if not alive:
            break
        r = s[:alive]
        r.mul_(decay)
        r.add_(k[t, :alive, :, :, None] * v[t, :alive, :, None, :])
        o[t, :alive] = torch.matmul(q[t, :alive, :, None, :], r)[:, :, 0]
    back = torch.empty_like(at)
    back[at] = torch.arange(b, device="cuda")
    return {"o": st["scale"] * o[:, back], "state": s[back]}


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "linear":
        n, nin, nout = case["n"], case["nin"], case["nout"]
        return {"bytes": e * (n * nin + nin * nout + n * nout * (2 if case["residual"] else 1) + (nout if case["bias"] else 0)),
                "flops": 2 * n * nin * nout}
    b, h, dk, dv = case["batch"], case["heads"], case["dk"], case["dv"]
    if case["op"] == "step":
        tokens, states = b, 2
    else:
        tokens, states = sum(_lengths(case)), 2 if case["carried"] else 1
    return {"bytes": tokens * h * 2 * (dk + dv) * e + states * b * h * dk * dv * 4 + 4 * h,
            "flops": tokens * h * 4 * dk * dv}
