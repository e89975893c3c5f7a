"""Linear attention (prompt and single-token forms) and the linear layer on the GPU
against their float64 oracle.

Tolerances, from the roundings alone (a rounding is off by at most eps/2 of the
value: 2^-8 in bf16, 2^-24 in fp32):

* fp32 sums of N products: |error| <= (N + 16) 2^-24 A, A the same sum over absolute
  values (16: the decay's powers, their exponents, the scale, the rounding of the
  result). Products of operands split into three bf16 parts drop less than 2^-24 of
  each product, one of the 16.
* bf16 linear attention rounds the decayed scores and the state to bf16 where they
  enter a product: elementwise at most 2^-8 A for both together, with A the sum over
  absolute values, and 2^-8 |o| for the result. Over a whole output these are three
  independent roundings of root mean square at most 2^-8 / sqrt(3) each, so the
  relative 2-norm of the error is at most 2^-8.
* the state is never rounded below fp32, whatever the inputs' type.
"""
import math

import numpy as np
import pytest

from oracle import ops

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U32, U16 = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def fi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_convolution_sequence_online_b200 import fi as _fi
    return _fi


def _rand(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _f64(t):
    return t.detach().double().cpu().numpy()


DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _check_la(o, S, q, k, v, ld, scale, s0, lens, dtype):
    """o [n][B][H][dv] and S against the oracle."""
    n = q.shape[0]
    want_o, want_S = ops.linattn(_f64(q), _f64(k), _f64(v), _f64(ld), scale, None if s0 is None else _f64(s0), lens)
    A_o, A_S = ops.linattn(np.abs(_f64(q)), np.abs(_f64(k)), np.abs(_f64(v)), _f64(ld), abs(scale),
                           None if s0 is None else np.abs(_f64(s0)), lens)
    N = n * 1.0 + q.shape[-1] + 16
    err = np.abs(_f64(o) - want_o)
    tol = N * U32 * A_o
    if dtype == "bf16":
        tol = tol + U16 * A_o + U16 * np.abs(want_o)
    assert np.all(err <= tol), (err - tol).max()
    if dtype == "bf16" and np.linalg.norm(want_o) > 0 and want_o.size >= 64:
        assert np.linalg.norm(err) <= U16 * np.linalg.norm(want_o)
    if S is not None:
        err = np.abs(_f64(S) - want_S)
        assert np.all(err <= N * U32 * A_S), (err / np.maximum(A_S, 1e-30)).max()


def _la_inputs(n, B, H, dk, dv, dtype, seed, fused=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[dtype]
    if fused:
        t = _rand(g, n, B, H * (2 * dk + dv), dtype=dt)
        q, k, v = (x.unflatten(-1, (H, -1)) for x in t.split([H * dk, H * dk, H * dv], dim=-1))
    else:
        q, k, v = _rand(g, n, B, H, dk, dtype=dt), _rand(g, n, B, H, dk, dtype=dt), _rand(g, n, B, H, dv, dtype=dt)
    ld = torch.log1p(-torch.exp2(-(1.0 + 9.0 * torch.rand(H, generator=g, device="cuda"))))
    s0 = _rand(g, B, H, dk, dv)
    return q, k, v, ld, s0


LA_CASES = [
    # n, B, H, dk, dv, fused, lengths, carried
    (1, 1, 1, 64, 64, False, None, False),
    (1, 2, 3, 128, 128, False, None, True),
    (2, 1, 2, 1, 1, False, None, True),
    (63, 1, 2, 64, 64, False, None, False),
    (64, 2, 1, 128, 128, False, None, True),
    (65, 1, 2, 128, 64, True, None, True),
    (127, 1, 1, 64, 128, False, None, False),
    (128, 1, 2, 96, 96, True, None, True),
    (129, 3, 2, 128, 128, True, [129, 1, 0], True),
    (200, 2, 2, 56, 104, False, [200, 77], False),
    (257, 2, 1, 128, 128, False, [128, 256], True),
    (300, 4, 2, 40, 72, True, [300, 128, 129, 0], True),
    (333, 1, 2, 33, 47, True, None, True),         # rows at no 16-byte boundary
    (600, 1, 1, 128, 128, False, None, True),      # several segments
    (1777, 1, 1, 96, 96, False, None, True),
    (2500, 2, 1, 64, 64, False, [2500, 1301], True),
    (150, 1, 2, 200, 256, False, None, True),      # dimensions above 128
    (400, 1, 1, 256, 130, False, None, False),
    (1500, 2, 1, 64, 128, True, [1500, 640], True),
    (1100, 1, 2, 128, 64, False, None, True),
    (900, 3, 1, 24, 100, True, [900, 128, 700], True),
    (640, 1, 1, 40, 40, False, None, True),        # whole chunks only
    (260, 160, 1, 16, 16, False, None, False),     # more heads than SMs: a CTA takes several
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,B,H,dk,dv,fused,lens,carried", LA_CASES)
def test_prefill(fi, n, B, H, dk, dv, fused, lens, carried, dtype):
    q, k, v, ld, s0 = _la_inputs(n, B, H, dk, dv, dtype, 7 * n + dk, fused)
    lengths = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    if lens is not None:               # what stands behind a length is not used
        for b, m in enumerate(lens):
            for t in (q, k, v):
                t[m:, b] = math.nan
    o = torch.full((n, B, H, dv), 7.0, dtype=DT[dtype], device="cuda")
    S = torch.full_like(s0, math.nan)
    scale = dk ** -0.5
    fi.linattn_prefill(q, k, v, ld, o, state_in=s0 if carried else None, state_out=S, lengths=lengths, scale=scale)
    torch.cuda.synchronize()
    if lens is not None:
        for b, m in enumerate(lens):
            assert torch.all(o[m:, b] == 7.0)
            o[m:, b] = 0
            for t in (q, k, v):
                t[m:, b] = 0
    _check_la(o, S, q, k, v, ld, scale, s0 if carried else None, lens, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prefill_strides_shared_heads_and_in_place_state(fi, dtype):
    # keys shared by all heads (a stride of 0), values with the head outside the
    # position, o with its dimensions in another order, the state updated in place
    n, B, H, dk, dv = 190, 2, 4, 64, 128
    g = torch.Generator(device="cuda").manual_seed(5)
    dt = DT[dtype]
    q = _rand(g, B, n, H, dk, dtype=dt).transpose(0, 1)
    k = _rand(g, n, B, 1, dk, dtype=dt).expand(n, B, H, dk)
    v = _rand(g, B, H, n, dv, dtype=dt).permute(2, 0, 1, 3)
    o = torch.empty(H, B, n, dv, dtype=dt, device="cuda").permute(2, 1, 0, 3)
    ld = torch.log(torch.tensor([0.5, 0.9, 0.99, 1.0], device="cuda"))
    s0 = _rand(g, B, H, dk, dv)
    S = s0.clone()
    fi.linattn_prefill(q, k, v, ld, o, state_in=S, state_out=S, scale=0.25)
    torch.cuda.synchronize()
    _check_la(o, S, q, k, v, ld, 0.25, s0, None, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_in_place_state_over_segments(fi, d, dtype):
    # one head: the prompt is cut into segments, one of which writes the state
    # that the others start from
    n = 2048 + 17
    q, k, v, ld, s0 = _la_inputs(n, 1, 1, d, d, dtype, 77)
    S = s0.clone()
    o = torch.empty(n, 1, 1, d, dtype=DT[dtype], device="cuda")
    fi.linattn_prefill(q, k, v, ld, o, state_in=S, state_out=S, scale=d ** -0.5)
    torch.cuda.synchronize()
    _check_la(o, S, q, k, v, ld, d ** -0.5, s0, None, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prefill_extreme_decays(fi, dtype):
    # none, almost none, strong, below the smallest normal number per position,
    # and a decay of zero; a positive logarithm counts as no decay
    n, d = 300, 128
    ld = torch.tensor([0.0, -1e-7, -3.0, -100.0, -math.inf, 2.0], device="cuda")
    H = ld.numel()
    q, k, v, _, s0 = _la_inputs(n, 1, H, d, d, dtype, 11)
    o = torch.empty(n, 1, H, d, dtype=DT[dtype], device="cuda")
    S = torch.empty_like(s0)
    fi.linattn_prefill(q, k, v, ld, o, state_in=s0, state_out=S, scale=d ** -0.5)
    torch.cuda.synchronize()
    assert torch.isfinite(o).all() and torch.isfinite(S).all()
    _check_la(o, S, q, k, v, ld, d ** -0.5, s0, None, dtype)


def test_prefill_without_positions_or_outputs(fi):
    q, k, v, ld, s0 = _la_inputs(3, 2, 2, 64, 64, "f32", 3)
    S = torch.empty_like(s0)
    o = torch.empty(0, 2, 2, 64, device="cuda")
    fi.linattn_prefill(q[:0], k[:0], v[:0], ld, o, state_in=s0, state_out=S)
    torch.cuda.synchronize()
    assert torch.equal(S, s0)
    fi.linattn_prefill(q[:0], k[:0], v[:0], ld, o, state_out=S)
    torch.cuda.synchronize()
    assert torch.all(S == 0)
    o = torch.empty(3, 2, 2, 64, device="cuda")
    fi.linattn_prefill(q, k, v, ld, o)       # no states at all
    torch.cuda.synchronize()
    _check_la(o, None, q, k, v, ld, 1.0, None, None, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,d", [(700, 64), (700, 128)])
def test_prefill_does_not_look_ahead(fi, n, d, dtype):
    # what comes later changes no earlier output, bit for bit
    q, k, v, ld, _ = _la_inputs(n, 1, 2, d, d, dtype, 21)
    o1 = torch.empty(n, 1, 2, d, dtype=DT[dtype], device="cuda")
    o2 = torch.empty_like(o1)
    fi.linattn_prefill(q, k, v, ld, o1)
    cut = 450
    for t in (q, k, v):
        t[cut:] *= -3
    fi.linattn_prefill(q, k, v, ld, o2)
    torch.cuda.synchronize()
    assert torch.equal(o1[:cut], o2[:cut]) and not torch.equal(o1[cut:], o2[cut:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prefill_not_finite_values(fi, dtype):
    # NaN at a position: its outputs and all later ones of that sequence and head
    # are NaN, other sequences and heads are untouched, and so is what ends at
    # least 127 positions before it
    n, B, H, d = 400, 2, 2, 64
    q, k, v, ld, _ = _la_inputs(n, B, H, d, d, dtype, 31)
    ld = torch.full_like(ld, -0.01)
    o1 = torch.empty(n, B, H, d, dtype=DT[dtype], device="cuda")
    o2, S = torch.empty_like(o1), torch.empty(B, H, d, d, device="cuda")
    fi.linattn_prefill(q, k, v, ld, o1)
    at = 260
    v[at, 1, 0] = math.nan
    fi.linattn_prefill(q, k, v, ld, o2, state_out=S)
    torch.cuda.synchronize()
    assert torch.isnan(o2[at:, 1, 0]).all() and torch.isnan(S[1, 0]).all()
    assert torch.equal(o1[: at - 127, 1, 0], o2[: at - 127, 1, 0])
    assert torch.equal(o1[:, 0], o2[:, 0]) and torch.equal(o1[:, 1, 1], o2[:, 1, 1])
    assert torch.isfinite(S[0]).all() and torch.isfinite(S[1, 1]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prefill_lengths_are_clamped(fi, dtype):
    n = 140
    q, k, v, ld, s0 = _la_inputs(n, 3, 1, 64, 64, dtype, 61)
    outs = []
    for lens in ([-7, 10 ** 6, 90], [0, n, 90]):
        o, S = torch.zeros(n, 3, 1, 64, dtype=DT[dtype], device="cuda"), torch.empty_like(s0)
        fi.linattn_prefill(q, k, v, ld, o, state_in=s0, state_out=S, lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        outs.append((o, S))
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert torch.equal(outs[0][1][0], s0[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1])
def test_prefill_positions_far_apart(fi, shift, dtype):
    # element offsets beyond 2^31, at 16-byte boundaries and not
    n, H, d = 280, 2, 32
    ld = (1 << 23) + 8
    g = torch.Generator(device="cuda").manual_seed(8)

    def far():
        t = torch.empty(n * ld + 8, dtype=DT[dtype], device="cuda")[shift:].as_strided((n, 1, H, d), (ld, ld, d, 1))
        t.copy_(_rand(g, n, 1, H, d))
        return t

    q, k, v, o = far(), far(), far(), far()
    ld_ = torch.log(torch.tensor([0.9, 0.99], device="cuda"))
    S = torch.empty(1, H, d, d, device="cuda")
    fi.linattn_prefill(q, k, v, ld_, o, state_out=S)
    torch.cuda.synchronize()
    _check_la(o, S, q, k, v, ld_, 1.0, None, None, dtype)
    B = n                                          # the positions as sequences: one step for each
    qs, ks, vs, os = (t.transpose(0, 1)[0] for t in (q, k, v, o))
    Ss = torch.zeros(B, H, d, d, device="cuda")
    fi.linattn_step(qs, ks, vs, ld_, Ss, os)
    torch.cuda.synchronize()
    want = np.einsum("bhd,bhd->bh", _f64(qs), _f64(ks))[..., None] * _f64(vs)
    A = np.einsum("bhd,bhd->bh", np.abs(_f64(qs)), np.abs(_f64(ks)))[..., None] * np.abs(_f64(vs))
    assert np.all(np.abs(_f64(os) - want) <= (d + 16) * U32 * A + (U16 * np.abs(want) if dtype == "bf16" else 0))


STEP_CASES = [(1, 1, 64, 64), (2, 3, 128, 128), (5, 9, 56, 104), (3, 2, 1, 1), (2, 2, 33, 47), (1, 2, 256, 256),
              (4, 1, 200, 130), (64, 16, 128, 128), (1, 12, 64, 64), (70, 2, 32, 200)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,dk,dv", STEP_CASES)
def test_step(fi, B, H, dk, dv, dtype):
    q, k, v, ld, s0 = _la_inputs(1, B, H, dk, dv, dtype, 13 * B + dk, fused=True)
    S = s0.clone()
    o = torch.empty(B, H, dv, dtype=DT[dtype], device="cuda")
    scale = dk ** -0.5
    fi.linattn_step(q[0], k[0], v[0], ld, S, o, scale=scale)
    torch.cuda.synchronize()
    q64, k64, v64, s64 = _f64(q[0]), _f64(k[0]), _f64(v[0]), _f64(s0)
    g = np.exp(_f64(ld))[:, None, None]
    want_S = g * s64 + k64[..., :, None] * v64[..., None, :]
    want_o = scale * np.einsum("bhd,bhde->bhe", q64, want_S)
    A = scale * np.einsum("bhd,bhde->bhe", np.abs(q64), g * np.abs(s64) + np.abs(k64[..., :, None] * v64[..., None, :]))
    A_S = g * np.abs(s64) + np.abs(k64[..., :, None] * v64[..., None, :])
    assert np.all(np.abs(_f64(S) - want_S) <= 16 * U32 * A_S)
    tol = (dk + 16) * U32 * A + (U16 * np.abs(want_o) if dtype == "bf16" else 0)
    assert np.all(np.abs(_f64(o) - want_o) <= tol)


def test_step_state_at_odd_addresses(fi):
    # a state that starts 4 bytes after a 16-byte boundary
    q, k, v, ld, s0 = _la_inputs(1, 2, 2, 64, 64, "f32", 4)
    buf = torch.empty(s0.numel() + 1, device="cuda")
    S = buf[1:].view_as(s0)
    S.copy_(s0)
    o, o2, S2 = torch.empty(2, 2, 64, device="cuda"), torch.empty(2, 2, 64, device="cuda"), s0.clone()
    fi.linattn_step(q[0], k[0], v[0], ld, S, o)
    fi.linattn_step(q[0], k[0], v[0], ld, S2, o2)
    torch.cuda.synchronize()
    assert torch.equal(S, S2)
    assert torch.allclose(o, o2, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_steps_continue_a_prompt(fi, dtype):
    # a prompt of 70, then 10 single tokens: the same as a prompt of 80
    n, p, B, H, d = 80, 70, 2, 3, 64
    q, k, v, ld, s0 = _la_inputs(n, B, H, d, d, dtype, 41)
    S = s0.clone()
    o = torch.empty(n, B, H, d, dtype=DT[dtype], device="cuda")
    fi.linattn_prefill(q[:p], k[:p], v[:p], ld, o[:p], state_in=S, state_out=S, scale=0.125)
    for t in range(p, n):
        fi.linattn_step(q[t], k[t], v[t], ld, S, o[t], scale=0.125)
    torch.cuda.synchronize()
    _check_la(o, S, q, k, v, ld, 0.125, s0, None, dtype)


# ------------------------------------------------------------------ linear layer

def _check_linear(y, x, w, b, r, act, dtype):
    f = lambda t: None if t is None else _f64(t)   # noqa: E731
    want = ops.linear(f(x), f(w), f(b), f(r), act)
    A = np.abs(f(x)) @ np.abs(f(w)).T + (np.abs(f(b)) if b is not None else 0)
    # GELU and SiLU have slopes of at most 1.13 and 1.1, the others 1; their own
    # evaluation in fp32 is within 8 roundings of a value of at most |u| (tanh: 1)
    slope = {"gelu": 1.13, "silu": 1.1}.get(act, 1.0)
    tol = slope * (x.shape[1] + 16) * U32 * A + 8 * U32 * (1 + np.abs(want))
    if r is not None:
        tol = tol + U32 * np.abs(f(r))
    if dtype == "bf16":
        tol = tol + U16 * np.abs(want)
    err = np.abs(_f64(y) - want)
    assert np.all(err <= tol), (err - tol).max()
    norm = np.linalg.norm(want)
    if norm > 0 and want.size >= 64:
        # root mean square: a rounding of the result; sums, where the roundings of a
        # sum of K add like a walk of sqrt(K) steps
        rms = (U16 if dtype == "bf16" else 0) * norm + 4 * math.sqrt(x.shape[1] + 16) * U32 * slope * np.linalg.norm(A) / math.sqrt(x.shape[1])
        assert np.linalg.norm(err) <= rms + 8 * U32 * norm


LIN_CASES = [
    # n, in, out, act, bias, residual
    (1, 1, 1, "none", False, False),
    (1, 64, 64, "gelu", True, False),
    (1, 2048, 520, "none", True, True),
    (2, 100, 33, "silu", True, True),
    (7, 865, 129, "tanh", True, True),
    (16, 256, 128, "relu", True, False),
    (17, 512, 300, "none", False, True),
    (33, 64, 1000, "gelu", True, True),
    (64, 2048, 256, "none", True, True),
    (65, 96, 257, "gelu", True, True),
    (100, 768, 768, "none", False, False),
    (127, 72, 200, "silu", False, True),
    (129, 136, 264, "tanh", True, False),
    (200, 63, 65, "relu", True, True),
    (256, 1024, 512, "gelu", True, True),
    (300, 864, 865, "none", True, True),
    (513, 33, 2000, "none", True, False),
    (1000, 200, 130, "gelu", True, True),
    (1777, 96, 1728, "tanh", True, True),          # one round of tiles
    (2304, 64, 4096, "none", False, True),         # several rounds
    (4100, 72, 2049, "relu", True, False),
    (3, 100, 5000, "none", True, True),
    (8, 1030, 5001, "relu", False, True),
    (9, 1000, 300, "silu", True, False),
    (31, 700, 200, "none", True, True),
    (40, 8200, 100, "none", False, False),
    (128, 512, 384, "tanh", False, True),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,nin,nout,act,bias,residual", LIN_CASES)
def test_linear(fi, n, nin, nout, act, bias, residual, dtype):
    g = torch.Generator(device="cuda").manual_seed(n + 3 * nin + 5 * nout)
    dt = DT[dtype]
    x, w = _rand(g, n, nin, dtype=dt), _rand(g, nout, nin, dtype=dt, scale=nin ** -0.5)
    b = _rand(g, nout, dtype=dt) if bias else None
    r = _rand(g, n, nout, dtype=dt) if residual else None
    guard = torch.full((n * nout + 64,), 7.0, dtype=dt, device="cuda")
    y = guard[: n * nout].view(n, nout)
    fi.linear(x, w, y, bias=b, residual=r, act=act)
    torch.cuda.synchronize()
    assert torch.all(guard[n * nout:] == 7.0)
    _check_linear(y, x, w, b, r, act, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [3, 40, 200])
@pytest.mark.parametrize("shift", [0, 1])
def test_linear_views_and_residual_in_place(fi, n, shift, dtype):
    # columns of wider buffers (aligned or one element off), the residual read
    # from and the result written to the same rows, nothing beside them touched
    g = torch.Generator(device="cuda").manual_seed(n + shift)
    dt = DT[dtype]
    nin, nout = 192, 136
    X, W, Y = _rand(g, n, 320, dtype=dt), _rand(g, nout, 256, dtype=dt, scale=nin ** -0.5), _rand(g, n, 320, dtype=dt)
    x, w, y = X[:, shift:shift + nin], W[:, shift:shift + nin], Y[:, 64 + shift:64 + shift + nout]
    before, r = Y.clone(), y.clone()
    fi.linear(x, w, y, residual=y, act="gelu")
    torch.cuda.synchronize()
    _check_linear(y, x, w, None, r, "gelu", dtype)
    before[:, 64 + shift:64 + shift + nout] = y
    assert torch.equal(Y, before)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_shared_rows(fi, dtype):
    # one row of x and one of the residual for all rows (strides of 0)
    g = torch.Generator(device="cuda").manual_seed(9)
    dt = DT[dtype]
    x, w = _rand(g, 1, 128, dtype=dt).expand(150, 128), _rand(g, 72, 128, dtype=dt, scale=0.1)
    r = _rand(g, 1, 72, dtype=dt).expand(150, 72)
    y = torch.empty(150, 72, dtype=dt, device="cuda")
    fi.linear(x, w, y, residual=r)
    torch.cuda.synchronize()
    _check_linear(y, x, w, None, r, "none", dtype)
    assert torch.equal(y, y[:1].expand_as(y))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 50, 300])
def test_linear_not_finite_rows_stay_apart(fi, n, dtype):
    # a NaN or infinity in one row of x reaches that row of y only
    g = torch.Generator(device="cuda").manual_seed(17)
    dt = DT[dtype]
    x, w = _rand(g, n + 2, 200, dtype=dt), _rand(g, 90, 200, dtype=dt, scale=0.1)
    y1, y2 = torch.empty(n + 2, 90, dtype=dt, device="cuda"), torch.empty(n + 2, 90, dtype=dt, device="cuda")
    fi.linear(x, w, y1)
    x[n // 2, 5], x[n + 1, 7] = math.nan, math.inf
    fi.linear(x, w, y2)
    torch.cuda.synchronize()
    assert torch.isnan(y2[n // 2]).all() and not torch.isfinite(y2[n + 1]).any()
    keep = torch.ones(n + 2, dtype=torch.bool, device="cuda")
    keep[n // 2] = keep[n + 1] = False
    assert torch.equal(y1[keep], y2[keep])


def test_linear_no_rows(fi):
    x, w, y = (torch.empty(s, device="cuda") for s in ((0, 8), (4, 8), (0, 4)))
    fi.linear(x, w, y)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 5, 40, 200])
def test_linear_rows_far_apart(fi, n, dtype):
    # element offsets beyond 2^31 in x, w, residual and y
    g = torch.Generator(device="cuda").manual_seed(n)
    dt = DT[dtype]
    ld, nin, nout = (1 << 24) + 8, 72, 130
    far = max(n, nout)

    def rows(count, cols, scale=1.0):
        t = torch.empty(far * ld, dtype=dt, device="cuda").as_strided((count, cols), (ld, 1))
        t.copy_(_rand(g, count, cols, scale=scale))
        return t

    x, w, r, y = rows(n, nin), rows(nout, nin, nin ** -0.5), rows(n, nout), rows(n, nout)
    fi.linear(x, w, y, residual=r, act="relu")
    torch.cuda.synchronize()
    _check_linear(y, x, w, None, r, "relu", dtype)


# ------------------------------------------------------------------ refusals of the binding

def test_binding_refusals(fi):
    q, k, v, ld, s0 = _la_inputs(4, 2, 2, 64, 64, "f32", 1)
    o = torch.empty_like(v)
    for bad in (
        lambda: fi.linattn_prefill(q, k[:3], v, ld, o),
        lambda: fi.linattn_prefill(q, k, v, ld, o.bfloat16()),
        lambda: fi.linattn_prefill(q, k, v.bfloat16(), ld, o),
        lambda: fi.linattn_prefill(q.half(), k.half(), v.half(), ld, o.half()),
        lambda: fi.linattn_prefill(q.transpose(2, 3).contiguous().transpose(2, 3), k, v, ld, o),
        lambda: fi.linattn_prefill(q, k, v, ld[:1], o),
        lambda: fi.linattn_prefill(q, k, v, ld.double(), o),
        lambda: fi.linattn_prefill(q, k, v, ld, o, state_out=s0.bfloat16()),
        lambda: fi.linattn_prefill(q, k, v, ld, o, state_in=s0.transpose(2, 3)),
        lambda: fi.linattn_prefill(q, k, v, ld, o, lengths=torch.tensor([1, 2], device="cuda")),
        lambda: fi.linattn_prefill(q, k, v, ld, o, lengths=torch.tensor([1], dtype=torch.int32, device="cuda")),
        lambda: fi.linattn_step(q, k, v, ld, s0, o),
        lambda: fi.linattn_step(q[0], k[0], v[0], ld, s0[:1], o[0]),
        lambda: fi.linear(q[:, 0, 0], q[:, 0, 0, :32], torch.empty(4, 4, device="cuda")),
        lambda: fi.linear(q[:, 0, 0], k[:, 0, 0], torch.empty(4, 4, device="cuda"), act="elu"),
        lambda: fi.linear(q[:, 0, 0], k[:, 0, 0], torch.empty(4, 4, device="cuda"), bias=torch.zeros(3, device="cuda")),
        lambda: fi.linear(q[:, 0, 0], k[:, 0, 0], torch.empty(4, 4, device="cuda"), residual=torch.zeros(1, 4, device="cuda")),
        lambda: fi.linear(q[:, 0, 0], k[:, 0, 0].bfloat16(), torch.empty(4, 4, device="cuda")),
    ):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(fi.FiError):
        fi.linattn_prefill(q, k, v, ld, o[:1].expand(4, 2, 2, 64))      # rows of o overlap
    y = torch.empty(4, 4, device="cuda")
    with pytest.raises(fi.FiError):
        fi.linear(y, y.clone(), y)


# ------------------------------------------------------------------ streams and graphs

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_graph_replays_with_new_inputs(fi, dtype):
    # a prompt, a step and a linear layer in one graph; replayed on other inputs
    # written into the same buffers, it gives what eager calls give, bit for bit
    n, B, H, d = 900, 1, 2, 64
    q, k, v, ld, s0 = _la_inputs(n, B, H, d, d, dtype, 51)
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(52)
    w = _rand(g, 96, H * d, dtype=dt, scale=0.1)
    o, S = torch.empty(n, B, H, d, dtype=dt, device="cuda"), torch.empty_like(s0)
    o1, y = torch.empty(B, H, d, dtype=dt, device="cuda"), torch.empty(n, 96, dtype=dt, device="cuda")
    y1 = torch.empty(B, 96, dtype=dt, device="cuda")

    def run():
        fi.linattn_prefill(q, k, v, ld, o, state_in=s0, state_out=S, scale=0.1)
        fi.linear(o.view(n, H * d), w, y, act="silu")
        fi.linattn_step(q[0], k[0], v[0], ld, S, o1, scale=0.1)
        fi.linear(o1.view(B, H * d), w, y1)
        return [t.clone() for t in (o, S, y, o1, y1)]

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in (1, 2):
        q2, k2, v2, _, s2 = _la_inputs(n, B, H, d, d, dtype, 60 + seed)
        for a, b in ((q, q2), (k, k2), (v, v2), (s0, s2)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (o, S, y, o1, y1)]
        want = run()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_graphs_with_scratch_at_once(fi):
    # two captured graphs whose calls need scratch (fp32 operands), replayed on two
    # streams at the same time, give what they give one after the other
    g = torch.Generator(device="cuda").manual_seed(4)
    graphs, outs, runs = [], [], []          # a graph's tensors live as long as it does
    for i in range(2):
        x, w, y = _rand(g, 700, 500), _rand(g, 300, 500, scale=0.05), torch.empty(700, 300, device="cuda")
        q, k, v, ld, s0 = _la_inputs(1500, 1, 2, 64, 64, "f32", 90 + i)
        o, S = torch.empty_like(v), torch.empty_like(s0)

        def run(x=x, w=w, y=y, q=q, k=k, v=v, ld=ld, s0=s0, o=o, S=S):
            fi.linear(x, w, y, act="gelu")
            fi.linattn_prefill(q, k, v, ld, o, state_in=s0, state_out=S)

        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graphs.append(graph)
        runs.append(run)
        outs.append((y, o, S))
    want = []
    for graph, out in zip(graphs, outs):
        graph.replay()
        torch.cuda.synchronize()
        want.append([t.clone() for t in out])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for out in outs:
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            for s, t in zip(a, b):
                assert torch.equal(s, t)
    fi.op_sync()


def test_a_context_reads_what_an_operator_has_just_written(fi):
    # the noise of a generation comes from a linear layer launched right before it; the
    # generation's first kernel reads noise before it waits for the launch ahead of it
    g = torch.Generator(device="cuda").manual_seed(12)
    M, D, L, B, n = 2, 64, 256, 16, 256
    h = torch.randn(M, D, L, generator=g, device="cuda") * torch.exp(-0.2 * torch.arange(L, device="cuda"))
    x, w = _rand(g, n * B, 2048), _rand(g, D, 2048, scale=0.02)
    x0 = _rand(g, B, D)
    ys = []
    for wait in (True, False, False):
        ctx = fi.Context(h, B, "f32")
        eps, y = torch.zeros(n, B, D, device="cuda"), torch.empty(n, B, D, device="cuda")
        torch.cuda.synchronize()
        fi.linear(x, w, eps.view(n * B, D))
        if wait:
            torch.cuda.synchronize()
        ctx.generate(n, x0, eps, y, 0.1)
        ctx.sync()
        ctx.close()
        ys.append(y)
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


def test_scratch_that_is_too_small_is_refused(fi):
    import ctypes
    x = torch.empty(300, 64, device="cuda")
    cfg = fi.LinearConfig(64, 300, fi.FI_F32, 0, 64, 64, 300, 300)
    y = torch.empty(300, 300, device="cuda")
    need = ctypes.c_uint64()
    at, p = ctypes.addressof(cfg), x.data_ptr()
    assert fi.lib.fi_linear_workspace(at, 300, p, p, ctypes.byref(need)) == fi.FI_OK and need.value > 0
    ws = torch.empty(need.value + 256, dtype=torch.uint8, device="cuda")
    for ptr, size in ((None, need.value), (ws.data_ptr(), need.value - 1), (ws.data_ptr() + 16, need.value)):
        assert fi.lib.fi_linear(at, 300, p, p, None, None, y.data_ptr(), ptr, size, None) == fi.FI_E_INVALID
        assert "workspace" in fi.lib.fi_last_error().decode()
    la = fi.LinattnConfig(1, 64, 64, 1, fi.FI_F32, 1.0)
    for name in ("q_stride", "k_stride", "v_stride", "o_stride"):
        getattr(la, name)[:] = (64, 64, 64)
    assert fi.lib.fi_linattn_workspace(ctypes.addressof(la), 300, p, p, p, ctypes.byref(need)) == fi.FI_OK and need.value > 0
    ld = torch.zeros(1, device="cuda")
    assert fi.lib.fi_linattn_prefill(ctypes.addressof(la), 300, p, p, p, ld.data_ptr(), None, None, None, y.data_ptr(),
                                     ws.data_ptr(), need.value - 1, None) == fi.FI_E_INVALID
    assert "workspace" in fi.lib.fi_last_error().decode()


def test_calls_on_two_streams_at_once(fi):
    # the same calls on two streams, in turn, give the results of one stream
    sets = [_la_inputs(1500, 1, 2, 64, 64, "bf16", 70 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]

    def run(i, stream):
        q, k, v, ld, s0 = sets[i]
        o, S = torch.empty_like(v), torch.empty_like(s0)
        fi.linattn_prefill(q, k, v, ld, o, state_in=s0, state_out=S, stream=stream)
        y = torch.empty(1500, 48, dtype=torch.bfloat16, device="cuda")
        fi.linear(o.view(1500, 128), q.reshape(1500, 128)[:48], y, stream=stream)
        return o, S, y

    want = [run(i, None) for i in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        got.append([run(i, streams[i]) for i in range(2)])
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            for s, t in zip(a, b):
                assert torch.equal(s, t)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_layer_of_a_hybrid_stack(fi, dtype):
    # projections, linear attention, output projection with the residual, and the
    # block's two products: a prompt, then single tokens, against the same layer
    # in float64 on the inputs as rounded between the calls
    n, p, B, H, d = 150, 140, 2, 2, 64
    D, Dh = H * d, 160
    g = torch.Generator(device="cuda").manual_seed(99)
    dt = DT[dtype]
    wqkv, wo = _rand(g, 3 * D, D, dtype=dt, scale=D ** -0.5), _rand(g, D, D, dtype=dt, scale=D ** -0.5)
    w1, b1 = _rand(g, Dh, D, dtype=dt, scale=D ** -0.5), _rand(g, Dh, dtype=dt, scale=0.1)
    w2, b2 = _rand(g, D, Dh, dtype=dt, scale=Dh ** -0.5), _rand(g, D, dtype=dt, scale=0.1)
    x = _rand(g, n, B, D, dtype=dt)
    ld = torch.log(torch.tensor([0.9, 0.99], device="cuda"))
    S = torch.zeros(B, H, d, d, device="cuda")

    def layer(xs):
        m = xs.shape[0]
        flat = xs.reshape(m * B, D)
        qkv = torch.empty(m * B, 3 * D, dtype=dt, device="cuda")
        fi.linear(flat, wqkv, qkv)
        q, k, v = (t.unflatten(-1, (H, d)) for t in qkv.view(m, B, 3 * D).split(D, dim=-1))
        o = torch.empty(m, B, H, d, dtype=dt, device="cuda")
        if m > 1:
            fi.linattn_prefill(q, k, v, ld, o, state_in=S, state_out=S, scale=d ** -0.5)
        else:
            fi.linattn_step(q[0], k[0], v[0], ld, S, o[0], scale=d ** -0.5)
        a, hid, y = torch.empty_like(flat), torch.empty(m * B, Dh, dtype=dt, device="cuda"), torch.empty_like(flat)
        fi.linear(o.view(m * B, D), wo, a, residual=flat)
        fi.linear(a, w1, hid, bias=b1, act="gelu")
        fi.linear(hid, w2, y, bias=b2, residual=a)
        return [t.view(m, B, -1) for t in (qkv, o, a, hid, y)]

    parts = [layer(x[:p])] + [layer(x[t:t + 1]) for t in range(p, n)]
    torch.cuda.synchronize()
    qkv, o, a, hid, y = (torch.cat(t) for t in zip(*parts))
    flat = lambda t: t.reshape(n * B, -1)   # noqa: E731
    q, k, v = (t.unflatten(-1, (H, d)) for t in qkv.split(D, dim=-1))
    _check_linear(flat(qkv), flat(x), wqkv, None, None, "none", dtype)
    _check_la(o.view(n, B, H, d), S, q, k, v, ld, d ** -0.5, None, None, dtype)
    _check_linear(flat(a), flat(o), wo, None, flat(x), "none", dtype)
    _check_linear(flat(hid), flat(a), w1, b1, None, "gelu", dtype)
    _check_linear(flat(y), flat(hid), w2, b2, flat(a), "none", dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,nin,nout", [(200, 2048, 128), (300, 2048, 769), (513, 1537, 200), (257, 4100, 33), (129, 256, 2100),
                                        (1000, 1600, 384)])
@pytest.mark.parametrize("act,bias,residual", [("none", False, False), ("tanh", True, True)])
def test_linear_shared_contraction(fi, n, nin, nout, act, bias, residual, dtype):
    # few tiles and a long contraction: several pairs of CTAs work on a tile
    g = torch.Generator(device="cuda").manual_seed(n + nin)
    dt = DT[dtype]
    x, w = _rand(g, n, nin, dtype=dt), _rand(g, nout, nin, dtype=dt, scale=nin ** -0.5)
    b = _rand(g, nout, dtype=dt) if bias else None
    r = _rand(g, n, nout, dtype=dt) if residual else None
    y = torch.full((n + 1, nout), float("nan"), dtype=dt, device="cuda")
    fi.linear(x, w, y[:n], bias=b, residual=r, act=act)
    again = torch.empty(n, nout, dtype=dt, device="cuda")
    fi.linear(x, w, again, bias=b, residual=r, act=act)
    fi.op_sync()
    _check_linear(y[:n], x, w, b, r, act, dtype)
    assert torch.equal(again, y[:n])
    assert y[n].isnan().all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,nin,nout", [(300, 512, 300), (300, 2048, 300), (2000, 96, 225)])
@pytest.mark.parametrize("sy,sr,dy,dr", [(0, 0, 8, 8), (1, 0, 3, 0), (0, 3, 0, 1), (5, 2, 2, 7), (7, 7, 1, 1), (6, 1, 8, 5)])
def test_linear_rows_at_any_alignment(fi, n, nin, nout, sy, sr, dy, dr, dtype):
    # y and the residual start sy, sr elements past a 16-byte boundary, their rows are
    # dy, dr elements longer than a row; what lies between the rows stays as it was
    g = torch.Generator(device="cuda").manual_seed(100 * sy + sr)
    dt = DT[dtype]
    x, w = _rand(g, n, nin, dtype=dt), _rand(g, nout, nin, dtype=dt, scale=nin ** -0.5)
    b = _rand(g, nout, dtype=dt)

    def view(shift, more):
        base = torch.full((n * (nout + more) + 16,), 7.0, dtype=dt, device="cuda")
        return base, base[shift:shift + n * (nout + more)].view(n, nout + more)[:, :nout]

    ybase, y = view(sy, dy)
    rbase, r = view(sr, dr)
    r.copy_(_rand(g, n, nout, dtype=dt))
    fi.linear(x, w, y, bias=b, residual=r, act="silu")
    fi.op_sync()
    _check_linear(y, x, w, b, r, "silu", dtype)
    y.fill_(7.0)
    assert (ybase == 7.0).all()
    # in place
    want = torch.empty(n, nout, dtype=dt, device="cuda")
    fi.linear(x, w, want, bias=b, residual=r, act="silu")
    fi.linear(x, w, r, bias=b, residual=r, act="silu")
    fi.op_sync()
    assert torch.equal(r, want)
    r.fill_(7.0)
    assert (rbase == 7.0).all()


@pytest.mark.parametrize("op", ["linear", "prefill"])
def test_scratch_of_a_call_on_another_stream(fi, op):
    # memory that work still waiting on the current stream uses is not scratch of a call
    # that goes ahead on another one
    g = torch.Generator(device="cuda").manual_seed(3)
    x, w, y = _rand(g, 1024, 512), _rand(g, 512, 512), torch.empty(1024, 512, device="cuda")
    q, k, v = (_rand(g, 512, 4, 4, 64) for _ in range(3))
    o, ld = torch.empty_like(v), torch.full((4,), -0.1, device="cuda")
    other = torch.cuda.Stream()

    def call(stream):
        if op == "linear":
            fi.linear(x, w, y, stream=stream)
        else:
            fi.linattn_prefill(q, k, v, ld, o, stream=stream)

    call(other.cuda_stream)                 # the kernels are loaded
    torch.cuda.synchronize()
    sizes = [need for _, need, _ in fi._configs.values() if need > 0]
    torch.cuda.empty_cache()
    held = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)           # some 10 ms
    kept = [h.clone() for h in held]
    del held
    call(other.cuda_stream)
    torch.cuda.synchronize()
    assert all((h == 7).all() for h in kept)


def test_sizes_beyond_32_bits_are_refused(fi):
    # shapes of which only one element exists: 2^32 + 5 would pass as 5
    big = 2 ** 32 + 5
    one = torch.zeros(1, 1, device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        fi.linear(one.expand(big, 1), one.expand(1, 1), one.expand(big, 1))
    with pytest.raises(ValueError, match="2\\^31"):
        fi.linear(one.expand(1, big), one.expand(1, big), one)
    with pytest.raises(ValueError, match="2\\^31"):
        fi.linear(one, one.expand(big, 1), one.expand(1, big))
    x = torch.zeros(1, 1, 1, 1, device="cuda")
    ld, S = torch.zeros(1, device="cuda"), torch.zeros(1, 1, 1, 1, device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        t = x.expand(big, 1, 1, 1)
        fi.linattn_prefill(t, t, t, ld, t)
    with pytest.raises(ValueError, match="2\\^31"):
        t = x[0].expand(big, 1, 1)
        fi.linattn_step(t, t, t, ld, S, t)


@pytest.mark.parametrize("n,B,H,dk,dv,fused,lens,carried", [
    (300, 2, 2, 65, 129, False, [300, 131], True),       # blocks of one dimension, odd rows of the state
    (1000, 1, 2, 130, 70, True, None, True),             # several segments
    (1300, 2, 1, 256, 256, False, [1300, 0], True),
    (129, 3, 1, 100, 40, True, [1, 129, 128], False),
    (700, 1, 1, 40, 200, False, None, True),
    (150, 90, 1, 72, 130, False, None, False),           # more blocks than SMs
])
def test_prefill_fp32_in_blocks_of_dimensions(fi, n, B, H, dk, dv, fused, lens, carried):
    q, k, v, ld, s0 = _la_inputs(n, B, H, dk, dv, "f32", n + dv, fused)
    lengths = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    if lens is not None:
        for b, m in enumerate(lens):
            for t in (q, k, v):
                t[m:, b] = math.nan
    base = torch.full((n, B, H, dv + 3), 7.0, device="cuda")
    o = base[..., 1:dv + 1]                               # rows at no 16-byte boundary
    state = s0.clone() if carried else torch.full_like(s0, math.nan)
    fi.linattn_prefill(q, k, v, ld, o, state_in=state if carried else None, state_out=state, lengths=lengths, scale=dk ** -0.5)
    again, S = torch.full((n, B, H, dv), 7.0, device="cuda"), torch.empty_like(s0)
    fi.linattn_prefill(q, k, v, ld, again, state_in=s0 if carried else None, state_out=S, lengths=lengths, scale=dk ** -0.5)
    fi.op_sync()
    assert torch.equal(o, again) and torch.equal(state, S)
    assert (base[..., 0] == 7.0).all() and (base[..., dv + 1:] == 7.0).all()
    if lens is not None:
        for b, m in enumerate(lens):
            assert (o[m:, b] == 7.0).all()
            o[m:, b] = 0
            for t in (q, k, v):
                t[m:, b] = 0
    _check_la(o, state, q, k, v, ld, dk ** -0.5, s0 if carried else None, lens, "f32")
