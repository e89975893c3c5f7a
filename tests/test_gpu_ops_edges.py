"""Linear attention and the linear layer on the GPU at the edges of what their calls allow:
rows that end inside a warp, padded outputs, decays of zero, tails of the activations,
values near the largest number, many sequences, waits that give up, several threads.

Tolerances are those of test_gpu_ops.py where nothing else is said.
"""
import math

import numpy as np
import pytest

from oracle import ops
from test_gpu_ops import DT, U16, U32, _check_la, _check_linear, _f64, _la_inputs, _rand, fi  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,pad,shift", [(64, 8, 0), (64, 3, 1), (128, 8, 0), (100, 1, 0), (33, 2, 0), (33, 7, 0), (20, 4, 0)])
def test_prefill_sequences_that_end_inside_a_warp(fi, d, pad, shift, dtype):  # noqa: F811
    # lengths at which the lanes of one warp stand on both sides of the end, at first,
    # middle and last rows of chunks; what lies between the rows of o, before the first and
    # behind the last one stays as it was
    lens = [1, 31, 33, 70, 97, 127, 129, 255, 300]
    n, B, H = 300, len(lens), 2
    q, k, v, ld, s0 = _la_inputs(n, B, H, d, d, dtype, 17 * d + pad)
    base = torch.full((n * B * H * (d + pad) + shift + 16,), 7.0, dtype=DT[dtype], device="cuda")
    o = base[shift:shift + n * B * H * (d + pad)].view(n, B, H, d + pad)[..., :d]
    for b, m in enumerate(lens):
        for t in (q, k, v):
            t[m:, b] = math.nan
    S = torch.empty_like(s0)
    fi.linattn_prefill(q, k, v, ld, o, state_in=s0, state_out=S, scale=d ** -0.5,
                       lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    fi.op_sync()
    got = torch.zeros(n, B, H, d, dtype=DT[dtype], device="cuda")
    for b, m in enumerate(lens):
        got[:m, b] = o[:m, b]
        o[:m, b] = 7.0
        for t in (q, k, v):
            t[m:, b] = 0
    assert (base == 7.0).all()
    _check_la(got, S, q, k, v, ld, d ** -0.5, s0, lens, dtype)


@pytest.mark.parametrize("n", [128, 300])
@pytest.mark.parametrize("dk,dv,pad", [(33, 33, 7), (20, 20, 4), (100, 100, 4), (128, 121, 7), (61, 64, 8), (40, 65, 7)])
def test_prefill_bf16_rows_padded_to_16_bytes(fi, n, dk, dv, pad):  # noqa: F811
    # rows whose elements end inside a unit of 16 bytes at 16-byte strides: what pads the
    # rows of o stays as it was, what pads those of q, k and v (NaN) is not used
    B, H = 2, 2
    g = torch.Generator(device="cuda").manual_seed(n + dk + dv)

    def padded(d, fill):
        base = torch.full((n, B, H, (d + 7) // 8 * 8), fill, dtype=torch.bfloat16, device="cuda")
        return base, base[..., :d]

    q, k, v = padded(dk, math.nan)[1], padded(dk, math.nan)[1], padded(dv, math.nan)[1]
    for t in (q, k, v):
        t.copy_(_rand(g, *t.shape))
    base = torch.full((n, B, H, dv + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    o = base[..., :dv]
    ld, s0 = torch.tensor([-0.1, -0.01], device="cuda"), _rand(g, B, H, dk, dv)
    S = torch.empty_like(s0)
    fi.linattn_prefill(q, k, v, ld, o, state_in=s0, state_out=S, scale=dk ** -0.5)
    fi.op_sync()
    assert (base[..., dv:] == 7.0).all()
    _check_la(o, S, q, k, v, ld, dk ** -0.5, s0, None, "bf16")


@pytest.mark.parametrize("n", [1, 5, 40, 100, 200, 600])
@pytest.mark.parametrize("nin,nout", [(33, 65), (865, 129), (2001, 300)])
def test_linear_bf16_rows_padded_to_16_bytes(fi, n, nin, nout):  # noqa: F811
    # as above: what pads the rows of x and w (NaN) is not used
    g = torch.Generator(device="cuda").manual_seed(n + nin)

    def padded(rows, cols, scale=1.0):
        base = torch.full((rows, (cols + 7) // 8 * 8), math.nan, dtype=torch.bfloat16, device="cuda")
        base[:, :cols] = _rand(g, rows, cols, scale=scale)
        return base[:, :cols]

    x, w, r = padded(n, nin), padded(nout, nin, nin ** -0.5), padded(n, nout)
    base = torch.full((n, (nout + 7) // 8 * 8), 7.0, dtype=torch.bfloat16, device="cuda")
    y = base[:, :nout]
    fi.linear(x, w, y, residual=r, act="tanh")
    fi.op_sync()
    assert (base[:, nout:] == 7.0).all()
    _check_linear(y, x, w, None, r, "tanh", "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,d", [(1, 64), (130, 64), (130, 128), (2065, 64), (2065, 128), (70, 200), (900, 200)])
def test_a_decay_of_zero_drops_any_state(fi, n, d, dtype):  # noqa: F811
    # infinities and NaN in the state before reach nothing where log_decay is -infinity,
    # and do where the decay only underflows; an empty sequence passes its state on
    H = 3
    q, k, v, _, s0 = _la_inputs(n, 2, H, d, d, dtype, n + d)
    ld = torch.tensor([-math.inf, -math.inf, -200.0], device="cuda")
    s0[:, 0, 3, 5], s0[:, 0, 4, 6], s0[:, 1] = math.inf, math.nan, -math.inf
    lengths = torch.tensor([n, 0], dtype=torch.int32, device="cuda")
    outs = []
    for state in (s0, torch.zeros_like(s0)):
        o, S = torch.zeros(n, 2, H, d, dtype=DT[dtype], device="cuda"), state.clone()
        fi.linattn_prefill(q, k, v, ld, o, state_in=S, state_out=S, lengths=lengths, scale=0.25)
        outs.append((o, S))
    fi.op_sync()
    (o, S), (want_o, want_S) = outs
    assert torch.isfinite(o).all() and torch.equal(o[:, :, :2], want_o[:, :, :2])
    assert torch.isfinite(S[0]).all() and torch.equal(S[0, :2], want_S[0, :2])
    assert torch.equal(S[1].nan_to_num(7.0), s0[1].nan_to_num(7.0)) and torch.equal(S[1].isnan(), s0[1].isnan())
    s0[0, 2, 1, 1] = math.inf
    S = s0.clone()
    fi.linattn_prefill(q, k, v, ld, o, state_in=S, state_out=S, lengths=lengths, scale=0.25)
    fi.op_sync()
    assert not torch.isfinite(S[0, 2, 1, 1]) and torch.isfinite(S[0, :2]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [63, 64, 66])
def test_a_decay_of_zero_drops_any_state_in_a_step(fi, d, dtype):  # noqa: F811
    q, k, v, _, s0 = _la_inputs(1, 2, 3, d, d, dtype, d)
    ld = torch.tensor([-math.inf, -math.inf, -200.0], device="cuda")
    s0[:, 0, 3, 5], s0[:, 0, 4, 6], s0[:, 1], s0[:, 2, 1, 1] = math.inf, math.nan, -math.inf, math.inf
    outs = []
    for state in (s0, torch.zeros_like(s0)):
        o, S = torch.empty(2, 3, d, dtype=DT[dtype], device="cuda"), state.clone()
        fi.linattn_step(q[0], k[0], v[0], ld, S, o)
        outs.append((o, S))
    fi.op_sync()
    assert torch.equal(outs[0][0][:, :2], outs[1][0][:, :2]) and torch.equal(outs[0][1][:, :2], outs[1][1][:, :2])
    assert not torch.isfinite(outs[0][1][:, 2, 1, 1]).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,shift", [(1, 0), (1, 1), (2, 1), (8, 0), (40, 0), (130, 0), (300, 1)])
def test_gelu_of_negative_arguments(fi, n, shift, dtype):  # noqa: F811
    # u Phi(u) at arguments -9 .. -3 to its own size, in every form of the layer. The
    # argument is rounded three times at most (its parts, their sum, the factor of
    # 1 / sqrt 2) and u^2 + 1 times that reaches the result; erfcf is within 4 steps of 2^-23,
    # the fit for bf16 results within 6.3e-7, products and sums around them within 8
    # roundings; the result's own rounding comes last.
    g = torch.Generator(device="cuda").manual_seed(n)
    dt, nin, nout = DT[dtype], 16, 400
    w = torch.zeros(nout, nin, dtype=dt, device="cuda")
    w[:, 3] = (-9.0 + 6.0 * torch.rand(nout, generator=g, device="cuda")).to(dt)
    x = torch.zeros(n * nin + 8, dtype=dt, device="cuda")[shift:shift + n * nin].view(n, nin)
    x[:, 3] = 1.0
    x[1::2, 3] = 0.5
    y = torch.empty(n, nout, dtype=dt, device="cuda")
    fi.linear(x, w, y, act="gelu")
    fi.op_sync()
    u = _f64(x) @ _f64(w).T
    want = u * np.array([0.5 * math.erfc(-t / math.sqrt(2.0)) for t in u.ravel()]).reshape(u.shape)
    tol = (3 * (1 + u * u) + 8 + 8 + 11) * U32 + (U16 if dtype == "bf16" else 0)
    err = np.abs(_f64(y) - want) / np.abs(want)
    assert np.all(err <= tol), (err / tol).max()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["none", "gelu", "silu", "relu", "tanh"])
@pytest.mark.parametrize("n,shift", [(1, 0), (1, 1), (2, 1), (40, 0), (130, 0), (300, 1)])
def test_activations_of_infinities(fi, n, shift, act, dtype):  # noqa: F811
    # bf16: what the formula gives, in every form of the layer. fp32 operands that are not
    # finite make the argument not finite: what the formula gives of it, or of NaN.
    dt, nin, nout = DT[dtype], 16, 40
    x = torch.zeros(n * nin + 8, dtype=dt, device="cuda")[shift:shift + n * nin].view(n, nin)
    x[:, 3] = 1.0
    for value in (math.inf, -math.inf, math.nan):
        w = torch.zeros(nout, nin, dtype=dt, device="cuda")
        w[5, 3] = value
        y = torch.empty(n, nout, dtype=dt, device="cuda")
        fi.linear(x, w, y, act=act)
        fi.op_sync()
        want = {"none": value, "gelu": value if value > 0 else math.nan, "silu": value if value > 0 else math.nan,
                "relu": max(value, 0.0) if value == value else math.nan, "tanh": math.copysign(1.0, value) if value == value else math.nan}[act]
        got = y[:, 5].double()
        same = torch.isnan(got) if math.isnan(want) else got == want
        if dtype == "f32":
            same = same | torch.isnan(got)
        assert same.all(), (value, got)
        y[:, 5] = 0
        assert (y == 0).all()


@pytest.mark.parametrize("n", [1, 9, 40, 130, 300])
def test_linear_fp32_values_near_the_largest(fi, n):  # noqa: F811
    # finite operands above 3.38e38, which round to no finite bf16 value
    g = torch.Generator(device="cuda").manual_seed(n)
    big = torch.finfo(torch.float32).max
    x, w = _rand(g, n, 70), _rand(g, 50, 70)
    x[:, ::3] = big
    x[:, 1::3] = -3.3961775e38
    w *= 2.0 ** -40
    for a, b in ((x, w), (w[:1].expand(n, 70).contiguous(), x[:1].expand(50, 70).contiguous())):
        y = torch.empty(n, 50, device="cuda")
        fi.linear(a, b, y)
        fi.op_sync()
        assert torch.isfinite(y).all()
        _check_linear(y, a, b, None, None, "none", "f32")


@pytest.mark.parametrize("d", [64, 100])
def test_prefill_fp32_values_near_the_largest(fi, d):  # noqa: F811
    q, k, v, ld, s0 = _la_inputs(300, 1, 2, d, d, "f32", d)
    q *= 2.0 ** -30
    k *= 2.0 ** -30
    v[::2], v[1::2] = 3.4e38, -3.3961775e38
    s0[:] = torch.finfo(torch.float32).max
    o, S = torch.empty_like(v), torch.empty_like(s0)
    fi.linattn_prefill(q, k, v, ld, o, state_in=s0, state_out=S, scale=0.125)
    fi.op_sync()
    assert torch.isfinite(o).all()
    _check_la(o, S, q, k, v, ld, 0.125, s0, None, "f32")


@pytest.mark.parametrize("dtype,dk,dv", [("f32", 8, 8), ("bf16", 8, 8), ("bf16", 1, 130), ("f32", 70, 3)])
def test_more_than_65535_sequences_and_heads(fi, dtype, dk, dv):  # noqa: F811
    # 4099 sequences of 16 heads: what smaller batches of them give
    n, B, H = 3, 4099, 16
    q, k, v, ld, s0 = _la_inputs(n, B, H, dk, dv, dtype, dk)
    o, S = torch.empty_like(v), s0.clone()
    fi.linattn_prefill(q, k, v, ld, o, state_in=S, state_out=S, scale=0.5)
    o1 = torch.empty_like(o[0])
    fi.linattn_step(q[0], k[0], v[0], ld, S, o1, scale=0.5)
    for at in (0, 1000, 2000, 3000, 4000):
        part = slice(at, min(at + 1000, B))
        T, p, p1 = s0[part].clone(), torch.empty_like(v[:, part]), torch.empty_like(v[0, part])
        fi.linattn_prefill(q[:, part], k[:, part], v[:, part], ld, p, state_in=T, state_out=T, scale=0.5)
        fi.linattn_step(q[0, part], k[0, part], v[0, part], ld, T, p1, scale=0.5)
        fi.op_sync()
        assert torch.equal(p, o[:, part]) and torch.equal(p1, o1[part]) and torch.equal(T, S[part])
    last = slice(B - 1, B)
    _check_la(o[:, last], None, q[:, last], k[:, last], v[:, last], ld, 0.5, s0[last], None, dtype)


@pytest.fixture()
def wait_limit(fi):  # noqa: F811
    yield fi.set_op_wait_limit
    fi.set_op_wait_limit(-1)


def _gives_up_and_recovers(fi, wait_limit, call, outputs, limits=(0, 1)):  # noqa: F811
    # a wait that gives up ends the call, op_sync says so once, and what comes after is as
    # it was before
    call()
    fi.op_sync()
    want = [t.clone() for t in outputs]
    for limit in limits:
        wait_limit(limit)
        call()
        call()
        wait_limit(-1)
        if limit == 0:
            with pytest.raises(fi.FiError) as e:
                fi.op_sync()
            assert e.value.status == fi.FI_E_TIMEOUT
        else:                                # may have been long enough
            try:
                fi.op_sync()
            except fi.FiError as e:
                assert e.status == fi.FI_E_TIMEOUT
        fi.op_sync()
        for t in outputs:
            t.zero_()
        call()
        fi.op_sync()
        for t, w in zip(outputs, want):
            assert torch.equal(t, w)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,nin,nout", [(20, 512, 300), (40, 2048, 2048), (64, 4096, 1000), (16, 8192, 8192), (100, 2048, 200), (64, 8192, 512)])
def test_waits_that_give_up_linear_few_rows(fi, wait_limit, n, nin, nout, dtype):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(n)
    x, w = _rand(g, n, nin, dtype=DT[dtype]), _rand(g, nout, nin, dtype=DT[dtype], scale=nin ** -0.5)
    if dtype == "f32":
        x = x[:64]                           # more rows run on tiles
    base = torch.full((n * nout + 64,), 7.0, dtype=DT[dtype], device="cuda")
    y = base[:x.shape[0] * nout].view(-1, nout)
    _gives_up_and_recovers(fi, wait_limit, lambda: fi.linear(x, w, y, act="gelu"), [y])
    assert (base[y.numel():] == 7.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,B,H,d,ragged", [(100, 1, 2, 64, False), (2065, 1, 2, 64, False), (2065, 2, 1, 128, True),
                                            (260, 160, 1, 40, False), (1000, 2, 3, 100, True)])
def test_waits_that_give_up_prefill(fi, wait_limit, n, B, H, d, ragged, dtype):  # noqa: F811
    q, k, v, ld, s0 = _la_inputs(n, B, H, d, d, dtype, n)
    lengths = torch.tensor([n - 37 * b for b in range(B)], dtype=torch.int32, device="cuda") if ragged else None
    base = torch.full((n * B * H * d + 64,), 7.0, dtype=DT[dtype], device="cuda")
    o, S = base[:v.numel()].view_as(v), torch.empty_like(s0)
    o.zero_()
    _gives_up_and_recovers(fi, wait_limit, lambda: fi.linattn_prefill(q, k, v, ld, o, state_in=s0, state_out=S, lengths=lengths,
                                                                      scale=d ** -0.5), [o, S])
    assert (base[v.numel():] == 7.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,nin,nout", [(300, 64, 300), (300, 2048, 2048), (200, 2048, 128), (600, 4096, 256), (4100, 512, 2049)])
def test_waits_that_give_up_linear_tiles(fi, wait_limit, n, nin, nout, dtype):  # noqa: F811
    # one stage of the ring and many, tiles shared by several pairs, several tiles to a pair
    g = torch.Generator(device="cuda").manual_seed(n)
    x, w = _rand(g, n, nin, dtype=DT[dtype]), _rand(g, nout, nin, dtype=DT[dtype], scale=nin ** -0.5)
    r = _rand(g, n, nout, dtype=DT[dtype])
    base = torch.full((n * nout + 64,), 7.0, dtype=DT[dtype], device="cuda")
    y = base[:n * nout].view(n, nout)
    _gives_up_and_recovers(fi, wait_limit, lambda: fi.linear(x, w, y, residual=r, act="silu"), [y])
    assert (base[n * nout:] == 7.0).all()


@pytest.mark.parametrize("n,B,H,dk,dv,fused,carried", [(1, 1, 2, 64, 64, False, True), (130, 1, 2, 128, 128, True, True), (700, 2, 2, 64, 128, False, True),
                                                       (2065, 1, 1, 128, 64, False, True), (900, 2, 3, 96, 40, True, False)])
@pytest.mark.parametrize("cancel", [False, True])
def test_prefill_bf16_results_are_rounded_once(fi, n, B, H, dk, dv, fused, carried, cancel):  # noqa: F811
    # The scores and the state enter their products as two bf16 parts. Each part is off by
    # at most 2^-8 of what it rounds, so two are by 2^-16 of it, and every term of an output
    # has one of the two: 2^-16 of the sum of absolute values besides the rounding of
    # the result, 2^-8 of itself. Over a whole output the roundings are
    # spread evenly: 2^-8 / sqrt 3 of the 2-norm. With `cancel` the state before takes away
    # most of what the first positions give.
    q, k, v, ld, s0 = _la_inputs(n, B, H, dk, dv, "bf16", n + dk, fused)
    if cancel:
        ld = torch.full_like(ld, -1e-4)
        v[1:] *= 0.01                        # the first position's k v^T is most of the state,
        s0 = -k[0].double()[..., :, None] * v[0].double()[..., None, :]
        s0 = s0.float() * math.exp(1e-4)     # taken away by what is carried in
    o, S = torch.empty_like(v), torch.empty_like(s0)
    fi.linattn_prefill(q, k, v, ld, o, state_in=s0 if carried else None, state_out=S, scale=dk ** -0.5)
    fi.op_sync()
    s = _f64(s0) if carried else None
    want, _ = ops.linattn(_f64(q), _f64(k), _f64(v), _f64(ld), dk ** -0.5, s)
    A, _ = ops.linattn(np.abs(_f64(q)), np.abs(_f64(k)), np.abs(_f64(v)), _f64(ld), dk ** -0.5, None if s is None else np.abs(s))
    err = np.abs(_f64(o) - want)
    tol = U16 * np.abs(want) + (2.0 ** -16 + (n + dk + 16) * U32) * A
    assert np.all(err <= tol), (err / tol).max()
    if not cancel and want.size >= 4096:
        assert np.linalg.norm(err) <= U16 / math.sqrt(3.0) * np.linalg.norm(want)


@pytest.mark.parametrize("n,nin,nout", [(10, 512, 300), (16, 16000, 200), (16, 2048, 8192), (30, 8192, 512), (64, 4096, 1000), (64, 4096, 8192),
                                        (64, 8192, 512), (30, 16000, 512), (9, 30000, 130), (100, 2048, 300), (300, 4096, 512), (600, 700, 600)])
def test_linear_fp32_error_does_not_grow_with_the_contraction(fi, n, nin, nout):  # noqa: F811
    # Inside a block of 64 only the products of the first parts, four steps of 16, add to a
    # sum of full size, each off by at most 2^-23 of it and 2^-24 on average (the tensor
    # core cuts off), so a block is off by 4 x 2^-24 of itself at most on average; blocks
    # are added up with rounding, and K / 64 <= 512 roundings of up to 2^-24 of a sum that
    # grows like a walk are sqrt(512 / 2) x 2^-24 / sqrt 3 on average. The blocks'
    # errors do not go one way, since blocks have either sign: over sqrt(K / 64) of them
    # the 2-norm stays at 4 x 2^-24, together with the roundings of the sums below
    # 4 x 2^-24 + sqrt(K / 128 / 3) 2^-24 and one for the result.
    g = torch.Generator(device="cuda").manual_seed(nin)
    x, w = _rand(g, n, nin), _rand(g, nout, nin, scale=nin ** -0.5)
    y = torch.empty(n, nout, device="cuda")
    fi.linear(x, w, y)
    fi.op_sync()
    want = x.double() @ w.double().T
    rel = float((y.double() - want).norm() / want.norm())
    assert rel <= (5 + math.sqrt(nin / 128 / 3)) * U32, rel


def _recurrence64(q, k, v, ld, scale, s0):
    """The recurrence position by position in float64, on the GPU: o [n][B][H][dv], S."""
    S = torch.zeros(*q.shape[1:], v.shape[-1], dtype=torch.float64, device="cuda") if s0 is None else s0.double()
    g = ld.double().clamp(max=0).exp()[:, None, None]
    o = torch.empty(v.shape, dtype=torch.float64, device="cuda")
    for t in range(q.shape[0]):
        S = g * S + k[t].double()[..., :, None] * v[t].double()[..., None, :]
        o[t] = scale * (q[t].double()[..., None, :] @ S)[..., 0, :]
    return o, S


def _off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,B,H,dk,dv", [(300, 2, 2, 64, 64), (2500, 2, 2, 64, 64), (2065, 1, 3, 100, 128), (700, 3, 2, 33, 47), (8200, 1, 2, 64, 64)])
def test_prefill_errors_in_the_2_norm(fi, n, B, H, dk, dv, dtype):  # noqa: F811
    # Of the products of a block of 64 only those of the first parts, four steps of 16,
    # add to a sum of full size. The tensor core cuts sums off: 2^-24 of them on average, of
    # sums that grow like a walk, (1 + sqrt 2 + sqrt 3 + 2) / 8 = 0.77 of the last one,
    # 3.1 x 2^-24 a product, always towards zero. An fp32 output goes through two products, Q K^T
    # and P V or K^T (w V) and Q S: 6.2; the powers of the decay, exponents of up to a few units
    # rounded to 2^-24 of themselves, 2; fp32 roundings of P, S and their factors 1.5: together
    # 9.7 x 2^-24 of its 2-norm. States go through one product: 6.6; bf16 inputs' have
    # one accumulator for a chunk, 4 steps and 12 at full size, 8 x 2^-24 more.
    # Losing a third part of an operand would add 1.8e-6 = 30 x 2^-24.
    q, k, v, ld, s0 = _la_inputs(n, B, H, dk, dv, dtype, 3 * n + dk)
    o, S = torch.empty_like(v), torch.empty_like(s0)
    fi.linattn_prefill(q, k, v, ld, o, state_in=s0, state_out=S, scale=dk ** -0.5)
    fi.op_sync()
    want_o, want_S = _recurrence64(q, k, v, ld, dk ** -0.5, s0)
    if dtype == "f32":
        assert _off(o, want_o) <= 9.7 * U32
        assert _off(S, want_S) <= 6.6 * U32
    else:
        assert _off(o, want_o) <= U16 / math.sqrt(3.0) + 2.0 ** -16
        assert _off(S, want_S) <= 14.6 * U32


def test_calls_from_several_threads(fi):  # noqa: F811
    # four threads, a stream and tensors each, call every operator at once, sizes that no call
    # has had before among them; the results are those of one thread
    import threading

    def work(i, stream):
        n = 130 + 64 * i
        with torch.cuda.stream(stream):
            q, k, v, ld, s0 = _la_inputs(n, 2, 2, 64, 64, "bf16" if i % 2 else "f32", i)
            g = torch.Generator(device="cuda").manual_seed(i)
            w, x = _rand(g, 96 + i, 128, dtype=v.dtype), _rand(g, 20 + i, 128, dtype=v.dtype)
            outs = []
            for _ in range(8):
                o, S = torch.empty_like(v), s0.clone()
                fi.linattn_prefill(q, k, v, ld, o, state_in=S, state_out=S)
                o1 = torch.empty_like(o[0])
                fi.linattn_step(q[0], k[0], v[0], ld, S, o1)
                y = torch.empty(n * 2, 96 + i, dtype=v.dtype, device="cuda")
                fi.linear(o.view(n * 2, 128), w, y, act="gelu")
                y1 = torch.empty(20 + i, 96 + i, dtype=v.dtype, device="cuda")
                fi.linear(x, w, y1)
                outs.append((o, S, o1, y, y1))
            stream.synchronize()
        return outs

    got, errors = [None] * 4, []
    gate = threading.Barrier(4)

    def body(i):
        try:
            stream = torch.cuda.Stream()
            gate.wait(60)
            got[i] = work(i, stream)
        except Exception as e:     # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=body, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not errors, errors
    torch.cuda.synchronize()
    fi.op_sync()
    for i in range(4):
        want = work(i, torch.cuda.Stream())[0]
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("n,nin,nout,positive", [(300, 16384, 300, False), (40, 65536, 130, False), (520, 65536, 256, False), (300, 1 << 20, 64, False),
                                                 (300, 1 << 18, 64, True), (16, 1 << 18, 64, True)])
def test_linear_bf16_long_contractions(fi, n, nin, nout, positive):  # noqa: F811
    # Products of 16 add to one accumulator (to 2 to 8, where CTAs share the contraction), each
    # sum cut off by 2^-24 of itself on average, always towards zero: over K / 16 of
    # them, of sums that grow like a walk, at most K / 16 x 2/3 x 2^-24 of the result; of
    # sums that grow evenly (positive values), K / 16 / 2 x 2^-24. That and the rounding of
    # the result, 2^-8 / sqrt 3 over a whole output.
    g = torch.Generator(device="cuda").manual_seed(nin)
    x, w = _rand(g, n, nin, dtype=torch.bfloat16), _rand(g, nout, nin, dtype=torch.bfloat16, scale=nin ** -0.5)
    if positive:
        x, w = x.abs(), w.abs()
    y = torch.empty(n, nout, dtype=torch.bfloat16, device="cuda")
    fi.linear(x, w, y)
    fi.op_sync()
    want = torch.zeros(n, nout, dtype=torch.float64, device="cuda")
    for c in range(0, nin, 1 << 16):
        want += x[:, c:c + (1 << 16)].double() @ w[:, c:c + (1 << 16)].double().T
    cut = nin / 16 * (0.5 if positive else 2 / 3) * U32
    assert _off(y, want) <= math.hypot(U16 / math.sqrt(3.0), cut)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,d", [(100, 64), (2065, 64), (2065, 128), (300, 200)])
def test_prefill_that_starts_from_a_state_and_keeps_none(fi, n, d, dtype):  # noqa: F811
    q, k, v, ld, s0 = _la_inputs(n, 1, 2, d, d, dtype, n)
    o, before = torch.empty_like(v), s0.clone()
    fi.linattn_prefill(q, k, v, ld, o, state_in=s0, scale=d ** -0.5)
    fi.op_sync()
    assert torch.equal(s0, before)
    _check_la(o, None, q, k, v, ld, d ** -0.5, s0, None, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prefill_of_300001_positions(fi, dtype):  # noqa: F811
    # without decay, outputs are products with running sums. Besides what a shorter prompt has
    # (9.7 x 2^-24), 37 chunks of a segment and 64 segments are added up with rounding, of sums
    # that grow like a walk: sqrt(37 / 6) + sqrt(64 / 6).
    n, H, d = 300001, 2, 8
    q, k, v, _, _ = _la_inputs(n, 1, H, d, d, dtype, 1)
    ld = torch.zeros(H, device="cuda")
    o, S = torch.empty_like(v), torch.empty(1, H, d, d, device="cuda")
    fi.linattn_prefill(q, k, v, ld, o, state_out=S)
    fi.op_sync()
    sums = torch.cumsum(k.double()[..., :, None] * v.double()[..., None, :], dim=0)
    want = (q.double()[..., None, :] @ sums)[..., 0, :]
    extra = (math.sqrt(37 / 6) + math.sqrt(64 / 6)) * U32
    assert _off(o, want) <= (9.7 * U32 + extra if dtype == "f32" else U16 / math.sqrt(3.0) + 2.0 ** -16)
    assert _off(S, sums[-1]) <= (6.6 if dtype == "f32" else 14.6) * U32 + extra


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,nin,nout", [((1 << 21) + 3, 16, 9), (1, 16, 1 << 20), (3, 8, (1 << 20) - 1), (20, 16, 1 << 20), (200, 8, (1 << 20) - 3)])
def test_linear_of_very_many_rows_or_columns(fi, n, nin, nout, dtype):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(nin)
    x, w, b = (_rand(g, *s, dtype=DT[dtype]) for s in ((n, nin), (nout, nin), (nout,)))
    y = torch.empty(n, nout, dtype=DT[dtype], device="cuda")
    fi.linear(x, w, y, bias=b, act="relu")
    fi.op_sync()
    for r in range(0, n, 1 << 20):
        part = slice(r, min(r + (1 << 20), n))
        want = (x[part].double() @ w.double().T + b.double()).clamp(min=0)
        A = x[part].double().abs() @ w.double().abs().T + b.double().abs()
        tol = (nin + 16) * U32 * A + (U16 if dtype == "bf16" else U32) * want
        assert ((y[part].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("n", [1, 40, 300])
def test_gelu_fp32_is_accurate_everywhere(fi, n):  # noqa: F811
    # relative to the result: the fit 1.9e-8, its 9 steps and the reciprocal (times 3.8 at
    # most, the fit's slope) 8 roundings, the exponential 3, products and the difference 4, and
    # 1.25 u^2 of them for the exponent: (16 + 1.5 u^2) 2^-24, one more for x w
    u = torch.cat([torch.linspace(-9, 9, 4001), torch.logspace(-30, 0, 301), -torch.logspace(-30, 0, 301), torch.tensor([0.0, -0.0, 20.0, 3e38])]).cuda()
    w = torch.zeros(u.numel(), 16, device="cuda")
    w[:, 2] = u
    x = torch.zeros(n, 16, device="cuda")
    x[:, 2] = 1.0
    y = torch.empty(n, u.numel(), device="cuda")
    fi.linear(x, w, y, act="gelu")
    fi.op_sync()
    u64 = _f64(u)
    want = u64 * np.array([0.5 * math.erfc(-t / math.sqrt(2.0)) for t in u64])
    err = np.abs(_f64(y) - want)
    assert np.all(err <= (17 + 1.5 * np.minimum(u64 * u64, 81)) * U32 * np.abs(want))
