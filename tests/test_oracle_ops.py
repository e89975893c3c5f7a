"""Pins of the operators' oracle, and the operators' refusals (no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest

from oracle import ops


def test_linattn_equals_the_quadratic_form():
    r = np.random.default_rng(1)
    n, B, H, dk, dv = 13, 2, 3, 4, 5
    q, k, v = r.standard_normal((n, B, H, dk)), r.standard_normal((n, B, H, dk)), r.standard_normal((n, B, H, dv))
    ld = np.log([0.5, 0.9, 1.0])
    o, S = ops.linattn(q, k, v, ld, 0.7)
    for h in range(H):
        lag = np.arange(n)[:, None] - np.arange(n)[None, :]
        D = np.where(lag >= 0, np.exp(np.maximum(lag, 0) * ld[h]), 0.0)
        for b in range(B):
            want = 0.7 * ((q[:, b, h] @ k[:, b, h].T) * D) @ v[:, b, h]
            assert np.allclose(o[:, b, h], want, rtol=1e-12, atol=1e-12)
            wt = np.exp((n - 1 - np.arange(n)) * ld[h])
            assert np.allclose(S[b, h], (k[:, b, h] * wt[:, None]).T @ v[:, b, h], rtol=1e-12, atol=1e-12)


def test_linattn_limits():
    r = np.random.default_rng(2)
    n = 6
    q, k, v = (r.standard_normal((n, 1, 2, 3)) for _ in range(3))
    # no decay with one-hot keys and queries: prefix sums; a decay of 0: the position alone
    q[:] = k[:] = np.array([1.0, 0, 0])
    o, _ = ops.linattn(q, k, v, np.array([0.0, -np.inf]))
    assert np.allclose(o[:, 0, 0], np.cumsum(v[:, 0, 0], axis=0))
    assert np.allclose(o[:, 0, 1], v[:, 0, 1])
    # two prompts in a row are one prompt
    q, k, v = (r.standard_normal((n, 2, 2, 3)) for _ in range(3))
    ld = np.array([-0.1, -0.5])
    whole, S = ops.linattn(q, k, v, ld)
    o1, S1 = ops.linattn(q[:4], k[:4], v[:4], ld)
    o2, S2 = ops.linattn(q[4:], k[4:], v[4:], ld, state=S1)
    assert np.allclose(np.concatenate([o1, o2]), whole) and np.allclose(S2, S)
    # lengths: the state stops there
    _, S3 = ops.linattn(q, k, v, ld, lengths=[4, 0])
    assert np.allclose(S3[0], S1[0]) and np.all(S3[1] == 0)


def test_linear_pins():
    torch = pytest.importorskip("torch")
    r = np.random.default_rng(3)
    x, w, b, res = r.standard_normal((4, 5)), r.standard_normal((3, 5)), r.standard_normal(3), r.standard_normal((4, 3))
    fn = {"none": lambda t: t, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu,
          "relu": torch.relu, "tanh": torch.tanh}
    for act, f in fn.items():
        want = f(torch.from_numpy(x) @ torch.from_numpy(w).T + torch.from_numpy(b)) + torch.from_numpy(res)
        assert np.allclose(ops.linear(x, w, b, res, act), want.numpy(), rtol=1e-12, atol=1e-12)


# ------------------------------------------------------------------ refusals, before the device is touched

P = ctypes.c_void_p(4096)      # an address that is never read


def _fi():
    from long_convolution_sequence_online_b200 import fi
    return fi


def _la(fi, **kw):
    f = dict(heads=2, key_dim=8, value_dim=16, batch=3, dtype=fi.FI_F32, scale=1.0)
    strides = dict(q_stride=(48, 16, 8), k_stride=(48, 16, 8), v_stride=(96, 32, 16), o_stride=(96, 32, 16))
    reserved = kw.pop("reserved", 0)
    for n in strides:
        strides[n] = kw.pop(n, strides[n])
    f.update(kw)
    c = fi.LinattnConfig(**f)
    for n, s in strides.items():
        getattr(c, n)[:] = s
    c.reserved[3] = reserved
    return c


LA_BAD = [
    (dict(heads=0), "heads"), (dict(batch=0), "batch"), (dict(key_dim=0), "key_dim"), (dict(key_dim=257), "key_dim"),
    (dict(value_dim=0), "value_dim"), (dict(value_dim=257), "value_dim"), (dict(heads=1 << 12, batch=1 << 12), "batch x heads"),
    (dict(dtype=2), "dtype"), (dict(scale=math.inf), "scale"), (dict(scale=math.nan), "scale"), (dict(reserved=1), "reserved"),
    (dict(q_stride=(-1, 16, 8)), "strides"), (dict(v_stride=(1 << 41, 32, 16)), "strides"),
    (dict(o_stride=(96, 32, 8)), "overlap"), (dict(o_stride=(96, 32, 0)), "overlap"), (dict(o_stride=(95, 32, 16)), "overlap"),
]


@pytest.mark.parametrize("kw,why", LA_BAD)
def test_linattn_refuses_bad_configurations(kw, why):
    fi = _fi()
    cfg = _la(fi, **kw)
    need = ctypes.c_uint64(7)
    calls = [lambda: fi.lib.fi_linattn_workspace(ctypes.addressof(cfg), 5, P, P, P, ctypes.byref(need)),
             lambda: fi.lib.fi_linattn_prefill(ctypes.addressof(cfg), 5, P, P, P, P, None, None, None, P, None, 0, None)]
    if kw.get("o_stride", (0,))[0] != 95:      # a step has no position dimension
        calls.append(lambda: fi.lib.fi_linattn_step(ctypes.addressof(cfg), P, P, P, P, P, P, None))
    for call in calls:
        assert call() == fi.FI_E_INVALID
        assert why in fi.lib.fi_last_error().decode()


def test_linattn_refuses_nulls_and_alignment():
    fi = _fi()
    cfg = _la(fi)
    at = ctypes.addressof(cfg)
    L = fi.lib
    assert L.fi_linattn_prefill(None, 5, P, P, P, P, None, None, None, P, None, 0, None) == fi.FI_E_INVALID
    assert L.fi_linattn_prefill(at, -1, P, P, P, P, None, None, None, P, None, 0, None) == fi.FI_E_INVALID
    assert L.fi_linattn_prefill(at, (1 << 30) + 1, P, P, P, P, None, None, None, P, None, 0, None) == fi.FI_E_INVALID
    assert L.fi_linattn_workspace(at, 5, P, P, P, None) == fi.FI_E_INVALID
    for miss in range(5):
        a = [P] * 5
        a[miss] = None
        assert L.fi_linattn_prefill(at, 5, a[0], a[1], a[2], a[3], None, None, None, a[4], None, 0, None) == fi.FI_E_INVALID
    for miss in range(6):
        a = [P] * 6
        a[miss] = None
        assert L.fi_linattn_step(at, *a, None) == fi.FI_E_INVALID
        a[miss] = ctypes.c_void_p(4098)
        assert L.fi_linattn_step(at, *a, None) == fi.FI_E_INVALID
        assert "aligned" in L.fi_last_error().decode()
    odd = ctypes.c_void_p(4098)
    for miss in range(8):
        a = [P] * 8
        a[miss] = odd
        assert L.fi_linattn_prefill(at, 5, a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], None, 0, None) == fi.FI_E_INVALID
        assert "aligned" in L.fi_last_error().decode()


LIN_BAD = [
    (dict(in_features=0), "in_features"), (dict(out_features=0), "out_features"), (dict(in_features=(1 << 20) + 1, ldx=1 << 21, ldw=1 << 21), "in_features"),
    (dict(dtype=9), "dtype"), (dict(act=5), "act"), (dict(act=-1), "act"), (dict(ldx=7), "ldx"), (dict(ldw=0), "ldw"),
    (dict(ldy=15), "ldy"), (dict(ldr=15), "ldr"), (dict(ldw=(1 << 40) + 1), "leading"), (dict(reserved=1), "reserved"),
]


def _lin(fi, **kw):
    f = dict(in_features=8, out_features=16, dtype=fi.FI_F32, act=0, ldx=8, ldw=8, ldr=16, ldy=16)
    reserved = kw.pop("reserved", 0)
    f.update(kw)
    c = fi.LinearConfig(**f)
    c.reserved[0] = reserved
    return c


@pytest.mark.parametrize("kw,why", LIN_BAD)
def test_linear_refuses_bad_configurations(kw, why):
    fi = _fi()
    cfg = _lin(fi, **kw)
    far = [ctypes.c_void_p(4096 * i) for i in range(1, 6)]
    assert fi.lib.fi_linear(ctypes.addressof(cfg), 4, *far, None, 0, None) == fi.FI_E_INVALID
    assert why in fi.lib.fi_last_error().decode()


def test_linear_refuses_nulls_alignment_and_aliases():
    fi = _fi()
    L = fi.lib
    cfg = _lin(fi)
    at = ctypes.addressof(cfg)
    x, w, b, r, y = (ctypes.c_void_p(1 << (12 + i)) for i in range(5))
    assert L.fi_linear(None, 4, x, w, b, r, y, None, 0, None) == fi.FI_E_INVALID
    assert L.fi_linear(at, -1, x, w, b, r, y, None, 0, None) == fi.FI_E_INVALID
    assert L.fi_linear(at, 4, None, w, b, r, y, None, 0, None) == fi.FI_E_INVALID
    assert L.fi_linear(at, 4, x, None, b, r, y, None, 0, None) == fi.FI_E_INVALID
    assert L.fi_linear(at, 4, x, w, b, r, None, None, 0, None) == fi.FI_E_INVALID
    odd = ctypes.c_void_p(4098)
    for i in range(5):
        a = [x, w, b, r, y]
        a[i] = odd
        assert L.fi_linear(at, 4, *a, None, 0, None) == fi.FI_E_INVALID
        assert "aligned" in L.fi_last_error().decode()
    assert L.fi_linear(at, 4, y, w, b, r, y, None, 0, None) == fi.FI_E_INVALID
    assert L.fi_linear(at, 4, x, y, b, r, y, None, 0, None) == fi.FI_E_INVALID
    bad = _lin(fi, ldr=24)
    assert L.fi_linear(ctypes.addressof(bad), 4, x, w, b, y, y, None, 0, None) == fi.FI_E_INVALID
    assert L.fi_linear(at, 0, x, w, b, r, y, None, 0, None) == fi.FI_OK      # no rows: nothing to do


def test_linear_scratch_is_known_without_a_device():
    fi = _fi()
    need = ctypes.c_uint64(7)
    at = ctypes.c_void_p
    aligned, odd = at(4096), at(4098)
    bf = _lin(fi, in_features=64, ldx=64, ldw=64, dtype=fi.FI_BF16)
    ask = lambda cfg, n, x, w: (fi.lib.fi_linear_workspace(ctypes.addressof(cfg), n, x, w, ctypes.byref(need)), need.value)   # noqa: E731
    assert ask(bf, 300, aligned, aligned) == (fi.FI_OK, 0)
    assert ask(bf, 300, odd, aligned) == (fi.FI_OK, 300 * 64 * 2)           # x alone
    assert ask(bf, 300, aligned, odd) == (fi.FI_OK, 16 * 64 * 2)            # w alone
    assert ask(bf, 1, odd, odd) == (fi.FI_OK, 0)                            # one row reads them as they stand
    f32 = _lin(fi, in_features=60, ldx=60, ldw=60)
    assert ask(f32, 300, aligned, aligned) == (fi.FI_OK, -(-3 * 300 * 64 * 2 // 256) * 256 + 3 * 16 * 64 * 2)
    assert ask(f32, 0, aligned, aligned) == (fi.FI_OK, 0)
    assert fi.lib.fi_linear_workspace(ctypes.addressof(f32), 300, aligned, aligned, None) == fi.FI_E_INVALID
    assert fi.lib.fi_linear(ctypes.addressof(f32), 300, at(1 << 20), at(1 << 21), None, None, at(1 << 22), None, 0, None) == fi.FI_E_INVALID
    assert "workspace" in fi.lib.fi_last_error().decode()


def test_linattn_refuses_outputs_among_inputs():
    fi = _fi()
    cfg = _la(fi)
    at = ctypes.addressof(cfg)
    p = [ctypes.c_void_p(1 << (12 + i)) for i in range(5)]
    for i in range(3):
        assert fi.lib.fi_linattn_prefill(at, 5, p[0], p[1], p[2], p[3], None, None, None, p[i], None, 0, None) == fi.FI_E_INVALID
        assert "o must not" in fi.lib.fi_last_error().decode()
        assert fi.lib.fi_linattn_step(at, p[0], p[1], p[2], p[3], p[4], p[i], None) == fi.FI_E_INVALID
        assert "o must not" in fi.lib.fi_last_error().decode()


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    fi = _fi()
    t = torch.zeros(4, 4)
    with pytest.raises(ValueError):
        fi.linear(t, t, t.clone())
    q = torch.zeros(2, 1, 1, 4)
    with pytest.raises(ValueError):
        fi.linattn_prefill(q, q, q, torch.zeros(1), q.clone())
    with pytest.raises(ValueError):
        fi.linattn_step(q[0], q[0], q[0], torch.zeros(1), torch.zeros(1, 1, 4, 4), q[0].clone())
