"""The operators' Python calls and C checks without a GPU: stand-ins for the tensors and
the library record what a call would do."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture()
def fi():
    from long_convolution_sequence_online_b200 import fi as _fi
    return _fi


class Stub:
    """What a call asks of a tensor, on CUDA device `dev`."""

    def __init__(self, *shape, dtype=torch.float32, dev=0, at=4096):
        self._t = torch.empty(shape, dtype=dtype, device="meta")
        self.shape, self.dtype, self._dev, self._at, self.device = self._t.shape, dtype, dev, at, f"cuda:{dev}"

    def stride(self, d=None):
        return self._t.stride() if d is None else self._t.stride(d)

    def dim(self):
        return self._t.dim()

    def is_contiguous(self):
        return True

    def get_device(self):
        return self._dev

    def data_ptr(self):
        return self._at


class Lib:
    """Stands in for the library: keeps each call's name and the configuration it was given."""

    def __init__(self, fi):
        self.calls, self.fi = [], fi

    def __getattr__(self, name):
        if not name.startswith("fi_"):
            raise AttributeError(name)

        def call(at, *args):
            kind = self.fi.LinearConfig if name.startswith("fi_linear") else self.fi.LinattnConfig
            self.calls.append((name, kind.from_buffer_copy(ctypes.string_at(at, ctypes.sizeof(kind)))))
            return 0
        return call


@pytest.fixture()
def stand_in(fi, monkeypatch):
    lib = Lib(fi)
    monkeypatch.setattr(fi, "lib", lib)
    monkeypatch.setattr(fi, "_configs", {})
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    return lib


def _prompt(fi, dev, **kw):
    t = lambda *s: Stub(*s, dev=dev)   # noqa: E731
    fi.linattn_prefill(t(5, 2, 3, 8), t(5, 2, 3, 8), t(5, 2, 3, 16), t(3), t(5, 2, 3, 16), **kw)


def _step(fi, dev, **kw):
    t = lambda *s: Stub(*s, dev=dev)   # noqa: E731
    fi.linattn_step(t(2, 3, 8), t(2, 3, 8), t(2, 3, 16), t(3), t(2, 3, 8, 16), t(2, 3, 16), **kw)


def _linear(fi, dev, **kw):
    t = lambda *s: Stub(*s, dev=dev)   # noqa: E731
    fi.linear(t(4, 8), t(6, 8), t(4, 6), **kw)


@pytest.mark.parametrize("call", [_prompt, _step, _linear])
def test_another_device_than_the_current_one_leaves_nothing_behind(fi, stand_in, call):
    # the scratch of a call depends on the current device: a refused call must not keep a
    # size that belongs to another one
    with pytest.raises(ValueError, match="not the current device"):
        call(fi, 1)
    assert not stand_in.calls and not fi._configs
    call(fi, 0)
    assert stand_in.calls and fi._configs
    with pytest.raises(ValueError, match="not the current device"):
        call(fi, 1)


@pytest.mark.parametrize("call", [_prompt, _step])
def test_a_scale_that_changes_in_place_is_read_anew(fi, stand_in, call):
    scale = torch.tensor(0.5)
    call(fi, 0, scale=scale)
    scale.fill_(2.0)
    call(fi, 0, scale=scale)
    assert stand_in.calls[0][1].scale == 0.5 and stand_in.calls[-1][1].scale == 2.0


def test_more_than_2_to_the_29_rows_or_positions_are_refused(fi):
    # three parts of as many rows are indexed below 2^31
    P, need = ctypes.c_void_p(4096), ctypes.c_uint64()
    la = fi.LinattnConfig(1, 8, 8, 1, fi.FI_F32, 1.0)
    for name in ("q_stride", "k_stride", "v_stride", "o_stride"):
        getattr(la, name)[:] = (8, 8, 8)
    lin = fi.LinearConfig(8, 8, fi.FI_F32, 0, 8, 8, 8, 8)
    at, al, most = ctypes.addressof(la), ctypes.addressof(lin), 1 << 29
    assert fi.lib.fi_linattn_prefill(at, most + 1, P, P, P, P, None, None, None, P, None, 0, None) == fi.FI_E_INVALID
    assert "2^29" in fi.lib.fi_last_error().decode()
    assert fi.lib.fi_linattn_workspace(at, most + 1, P, P, P, ctypes.byref(need)) == fi.FI_E_INVALID
    assert "2^29" in fi.lib.fi_last_error().decode()
    assert fi.lib.fi_linear(al, most + 1, P, P, None, None, P, None, 0, None) == fi.FI_E_INVALID
    assert "2^29" in fi.lib.fi_last_error().decode()
    assert fi.lib.fi_linear_workspace(al, most + 1, P, P, ctypes.byref(need)) == fi.FI_E_INVALID
    assert "2^29" in fi.lib.fi_last_error().decode()
    assert fi.lib.fi_linear_workspace(al, most, P, P, ctypes.byref(need)) == fi.FI_OK
    assert need.value == 3 * 8 * 2 * most + 512        # x's parts, and w's in units of 256


def test_states_that_overlap_in_part_are_refused(fi):
    la = fi.LinattnConfig(2, 8, 4, 3, fi.FI_F32, 1.0)
    for name, d in (("q_stride", 8), ("k_stride", 8), ("v_stride", 4), ("o_stride", 4)):
        getattr(la, name)[:] = (6 * d, 2 * d, d)
    p = [ctypes.c_void_p(1 << (12 + i)) for i in range(5)]
    at, bytes_ = ctypes.addressof(la), 2 * 3 * 8 * 4 * 4
    for shift in (4, 128, bytes_ - 4, -4, 4 - bytes_):
        s_in, s_out = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + shift)
        assert fi.lib.fi_linattn_prefill(at, 5, p[0], p[1], p[2], p[3], None, s_in, s_out, p[4], None, 0, None) == fi.FI_E_INVALID
        assert "overlap" in fi.lib.fi_last_error().decode()
