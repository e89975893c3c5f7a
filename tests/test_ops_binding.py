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
