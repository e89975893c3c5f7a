"""Thin ctypes binding of libfi.so (include/fi.h): argument marshalling only.

Every computation runs in the library's CUDA kernels. PyTorch supplies device
memory (tensors' data pointers) and the current CUDA stream. If libfi.so is
missing or fails to load, importing this module raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfi.so")

FI_OK, FI_E_INVALID, FI_E_OOM, FI_E_CUDA, FI_E_STATE, FI_E_TIMEOUT, FI_E_UNSUPPORTED = range(7)
FI_F32, FI_BF16 = 0, 1
NUM_KERNEL_CLASSES = 6
KERNEL_CLASSES = ("chunk", "direct", "fft", "token", "lazy", "tc")

EXPORTED = ("fi_init", "fi_step", "fi_generate", "fi_generate_host", "fi_generate_lazy", "fi_sync", "fi_reset",
            "fi_position", "fi_read_activations", "fi_set_stream", "fi_get_plan", "fi_profile",
            "fi_profile_read", "fi_destroy", "fi_status_str", "fi_last_error", "fi_debug_fft",
            "fi_generate_noalloc", "fi_debug_set_wait_limit", "fi_debug_chunk_schedule", "fi_prefill", "fi_profile_read_sides",
            "fi_set_mlp_block", "fi_linattn_workspace", "fi_linattn_prefill", "fi_linattn_step", "fi_linear", "fi_linear_workspace",
            "fi_op_sync", "fi_debug_set_op_wait_limit")


class FiError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: status {status}: {message}")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [("layers", ctypes.c_int32), ("channels", ctypes.c_int32), ("max_len", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("dtype", ctypes.c_int32), ("chunk", ctypes.c_int32),
                ("fft_from", ctypes.c_int32), ("tc_max", ctypes.c_int32), ("reserved", ctypes.c_int32 * 4)]


class LinattnConfig(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int32), ("key_dim", ctypes.c_int32), ("value_dim", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("q_stride", ctypes.c_int64 * 3), ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3),
                ("o_stride", ctypes.c_int64 * 3), ("reserved", ctypes.c_int32 * 4)]


class LinearConfig(ctypes.Structure):
    _fields_ = [("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("act", ctypes.c_int32), ("ldx", ctypes.c_int64), ("ldw", ctypes.c_int64), ("ldr", ctypes.c_int64),
                ("ldy", ctypes.c_int64), ("reserved", ctypes.c_int32 * 4)]


ACTIVATIONS = {"none": 0, "gelu": 1, "silu": 2, "relu": 3, "tanh": 4}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m long_convolution_sequence_online_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float
    sig = {
        "fi_init": [ctypes.POINTER(vp), ctypes.POINTER(Config), vp, vp],
        "fi_step": [vp, vp, vp],
        "fi_generate": [vp, i32, vp, vp, f32, vp, vp],
        "fi_generate_host": [vp, i32, vp, vp, f32, vp],
        "fi_generate_lazy": [vp, i32, vp, vp, f32, vp],
        "fi_reset": [vp],
        "fi_sync": [vp],
        "fi_position": [vp, ctypes.POINTER(i32)],
        "fi_read_activations": [vp, i32, vp],
        "fi_set_stream": [vp, vp],
        "fi_get_plan": [vp, ctypes.POINTER(i32), ctypes.POINTER(i32), ctypes.POINTER(i32)],
        "fi_profile": [vp, i32],
        "fi_profile_read": [vp, ctypes.POINTER(i32), ctypes.POINTER(ctypes.c_double)],
        "fi_destroy": [vp],
        "fi_debug_fft": [i32, i32, vp, vp, i32, vp],
        "fi_generate_noalloc": [ctypes.POINTER(Config), vp, i32, vp, vp, f32, vp, vp],
        "fi_debug_set_wait_limit": [vp, i32],
        "fi_debug_chunk_schedule": [i32, i32, vp, i32, ctypes.POINTER(i32), ctypes.POINTER(i32)],
        "fi_prefill": [vp, i32, vp, vp, vp],
        "fi_set_mlp_block": [vp, i32, vp, vp, vp, vp],
        "fi_profile_read_sides": [vp, ctypes.POINTER(i32), ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i32),
                                  ctypes.POINTER(ctypes.c_double)],
        "fi_linattn_workspace": [vp, i32, vp, vp, vp, ctypes.POINTER(ctypes.c_uint64)],
        "fi_linattn_prefill": [vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_uint64, vp],
        "fi_linattn_step": [vp, vp, vp, vp, vp, vp, vp, vp],
        "fi_op_sync": [vp],
        "fi_debug_set_op_wait_limit": [i32],
        "fi_linear_workspace": [vp, i32, vp, vp, ctypes.POINTER(ctypes.c_uint64)],
        "fi_linear": [vp, i32, vp, vp, vp, vp, vp, vp, ctypes.c_uint64, vp],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.fi_status_str.argtypes = [ctypes.c_int]
    lib.fi_status_str.restype = ctypes.c_char_p
    lib.fi_last_error.argtypes = []
    lib.fi_last_error.restype = ctypes.c_char_p
    return lib


lib = _load()


def _check(status: int, where: str):
    if status != FI_OK:
        raise FiError(status, where, (lib.fi_last_error() or b"").decode())


def _ptr(t) -> int | None:
    """Device address of a contiguous CUDA tensor (None passes through as NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return int(stream) if not hasattr(stream, "cuda_stream") else stream.cuda_stream


class Context:
    """One fi_ctx: filters, spectra and state of an M-layer online mixer stack."""

    def __init__(self, h, batch: int, dtype: str = "f32", chunk: int = 0, fft_from: int = 0, stream=None,
                 tc_max: int = 0):
        import torch
        if h.dim() != 3:
            raise ValueError("h must be [M][D][L]")
        want = torch.bfloat16 if dtype == "bf16" else torch.float32
        if h.dtype != want:
            raise ValueError(f"h must be {want} for dtype {dtype}")
        M, D, L = h.shape
        self.M, self.D, self.L, self.B = int(M), int(D), int(L), int(batch)
        self.dtype = dtype
        self.torch_dtype = want
        cfg = Config(self.M, self.D, self.L, self.B, FI_BF16 if dtype == "bf16" else FI_F32, chunk, fft_from, tc_max)
        self._cfg = cfg
        self._h = ctypes.c_void_p()
        _check(lib.fi_init(ctypes.byref(self._h), ctypes.byref(cfg), _ptr(h), _stream(stream)), "fi_init")

    # -- lifetime
    def close(self):
        if self._h:
            _check(lib.fi_destroy(self._h), "fi_destroy")
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    # -- calls
    def set_stream(self, stream):
        _check(lib.fi_set_stream(self._h, _stream(stream)), "fi_set_stream")

    def step(self, x_t, y_t):
        _check(lib.fi_step(self._h, _ptr(x_t), _ptr(y_t)), "fi_step")

    def step_ptr(self, x_ptr: int, y_ptr: int):
        """fi_step on raw device addresses (a loop over positions without tensor views)."""
        _check(lib.fi_step(self._h, x_ptr, y_ptr), "fi_step")

    def generate(self, n: int, x0, eps, y_out, eps_scale: float = 0.1, rec=None):
        _check(lib.fi_generate(self._h, n, _ptr(x0), _ptr(eps), eps_scale, _ptr(y_out), _ptr(rec)), "fi_generate")

    def prefill(self, p: int, x, y_out=None, rec=None):
        _check(lib.fi_prefill(self._h, p, _ptr(x), _ptr(y_out), _ptr(rec)), "fi_prefill")

    def set_mlp_block(self, w1=None, b1=None, w2=None, b2=None):
        """Channel-mixing block W2 GELU(W1 y + b1) + b2 after every layer (fp32 CUDA
        tensors w1 [M][Dh][D], b1 [M][Dh], w2 [M][D][Dh], b2 [M][D]); no arguments
        return to the elementwise tanh block."""
        hidden = 0 if w1 is None else int(w1.shape[1])
        _check(lib.fi_set_mlp_block(self._h, hidden, _ptr(w1), _ptr(b1), _ptr(w2), _ptr(b2)), "fi_set_mlp_block")

    def generate_host(self, n: int, x0: np.ndarray, eps: np.ndarray, y_out: np.ndarray, eps_scale: float = 0.1):
        for a in (x0, eps, y_out):
            if not a.flags["C_CONTIGUOUS"]:
                raise ValueError("host arrays must be C-contiguous")
        _check(lib.fi_generate_host(self._h, n, x0.ctypes.data, eps.ctypes.data, eps_scale, y_out.ctypes.data),
               "fi_generate_host")

    def generate_host_ptr(self, n: int, x0_ptr: int, eps_ptr: int, y_ptr: int, eps_scale: float = 0.1):
        _check(lib.fi_generate_host(self._h, n, x0_ptr, eps_ptr, eps_scale, y_ptr), "fi_generate_host")

    def generate_lazy(self, n: int, x0, eps, y_out, eps_scale: float = 0.1):
        _check(lib.fi_generate_lazy(self._h, n, _ptr(x0), _ptr(eps), eps_scale, _ptr(y_out)), "fi_generate_lazy")

    def sync(self):
        _check(lib.fi_sync(self._h), "fi_sync")

    def reset(self):
        _check(lib.fi_reset(self._h), "fi_reset")

    def set_wait_limit(self, limit: int):
        _check(lib.fi_debug_set_wait_limit(self._h, limit), "fi_debug_set_wait_limit")

    @property
    def position(self) -> int:
        p = ctypes.c_int32()
        _check(lib.fi_position(self._h, ctypes.byref(p)), "fi_position")
        return p.value

    def read_activations(self, layer: int, dst):
        _check(lib.fi_read_activations(self._h, layer, _ptr(dst)), "fi_read_activations")

    def plan(self):
        """(chunk, fft_from, tc_max) after automatic selection; 0 = that kind of block is not used."""
        c, f, t = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
        _check(lib.fi_get_plan(self._h, ctypes.byref(c), ctypes.byref(f), ctypes.byref(t)), "fi_get_plan")
        return c.value, f.value, t.value

    def profile(self, enable: bool):
        _check(lib.fi_profile(self._h, 1 if enable else 0), "fi_profile")

    def profile_read(self):
        counts = (ctypes.c_int32 * NUM_KERNEL_CLASSES)()
        ms = (ctypes.c_double * NUM_KERNEL_CLASSES)()
        _check(lib.fi_profile_read(self._h, counts, ms), "fi_profile_read")
        return {KERNEL_CLASSES[k]: (counts[k], ms[k]) for k in range(NUM_KERNEL_CLASSES)}

    def profile_read_sides(self):
        """(per-class dict as profile_read, {block side: (launches, ms)})."""
        counts = (ctypes.c_int32 * NUM_KERNEL_CLASSES)()
        ms = (ctypes.c_double * NUM_KERNEL_CLASSES)()
        sc = (ctypes.c_int32 * 32)()
        sm = (ctypes.c_double * 32)()
        _check(lib.fi_profile_read_sides(self._h, counts, ms, sc, sm), "fi_profile_read_sides")
        return ({KERNEL_CLASSES[k]: (counts[k], ms[k]) for k in range(NUM_KERNEL_CLASSES)},
                {1 << q: (sc[q], sm[q]) for q in range(32) if sc[q]})


def debug_fft(log2n: int, x, out, inverse: bool = False, stream=None):
    """The library's device FFT on x (complex64 CUDA tensor [count][2^log2n]) into out."""
    count = x.numel() >> log2n
    _check(lib.fi_debug_fft(log2n, count, _ptr(x), _ptr(out), 1 if inverse else 0, _stream(stream)), "fi_debug_fft")


def generate_noalloc(h, batch: int, n: int, x0, eps, y_out, dtype: str = "f32", eps_scale: float = 0.1,
                     chunk: int = 0, stream=None):
    """fi_generate_noalloc: one generation from position 0 with no device allocation."""
    M, D, L = (int(v) for v in h.shape)
    cfg = Config(M, D, L, int(batch), FI_BF16 if dtype == "bf16" else FI_F32, chunk, 0)
    _check(lib.fi_generate_noalloc(ctypes.byref(cfg), _ptr(h), n, _ptr(x0), _ptr(eps), eps_scale, _ptr(y_out),
                                   _stream(stream)), "fi_generate_noalloc")


# -- operators (no context): linear attention and the linear layer; inference only, autograd does
# not see what they write
#
# What a call's tensors look like (shapes, strides, types, devices) is checked once
# per combination and kept with the configuration it gives; of the tensors' addresses
# only the alignment is part of it, where scratch depends on it.

_DTYPE_CODE = {}          # torch dtype -> fi_dtype, filled on first use
_configs: dict = {}       # what the tensors look like -> (address of the configuration, scratch bytes, the configuration)


def _look(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _keep(key, cfg, need=0):
    if len(_configs) >= 4096:      # a program with ever new sizes does not grow without bound
        _configs.clear()
    got = _configs[key] = (ctypes.addressof(cfg), need, cfg)
    return got


def _check_sizes(*shapes):
    """The C structures hold sizes in 32 bits; larger ones would pass as their remainder."""
    if any(n > 2 ** 31 - 1 for shape in shapes for n in shape):
        raise ValueError("a dimension is larger than 2^31 - 1")


def _current(dev):
    import torch
    if torch._C._cuda_getDevice() != dev:
        raise ValueError(f"the tensors are on cuda:{dev}, which is not the current device")


def _op_stream(stream, dev):
    """The stream of a call whose tensors are on CUDA device `dev`, which must be the current one."""
    import torch
    _current(dev)
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _scratch(need, like, stream, st):
    """Scratch of one call, from the memory of the call's stream: whatever used it before, and whatever
    is given it next, runs on that stream as well."""
    import torch
    if stream is None:
        return torch.empty(need, dtype=torch.uint8, device=like.device)
    with torch.cuda.stream(torch.cuda.ExternalStream(st, device=like.device) if st else torch.cuda.default_stream(like.device)):
        return torch.empty(need, dtype=torch.uint8, device=like.device)


def _check_tensors(tensors, dtype):
    """One CUDA device, the current one (scratch sizes depend on it), and one of the library's types for
    those of `tensors` that are not None; its code."""
    import torch
    if not _DTYPE_CODE:
        _DTYPE_CODE.update({torch.float32: FI_F32, torch.bfloat16: FI_BF16})
    if dtype not in _DTYPE_CODE:
        raise ValueError(f"expected float32 or bfloat16 tensors, got {dtype}")
    devices = {t.get_device() for t in tensors if t is not None}
    if len(devices) != 1 or -1 in devices:
        raise ValueError("expected CUDA tensors on one device")
    _current(devices.pop())
    return _DTYPE_CODE[dtype]


def _linattn_config(key, q, k, v, log_decay, o, states, lengths, scale, n):
    """Checks the tensors of a linear-attention call and keeps its configuration; n: positions, or
    None for a step, whose tensors have no position dimension."""
    import torch
    code = _check_tensors((q, k, v, log_decay, o, lengths, *states), q.dtype)
    lead, want = ("", 3) if n is None else ("[n]", 4)
    if q.dim() != want or k.shape != q.shape or o.shape != v.shape or v.dim() != want or v.shape[:-1] != q.shape[:-1]:
        raise ValueError(f"expected q, k {lead}[B][H][key_dim] and v, o {lead}[B][H][value_dim]")
    _check_sizes(q.shape, v.shape)
    if not (k.dtype == v.dtype == o.dtype == q.dtype):
        raise ValueError("q, k, v and o must have one dtype")
    if any(t.shape[-1] > 1 and t.stride(-1) != 1 for t in (q, k, v, o)):
        raise ValueError("the innermost dimension of q, k, v and o must be contiguous")
    B, H, dk, dv = *(int(x) for x in q.shape[-3:]), int(v.shape[-1])
    if log_decay.shape != (H,) or log_decay.dtype != torch.float32 or not log_decay.is_contiguous():
        raise ValueError(f"log_decay must be a contiguous float32 tensor [{H}]")
    if lengths is not None and (lengths.shape != (B,) or lengths.dtype != torch.int32 or not lengths.is_contiguous()):
        raise ValueError(f"lengths must be a contiguous int32 tensor [{B}]")
    for s in states:
        if s is not None and (s.shape != (B, H, dk, dv) or s.dtype != torch.float32 or not s.is_contiguous()):
            raise ValueError(f"a state must be a contiguous float32 tensor [{B}][{H}][{dk}][{dv}]")
    cfg = LinattnConfig(H, dk, dv, B, code, scale)
    for name, t in (("q_stride", q), ("k_stride", k), ("v_stride", v), ("o_stride", o)):
        getattr(cfg, name)[:] = t.stride()[:-1] if n is not None else (0, *t.stride()[:-1])
    need = ctypes.c_uint64()
    if n is not None:
        _check(lib.fi_linattn_workspace(ctypes.addressof(cfg), n, q.data_ptr(), k.data_ptr(), v.data_ptr(), ctypes.byref(need)),
               "fi_linattn_workspace")
    return _keep(key, cfg, need.value)


def linattn_prefill(q, k, v, log_decay, o, state_in=None, state_out=None, lengths=None, scale: float = 1.0, stream=None):
    """Linear attention with a decay per head over a prompt (fi_linattn_prefill):
    S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T, o_t = scale q_t^T S_t.

    q, k [n][B][H][key_dim], v, o [n][B][H][value_dim], float32 or bfloat16, any
    strides with a contiguous innermost dimension; log_decay [H] float32;
    lengths [B] int32 or None; state_in, state_out [B][H][key_dim][value_dim]
    float32, contiguous, or None (they may be the same tensor)."""
    scale = float(scale)      # part of what is kept: by its value, whatever holds it
    pq, pk, pv = q.data_ptr(), k.data_ptr(), v.data_ptr()
    key = (q.shape, k.shape, v.shape, o.shape, q.stride(), k.stride(), v.stride(), o.stride(), q.dtype, k.dtype, v.dtype,
           o.dtype, q.get_device(), k.get_device(), v.get_device(), o.get_device(), _look(log_decay), _look(state_in),
           _look(state_out), _look(lengths), scale, pq & 15, pk & 15, pv & 15)
    at, need, _cfg = _configs.get(key) or _linattn_config(key, q, k, v, log_decay, o, (state_in, state_out), lengths, scale,
                                                       int(q.shape[0]))
    st = _op_stream(stream, key[12])
    ws = _scratch(need, q, stream, st) if need else None
    s = lib.fi_linattn_prefill(at, q.shape[0], pq, pk, pv, log_decay.data_ptr(),
                               None if lengths is None else lengths.data_ptr(),
                               None if state_in is None else state_in.data_ptr(),
                               None if state_out is None else state_out.data_ptr(), o.data_ptr(),
                               None if ws is None else ws.data_ptr(), need, st)
    if s:
        _check(s, "fi_linattn_prefill")


def linattn_step(q, k, v, log_decay, state, o, scale: float = 1.0, stream=None):
    """One position of every sequence (fi_linattn_step): q, k [B][H][key_dim],
    v, o [B][H][value_dim], state [B][H][key_dim][value_dim] float32, updated in place."""
    scale = float(scale)
    key = (q.shape, k.shape, v.shape, o.shape, q.stride(), k.stride(), v.stride(), o.stride(), q.dtype, k.dtype, v.dtype,
           o.dtype, q.get_device(), k.get_device(), v.get_device(), o.get_device(), state.shape, state.stride(),
           state.dtype, state.get_device(), log_decay.shape, log_decay.stride(), log_decay.dtype, log_decay.get_device(),
           scale)
    at, _, _cfg = _configs.get(key) or _linattn_config(key, q, k, v, log_decay, o, (state,), None, scale, None)   # held by _cfg
    s = lib.fi_linattn_step(at, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), state.data_ptr(),
                            o.data_ptr(), _op_stream(stream, key[12]))
    if s:
        _check(s, "fi_linattn_step")


def _linear_config(key, x, w, y, bias, residual, act):
    code = _check_tensors((x, w, y, bias, residual), x.dtype)
    if x.dim() != 2 or w.dim() != 2 or y.dim() != 2 or x.shape[1] != w.shape[1] or tuple(y.shape) != (x.shape[0], w.shape[0]):
        raise ValueError("expected x [n][in], w [out][in] and y [n][out]")
    _check_sizes(x.shape, w.shape)
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}")
    if any(t is not None and t.dtype != x.dtype for t in (w, y, bias, residual)):
        raise ValueError("x, w, y, bias and residual must have one dtype")
    if bias is not None and (tuple(bias.shape) != (w.shape[0],) or not bias.is_contiguous()):
        raise ValueError("bias must be contiguous, [out]")
    if residual is not None and residual.shape != y.shape:
        raise ValueError("residual must have y's shape")
    if any(t is not None and t.shape[-1] > 1 and t.stride(-1) != 1 for t in (x, w, y, residual)):
        raise ValueError("the rows of x, w, y and residual must be contiguous")
    nin, nout = int(x.shape[1]), int(w.shape[0])

    def ld(t, cols):     # the stride of a single row says nothing
        return int(t.stride(0)) if t.shape[0] > 1 else cols

    cfg = LinearConfig(nin, nout, code, ACTIVATIONS[act], ld(x, nin), ld(w, nin),
                       nout if residual is None else ld(residual, nout), ld(y, nout))
    need = ctypes.c_uint64()
    _check(lib.fi_linear_workspace(ctypes.addressof(cfg), x.shape[0], x.data_ptr(), w.data_ptr(), ctypes.byref(need)),
           "fi_linear_workspace")
    return _keep(key, cfg, need.value)


def linear(x, w, y, bias=None, residual=None, act: str = "none", stream=None):
    """y = act(x w^T + bias) + residual (fi_linear): x [n][in], w [out][in], y and
    residual [n][out], bias [out], all float32 or all bfloat16, rows of any stride
    with contiguous elements. act: none, gelu, silu, relu or tanh. residual may be y.
    A float32 operand that is not finite makes act's argument not finite (NaN or an infinity)."""
    px, pw = x.data_ptr(), w.data_ptr()
    key = (x.shape, w.shape, y.shape, x.stride(), w.stride(), y.stride(), x.dtype, w.dtype, y.dtype, x.get_device(),
           w.get_device(), y.get_device(), _look(bias), _look(residual), act, px & 15, pw & 15)
    at, need, _cfg = _configs.get(key) or _linear_config(key, x, w, y, bias, residual, act)
    st = _op_stream(stream, key[9])
    ws = _scratch(need, x, stream, st) if need else None
    s = lib.fi_linear(at, x.shape[0], px, pw, None if bias is None else bias.data_ptr(),
                      None if residual is None else residual.data_ptr(), y.data_ptr(),
                      None if ws is None else ws.data_ptr(), need, st)
    if s:
        _check(s, "fi_linear")


def op_sync(stream=None):
    """Waits for the stream; raises FiError (FI_E_TIMEOUT) if a bounded wait in an operator's kernel gave up."""
    _check(lib.fi_op_sync(_stream(stream)), "fi_op_sync")


def set_op_wait_limit(limit: int):
    """Test hook: barrier checks after which a wait in an operator's kernel gives up (negative: the default)."""
    _check(lib.fi_debug_set_op_wait_limit(limit), "fi_debug_set_op_wait_limit")


def chunk_schedule(chunk: int, retimed: bool, coarse: bool = False):
    """The chunk kernel's table of on-chip block pieces (host only): (lags the
    chain adds itself, [(step, first source, sources, first target, targets)]),
    chunk-relative. coarse: the cut used for stacks of at most 8 layers."""
    cap = 4 * chunk
    out = (ctypes.c_int32 * (5 * cap))()
    n, lags = ctypes.c_int32(), ctypes.c_int32()
    mode = (2 if coarse else 1) if retimed else 0
    _check(lib.fi_debug_chunk_schedule(chunk, mode, ctypes.cast(out, ctypes.c_void_p), cap,
                                       ctypes.byref(n), ctypes.byref(lags)), "fi_debug_chunk_schedule")
    return lags.value, [tuple(out[5 * j: 5 * j + 5]) for j in range(min(n.value, cap))]


def status_str(s: int) -> str:
    return lib.fi_status_str(s).decode()
