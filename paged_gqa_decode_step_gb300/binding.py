"""ctypes binding of libpdattn (include/pdattn.h).

Argument marshalling only: every function takes torch tensors that already
live on the GPU, checks their shapes and dtypes against the parameters, and
passes raw device pointers and the current CUDA stream to the C-ABI call of
the same name.  No computation happens here, and there is no fallback: if the
library is missing, importing this module raises.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libpdattn.so")

OK, EINVAL, EUNSUPPORTED, ECUDA, EBADPAGE, ETIMEOUT, EBADPOS, ENOPAGES = range(8)
BF16, F32 = 0, 1
_DTYPES = {torch.bfloat16: BF16, torch.float32: F32}


class PdattnError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"pdattn status {status}: {msg}")
        self.status = status


class Params(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int32), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("pages_per_row", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("window", ctypes.c_int32), ("scale", ctypes.c_float), ("rope_cos", ctypes.c_void_p),
        ("rope_sin", ctypes.c_void_p), ("rope_len", ctypes.c_int32), ("chunk_pages", ctypes.c_int32),
        ("sinks", ctypes.c_void_p),
    ]


class Layer(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p),
        ("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("window", ctypes.c_int32), ("reserved", ctypes.c_int32), ("sinks", ctypes.c_void_p),
    ]


class CodedCache(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("code", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


class RotarySpec(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
        ("scaling", ctypes.c_int32), ("original_len", ctypes.c_int32), ("whole_pairs", ctypes.c_int32),
        ("theta", ctypes.c_double), ("factor", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double),
        ("gain", ctypes.c_double),
    ]


class Rotary(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
        ("gain", ctypes.c_float), ("made", ctypes.c_uint32), ("reserved", ctypes.c_uint32),
        ("turns", ctypes.c_uint64 * 64),
    ]


class Pool(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("heads", ctypes.c_int32), ("row_bytes", ctypes.c_int32)]


LAYERS_PER_LAUNCH = 32
SCALINGS = {"none": 0, "linear": 1, "wavelength": 2, "ramp": 3}
STATUS_BYTES = 256
E4M3, INT8 = 0, 1
_CODES = {torch.float8_e4m3fn: E4M3, torch.int8: INT8}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m paged_gqa_decode_step_gb300.build` (nvcc, sm_103a)")
    L = ctypes.CDLL(LIB_PATH)
    vp, sz, i32, P = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.POINTER(Params)
    i64 = ctypes.c_int64
    sig = {
        "pdattn_workspace_size": (sz, [P]),
        "pdattn_rope_tables": (i32, [ctypes.c_float, i32, i32, i32, vp, vp, vp]),
        "pdattn_rope_write_kv": (i32, [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "pdattn_plan": (i32, [P, vp, vp, sz, vp]),
        "pdattn_attend": (i32, [P, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "pdattn_decode": (i32, [P, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "pdattn_decode_fused": (i32, [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "pdattn_decode_fused_noalloc": (i32, [P, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "pdattn_layers_workspace_size": (sz, [P, i32]),
        "pdattn_decode_layers": (i32, [P, i32, ctypes.POINTER(Layer), vp, vp, vp, sz, vp]),
        "pdattn_shared_workspace_size": (sz, [P, i32]),
        "pdattn_decode_shared": (i32, [P, i32] + [vp] * 11 + [sz, vp]),
        "pdattn_prefill_workspace_size": (sz, [P, i32]),
        "pdattn_prefill_paged": (i32, [P, i32] + [vp] * 11 + [sz, vp]),
        "pdattn_prefill_attend": (i32, [P, i32] + [vp] * 6 + [sz, vp]),
        "pdattn_packed_workspace_size": (sz, [P, i32]),
        "pdattn_packed": (i32, [P, i32] + [vp] * 7 + [sz, vp]),
        "pdattn_packed_attend": (i32, [P, i32] + [vp] * 4 + [sz, vp]),
        "pdattn_coded_workspace_size": (sz, [P, i32]),
        "pdattn_coded_write": (i32, [P, ctypes.POINTER(CodedCache), i32] + [vp] * 5 + [sz, vp]),
        "pdattn_coded_read": (i32, [P, ctypes.POINTER(CodedCache), i32] + [vp] * 4 + [sz, vp]),
        "pdattn_coded_decode": (i32, [P, ctypes.POINTER(CodedCache)] + [vp] * 7 + [sz, vp]),
        "pdattn_coded_prefill": (i32, [P, ctypes.POINTER(CodedCache), i32] + [vp] * 9 + [sz, vp]),
        "pdattn_rotary_make": (i32, [ctypes.POINTER(RotarySpec), ctypes.POINTER(Rotary)]),
        "pdattn_rotary_tables": (i32, [ctypes.POINTER(Rotary), i32, i32, vp, vp, vp]),
        "pdattn_rotary_apply": (i32, [ctypes.POINTER(Rotary), i32, i32, i32, i32, vp, i64, vp, i64, i32, vp, i64, vp,
                                      i64, vp, vp, sz, vp]),
        "pdattn_pages_workspace_size": (sz, [P]),
        "pdattn_pages_update": (i32, [P, i32, ctypes.POINTER(Pool)] + [vp] * 8 + [sz, vp]),
        "pdattn_pages_compact": (i32, [P, i32, ctypes.POINTER(Pool)] + [vp] * 7 + [sz, vp]),
        "pdattn_check_status": (i32, [vp, vp]),
        "pdattn_last_error": (ctypes.c_char_p, []),
        "pdattn_last_launch_count": (i32, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    return L


lib = _load()


def _check(status):
    if status != OK:
        raise PdattnError(status, lib.pdattn_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def make_params(rows, heads, kv_heads, head_dim, pages_per_row, num_pages, dtype, window=0, scale=0.0,
                rope_cos=None, rope_sin=None, chunk_pages=0, sinks=None):
    """Parameter block; rope tables (torch tensors [len, D]) keep rotation on;
    sinks: optional [heads] tensor of the element type (attention sinks)."""
    p = Params(rows, heads, kv_heads, head_dim, 64, pages_per_row, num_pages, _DTYPES[dtype], window,
               scale, None, None, 0, chunk_pages, None)
    if sinks is not None:
        _expect("sinks", sinks, (heads,), dtype)
        p.sinks = sinks.data_ptr()
        p._sinks = sinks
    if rope_cos is not None:
        for name, t in (("rope_cos", rope_cos), ("rope_sin", rope_sin)):
            _expect(name, t, (rope_cos.shape[0], head_dim), dtype)
        p.rope_cos, p.rope_sin, p.rope_len = rope_cos.data_ptr(), rope_sin.data_ptr(), rope_cos.shape[0]
        # the block holds raw pointers: keep the tables alive as long as it lives
        p._tables = (rope_cos, rope_sin)
    devices = {t.get_device() for t in (sinks, rope_cos, rope_sin) if t is not None}
    if len(devices) > 1:
        raise ValueError("rope tables and sinks are on different devices")
    p._device = devices.pop() if devices else None
    return p


def workspace_size(p):
    n = lib.pdattn_workspace_size(ctypes.byref(p))
    if n == 0:
        raise PdattnError(EINVAL, lib.pdattn_last_error().decode())
    return n


def new_workspace(p, device="cuda"):
    """A zero-filled workspace of the right size (uint8 tensor, 256-byte aligned)."""
    return torch.zeros(workspace_size(p), dtype=torch.uint8, device=device)


def rope_tables(theta, head_dim, length, dtype, device="cuda", stream=None):
    cos = torch.empty(length, head_dim, dtype=dtype, device=device)
    sin = torch.empty(length, head_dim, dtype=dtype, device=device)
    _check(lib.pdattn_rope_tables(theta, head_dim, length, _DTYPES[dtype], _ptr(cos), _ptr(sin), _stream(stream)))
    return cos, sin


def _ws(ws):
    if not (ws.is_cuda and ws.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return _ptr(ws), ws.numel() * ws.element_size()


def _expect(name, t, shape, dtype):
    """Shape, dtype, device and contiguity of one argument."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _dt(p):
    return torch.bfloat16 if p.dtype == BF16 else torch.float32


def _check_common(p, positions, table, k_pool, v_pool):
    _expect("positions", positions, (p.rows,), torch.int32)
    _expect("table", table, (p.rows, p.pages_per_row), torch.int32)
    pool = (p.num_pages, p.kv_heads, 64, p.head_dim)
    _expect("k_pool", k_pool, pool, _dt(p))
    _expect("v_pool", v_pool, pool, _dt(p))


def _check_q(p, **named):
    for name, t in named.items():
        h = p.heads if name in ("q", "q_rot", "q_out", "out") else p.kv_heads
        _expect(name, t, (p.rows, h, p.head_dim), _dt(p))


def rope_write_kv(p, q, k_new, v_new, positions, table, q_out, k_pool, v_pool, ws, stream=None):
    _check_common(p, positions, table, k_pool, v_pool)
    _check_q(p, q=q, k_new=k_new, v_new=v_new, q_out=q_out)
    w, n = _ws(ws)
    _check(lib.pdattn_rope_write_kv(ctypes.byref(p), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(positions),
                                    _ptr(table), _ptr(q_out), _ptr(k_pool), _ptr(v_pool), w, n, _stream(stream)))


def plan(p, positions, ws, stream=None):
    _expect("positions", positions, (p.rows,), torch.int32)
    w, n = _ws(ws)
    _check(lib.pdattn_plan(ctypes.byref(p), _ptr(positions), w, n, _stream(stream)))


def attend(p, q_rot, positions, table, k_pool, v_pool, out, ws, stream=None):
    _check_common(p, positions, table, k_pool, v_pool)
    _check_q(p, q_rot=q_rot, out=out)
    w, n = _ws(ws)
    _check(lib.pdattn_attend(ctypes.byref(p), _ptr(q_rot), _ptr(positions), _ptr(table), _ptr(k_pool),
                             _ptr(v_pool), _ptr(out), w, n, _stream(stream)))


def decode(p, q_rot, positions, table, k_pool, v_pool, out, ws, stream=None):
    _check_common(p, positions, table, k_pool, v_pool)
    _check_q(p, q_rot=q_rot, out=out)
    w, n = _ws(ws)
    _check(lib.pdattn_decode(ctypes.byref(p), _ptr(q_rot), _ptr(positions), _ptr(table), _ptr(k_pool),
                             _ptr(v_pool), _ptr(out), w, n, _stream(stream)))


def decode_fused(p, q, k_new, v_new, positions, table, k_pool, v_pool, out, ws, stream=None):
    _check_common(p, positions, table, k_pool, v_pool)
    _check_q(p, q=q, k_new=k_new, v_new=v_new, out=out)
    w, n = _ws(ws)
    _check(lib.pdattn_decode_fused(ctypes.byref(p), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(positions),
                                   _ptr(table), _ptr(k_pool), _ptr(v_pool), _ptr(out), w, n, _stream(stream)))


def decode_fused_noalloc(p, q, k_new, v_new, positions, table, k_pool, v_pool, out, stream=None):
    """decode_fused with the library's fixed scratch array instead of a workspace."""
    _check_common(p, positions, table, k_pool, v_pool)
    _check_q(p, q=q, k_new=k_new, v_new=v_new, out=out)
    _check(lib.pdattn_decode_fused_noalloc(ctypes.byref(p), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(positions),
                                           _ptr(table), _ptr(k_pool), _ptr(v_pool), _ptr(out), _stream(stream)))


def layers_workspace_size(p, n_layers):
    n = lib.pdattn_layers_workspace_size(ctypes.byref(p), n_layers)
    if n == 0:
        raise PdattnError(EINVAL, lib.pdattn_last_error().decode() or "invalid parameters")
    return n


def new_layers_workspace(p, n_layers, device="cuda"):
    return torch.zeros(layers_workspace_size(p, n_layers), dtype=torch.uint8, device=device)


def decode_layers(p, layers, positions, table, ws, stream=None):
    """The decode step of several layers in one group of launches (per 32 layers).
    layers: a sequence of dicts with q, k_new, v_new, k_pool, v_pool, out
    (tensors shaped as for decode_fused) and optional window (int) and sinks
    ([heads] tensor); p.window and p.sinks are not read."""
    _expect("positions", positions, (p.rows,), torch.int32)
    _expect("table", table, (p.rows, p.pages_per_row), torch.int32)
    arr = (Layer * max(1, len(layers)))()
    keep = []
    pool = (p.num_pages, p.kv_heads, 64, p.head_dim)
    for i, y in enumerate(layers):
        _check_q(p, q=y["q"], k_new=y["k_new"], v_new=y["v_new"], out=y["out"])
        _expect("k_pool", y["k_pool"], pool, _dt(p))
        _expect("v_pool", y["v_pool"], pool, _dt(p))
        sinks = y.get("sinks")
        if sinks is not None:
            _expect("sinks", sinks, (p.heads,), _dt(p))
        arr[i] = Layer(y["q"].data_ptr(), y["k_new"].data_ptr(), y["v_new"].data_ptr(), y["k_pool"].data_ptr(),
                       y["v_pool"].data_ptr(), y["out"].data_ptr(), int(y.get("window", 0)), 0,
                       None if sinks is None else sinks.data_ptr())
        keep.append(y)
    w, n = _ws(ws)
    _check(lib.pdattn_decode_layers(ctypes.byref(p), len(layers), arr, _ptr(positions), _ptr(table), w, n,
                                    _stream(stream)))


def prefill_workspace_size(p, n_tokens):
    n = lib.pdattn_prefill_workspace_size(ctypes.byref(p), n_tokens)
    if n == 0:
        raise PdattnError(EINVAL, lib.pdattn_last_error().decode() or "invalid parameters")
    return n


def new_prefill_workspace(p, n_tokens, device="cuda"):
    return torch.zeros(prefill_workspace_size(p, n_tokens), dtype=torch.uint8, device=device)


def prefill_paged(p, q, k_new, v_new, positions, rows, slots, table, k_pool, v_pool, out, ws, stream=None):
    """Packed prompt tokens: q / out [P, heads, D], k_new / v_new [P, kv_heads, D],
    positions / rows / slots [P] int32; p.rows is the number of table rows."""
    n = q.shape[0] if isinstance(q, torch.Tensor) else -1
    _expect("table", table, (p.rows, p.pages_per_row), torch.int32)
    pool = (p.num_pages, p.kv_heads, 64, p.head_dim)
    _expect("k_pool", k_pool, pool, _dt(p))
    _expect("v_pool", v_pool, pool, _dt(p))
    for name, t in (("positions", positions), ("rows", rows), ("slots", slots)):
        _expect(name, t, (n,), torch.int32)
    for name, t, h in (("q", q, p.heads), ("k_new", k_new, p.kv_heads), ("v_new", v_new, p.kv_heads),
                       ("out", out, p.heads)):
        _expect(name, t, (n, h, p.head_dim), _dt(p))
    w, nb = _ws(ws)
    _check(lib.pdattn_prefill_paged(ctypes.byref(p), n, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(positions),
                                    _ptr(rows), _ptr(slots), _ptr(table), _ptr(k_pool), _ptr(v_pool), _ptr(out),
                                    w, nb, _stream(stream)))


def prefill_attend(p, positions, table, k_pool, v_pool, out, ws, stream=None):
    """Attention half of prefill_paged, over what its last call left in ws."""
    n = out.shape[0] if isinstance(out, torch.Tensor) else -1
    _expect("positions", positions, (n,), torch.int32)
    _expect("table", table, (p.rows, p.pages_per_row), torch.int32)
    pool = (p.num_pages, p.kv_heads, 64, p.head_dim)
    _expect("k_pool", k_pool, pool, _dt(p))
    _expect("v_pool", v_pool, pool, _dt(p))
    _expect("out", out, (n, p.heads, p.head_dim), _dt(p))
    w, nb = _ws(ws)
    _check(lib.pdattn_prefill_attend(ctypes.byref(p), n, _ptr(positions), _ptr(table), _ptr(k_pool), _ptr(v_pool),
                                     _ptr(out), w, nb, _stream(stream)))


def new_packed_workspace(p, n_tokens, device="cuda"):
    n = lib.pdattn_packed_workspace_size(ctypes.byref(p), n_tokens)
    if n == 0:
        raise PdattnError(EINVAL, lib.pdattn_last_error().decode() or "invalid parameters")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def packed(p, q, k, v, positions, segments, out, ws, stream=None):
    """Sequences packed into one row: q / out [n, heads, D], k / v [n, kv_heads, D],
    positions / segments [n] int32."""
    n = q.shape[0] if isinstance(q, torch.Tensor) else -1
    for name, t in (("positions", positions), ("segments", segments)):
        _expect(name, t, (n,), torch.int32)
    for name, t, h in (("q", q, p.heads), ("k", k, p.kv_heads), ("v", v, p.kv_heads), ("out", out, p.heads)):
        _expect(name, t, (n, h, p.head_dim), _dt(p))
    w, nb = _ws(ws)
    _check(lib.pdattn_packed(ctypes.byref(p), n, _ptr(q), _ptr(k), _ptr(v), _ptr(positions), _ptr(segments),
                             _ptr(out), w, nb, _stream(stream)))


def packed_attend(p, v, positions, out, ws, stream=None):
    """Attention half of packed, over what its last call left in ws."""
    n = out.shape[0] if isinstance(out, torch.Tensor) else -1
    _expect("positions", positions, (n,), torch.int32)
    _expect("v", v, (n, p.kv_heads, p.head_dim), _dt(p))
    _expect("out", out, (n, p.heads, p.head_dim), _dt(p))
    w, nb = _ws(ws)
    _check(lib.pdattn_packed_attend(ctypes.byref(p), n, _ptr(v), _ptr(positions), _ptr(out), w, nb, _stream(stream)))


def make_coded_cache(p, k, v, k_scale, v_scale):
    """Descriptor of a coded (8-bit) cache: codes k, v [num_pages, kv_heads, 64, D]
    of torch.float8_e4m3fn or torch.int8 and their scales [num_pages, kv_heads, 64] f32."""
    if not isinstance(k, torch.Tensor) or k.dtype not in _CODES:
        raise ValueError("codes must be torch.float8_e4m3fn or torch.int8 tensors")
    pool = (p.num_pages, p.kv_heads, 64, p.head_dim)
    for name, t in (("k", k), ("v", v)):
        _expect(name, t, pool, k.dtype)
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        _expect(name, t, pool[:3], torch.float32)
    _same_device(k, v, k_scale, v_scale)
    c = CodedCache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), _CODES[k.dtype], 0)
    # the block holds raw pointers: keep the tensors alive as long as it lives
    c._tensors = (k, v, k_scale, v_scale)
    c._pool, c._device = pool, k.get_device()
    return c


def new_coded_cache(p, code=torch.float8_e4m3fn, device="cuda"):
    """An empty coded cache of p's pool shape (codes and scales zero); its tensors are
    in cache._tensors: k, v, k_scale, v_scale."""
    pool = (p.num_pages, p.kv_heads, 64, p.head_dim)
    codes = [torch.zeros(pool, dtype=torch.uint8, device=device).view(code) for _ in range(2)]
    return make_coded_cache(p, *codes, *(torch.zeros(pool[:3], dtype=torch.float32, device=device) for _ in range(2)))


def coded_workspace_size(p, n_tokens=0):
    n = lib.pdattn_coded_workspace_size(ctypes.byref(p), n_tokens)
    if n == 0:
        raise PdattnError(EINVAL, lib.pdattn_last_error().decode() or "invalid parameters")
    return n


def new_coded_workspace(p, n_tokens=0, device="cuda"):
    """A workspace for the coded calls: coded_decode of p.rows rows, coded_prefill of up to n_tokens tokens."""
    return torch.zeros(coded_workspace_size(p, n_tokens), dtype=torch.uint8, device=device)


def _same_device(*tensors):
    """Every tensor on the current device: the calls launch there."""
    here = torch.cuda.current_device()
    for t in tensors:
        if t.get_device() != here:
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{here}")
    return here


def _check_coded(p, cache, ws, n, heads, ints, table, **named):
    """Arguments of a coded call: `named` of [n, heads, D] (heads by name), ints of [n] int32."""
    if not isinstance(cache, CodedCache) or not hasattr(cache, "_pool"):
        raise TypeError("cache must come from make_coded_cache or new_coded_cache")
    if cache._pool != (p.num_pages, p.kv_heads, 64, p.head_dim):
        raise ValueError(f"cache has pools {cache._pool}, the parameters another shape")
    here = torch.cuda.current_device()
    if getattr(p, "_device", None) not in (None, here):
        raise ValueError(f"rope tables or sinks are on cuda:{p._device}, the current device is cuda:{here}")
    dt, D, Hk, Hq = _dt(p), p.head_dim, p.kv_heads, p.heads
    kv, qs = (n, Hk, D), (n, Hq, D)
    # one pass over each tensor's attributes; _expect names what is wrong
    for name, t in named.items():
        shape = qs if name in heads else kv
        if not (isinstance(t, torch.Tensor) and t.dtype is dt and t.shape == shape and t.get_device() == here
                and t.is_contiguous()):
            _expect(name, t, shape, dt)
            _same_device(t)
    for name, t in ints.items():
        if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.shape == (n,) and t.get_device() == here
                and t.is_contiguous()):
            _expect(name, t, (n,), torch.int32)
            _same_device(t)
    if table is not None:
        shape = (p.rows, p.pages_per_row)
        if not (isinstance(table, torch.Tensor) and table.dtype is torch.int32 and table.shape == shape
                and table.get_device() == here and table.is_contiguous()):
            _expect("table", table, shape, torch.int32)
            _same_device(table)
    if not isinstance(ws, torch.Tensor):
        raise TypeError("workspace must be a torch tensor")
    if cache._device != here or ws.get_device() != here or not ws.is_contiguous():
        _ws(ws)
        _same_device(cache._tensors[0], ws)


# Torch's own short ways to the current device and to a stream's handle (the
# public ones take three times as long, and 3 us for a Stream object); where a
# version of torch lacks them, the public ones.
_get_device = getattr(torch._C, "_cuda_getDevice", None)
_get_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _here():
    """The current device, -1 without a GPU."""
    if _get_device is not None and torch.cuda.is_initialized():
        return _get_device()
    return torch.cuda.current_device() if torch.cuda.is_available() else -1


def _stream_of(stream, here):
    if stream is not None:
        return stream.cuda_stream
    return _get_raw_stream(here) if _get_raw_stream is not None else torch.cuda.current_stream(here).cuda_stream


def _tokens(t):
    return t.shape[0] if isinstance(t, torch.Tensor) and t.dim() else -1


def _raw_stream(stream):
    return stream.cuda_stream if stream is not None else _stream_of(None, torch.cuda.current_device())


def coded_write(p, cache, k_new, v_new, positions, slots, ws, stream=None):
    """Codes of new keys (rotated at positions) and values [n, kv_heads, D] into pool slots [n] int32."""
    n = _tokens(k_new)
    _check_coded(p, cache, ws, n, (), dict(positions=positions, slots=slots), None, k_new=k_new, v_new=v_new)
    _check(lib.pdattn_coded_write(p, cache, n, k_new.data_ptr(), v_new.data_ptr(), positions.data_ptr(),
                                  slots.data_ptr(), ws.data_ptr(), ws.nbytes, _raw_stream(stream)))


def coded_read(p, cache, slots, k_out, v_out, ws, stream=None):
    """What the codes of pool slots [n] int32 stand for, as k_out, v_out [n, kv_heads, D]."""
    n = _tokens(slots)
    _check_coded(p, cache, ws, n, (), dict(slots=slots), None, k_out=k_out, v_out=v_out)
    _check(lib.pdattn_coded_read(p, cache, n, slots.data_ptr(), k_out.data_ptr(), v_out.data_ptr(), ws.data_ptr(),
                                 ws.nbytes, _raw_stream(stream)))


def coded_decode(p, cache, q, k_new, v_new, positions, table, out, ws, stream=None):
    """decode_fused over a coded cache."""
    _check_coded(p, cache, ws, p.rows, ("q", "out"), dict(positions=positions), table, q=q, k_new=k_new, v_new=v_new,
                 out=out)
    _check(lib.pdattn_coded_decode(p, cache, q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), positions.data_ptr(),
                                   table.data_ptr(), out.data_ptr(), ws.data_ptr(), ws.nbytes, _raw_stream(stream)))


def coded_prefill(p, cache, q, k_new, v_new, positions, rows, slots, table, out, ws, stream=None):
    """prefill_paged over a coded cache (bf16)."""
    n = _tokens(q)
    _check_coded(p, cache, ws, n, ("q", "out"), dict(positions=positions, rows=rows, slots=slots), table, q=q,
                 k_new=k_new, v_new=v_new, out=out)
    _check(lib.pdattn_coded_prefill(p, cache, n, q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
                                    positions.data_ptr(), rows.data_ptr(), slots.data_ptr(), table.data_ptr(),
                                    out.data_ptr(), ws.data_ptr(), ws.nbytes, _raw_stream(stream)))


def new_status(device="cuda"):
    """A workspace of the status word alone, for calls that use no more (rotary_apply, coded_write, coded_read)."""
    return torch.zeros(STATUS_BYTES, dtype=torch.uint8, device=device)


def _check_ws(ws):
    """A contiguous workspace tensor on the current device."""
    if not isinstance(ws, torch.Tensor):
        raise TypeError("workspace must be a torch tensor")
    _ws(ws)
    _same_device(ws)


def _check_all(here, ws, specs):
    """(name, tensor, shape, dtype) of every argument and the workspace, on device `here`: one pass over each tensor's
    attributes (0.5 us), and _expect to name what is wrong."""
    for name, t, shape, dtype in specs:
        if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == here >= 0
                and t.is_contiguous()):
            _expect(name, t, shape, dtype)
            _same_device(t)
    if not (isinstance(ws, torch.Tensor) and ws.get_device() == here and ws.is_contiguous()):
        _check_ws(ws)


def make_rotary(head_dim, theta, rot_dim=None, interleaved=False, scaling="none", factor=1.0, low=1.0, high=1.0,
                original_len=0, whole_pairs=False, gain=0.0):
    """Rotary frequencies (host only): pairs over the first rot_dim dimensions (all by default), halves apart or
    interleaved, scaled for long contexts ("none", "linear", "wavelength" or "ramp")."""
    if scaling not in SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(SCALINGS)}")
    spec = RotarySpec(head_dim, head_dim if rot_dim is None else rot_dim, int(bool(interleaved)), SCALINGS[scaling],
                      int(original_len), int(bool(whole_pairs)), theta, factor, low, high, gain)
    r = Rotary()
    _check(lib.pdattn_rotary_make(spec, r))
    return r


def _check_rotary(rotary):
    if not isinstance(rotary, Rotary):
        raise TypeError("rotary must come from make_rotary")


def rotary_tables(rotary, length, dtype, device="cuda", stream=None):
    """cos and sin [length, head_dim] for make_params: half pairs over the whole head."""
    _check_rotary(rotary)
    cos = torch.empty((length, rotary.head_dim), dtype=dtype, device=device)
    sin = torch.empty((length, rotary.head_dim), dtype=dtype, device=device)
    here = _here()
    if cos.get_device() != here:
        _same_device(cos)
    _check(lib.pdattn_rotary_tables(rotary, length, _DTYPES[dtype], cos.data_ptr(), sin.data_ptr(), _stream_of(stream, here)))
    return cos, sin


def _heads_of(name, t, n, D, dtype, here):
    """(heads, token stride) of t [n, heads, D], its heads contiguous within a token."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    shape, device = t.shape, t.get_device()
    if t.dtype is not dtype or len(shape) != 3 or shape[0] != n or shape[2] != D or device < 0:
        raise ValueError(f"{name} must be a CUDA tensor [{n}, heads, {D}] of {dtype}, got {tuple(shape)} of {t.dtype}")
    if device != here:
        _same_device(t)
    h, (token, head, one) = shape[1], t.stride()
    if n and h and (one != 1 or (h > 1 and head != D)):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    return h, (token if n > 1 else h * D)


def rotary_apply(rotary, q, k, positions, q_out, k_out, ws, inverse=False, stream=None):
    """q [n, heads, D] and k [n, kv_heads, D] (or None, with k_out None) turned at positions [n] int32, or with
    inverse turned back (the gradient).  Tokens may be strided; q_out may be q and k_out k."""
    _check_rotary(rotary)
    if not isinstance(q, torch.Tensor) or q.dtype not in _DTYPES or q.dim() != 3:
        raise ValueError("q must be a bf16 or f32 tensor [n, heads, D]")
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out must be both given or both None")
    n, D, dt, here = q.shape[0], rotary.head_dim, q.dtype, _here()
    hq, sq = _heads_of("q", q, n, D, dt, here)
    ho, so = _heads_of("q_out", q_out, n, D, dt, here)
    hk = sk = hl = sl = kp = kop = 0
    if k is not None:
        hk, sk = _heads_of("k", k, n, D, dt, here)
        hl, sl = _heads_of("k_out", k_out, n, D, dt, here)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    if ho != hq or hl != hk:
        raise ValueError("q_out and k_out must have the heads of q and k")
    _check_all(here, ws, (("positions", positions, (n,), torch.int32),))
    _check(lib.pdattn_rotary_apply(rotary, n, _DTYPES[dt], 1 if inverse else 0, hq, q.data_ptr(), sq, q_out.data_ptr(), so,
                                   hk, kp, sk, kop, sl, positions.data_ptr(), ws.data_ptr(), ws.nbytes,
                                   _stream_of(stream, here)))


def shared_workspace_size(p, n_groups):
    n = lib.pdattn_shared_workspace_size(ctypes.byref(p), n_groups)
    if n == 0:
        raise PdattnError(EINVAL, lib.pdattn_last_error().decode() or "invalid parameters")
    return n


def new_shared_workspace(p, n_groups, device="cuda"):
    """A workspace for decode_shared of p.rows rows in up to n_groups groups."""
    return torch.zeros(shared_workspace_size(p, n_groups), dtype=torch.uint8, device=device)


def decode_shared(p, q, k_new, v_new, positions, table, group_start, group_pages, k_pool, v_pool, out, ws, stream=None):
    """decode_fused (bf16) where rows [group_start[i], group_start[i + 1]) hold the same first group_pages[i] pages,
    which are read once for the group; group_start [n + 1] and group_pages [n] int32."""
    n, here, T, i32 = _tokens(group_pages), _here(), torch.bfloat16, torch.int32
    if p.dtype != BF16:
        raise PdattnError(EUNSUPPORTED, "shared pages are attended on the tensor cores: dtype must be bf16")
    if getattr(p, "_device", None) not in (None, here):
        raise ValueError(f"rope tables or sinks are on cuda:{p._device}, the current device is cuda:{here}")
    R, D = p.rows, p.head_dim
    qs, kv, pool = (R, p.heads, D), (R, p.kv_heads, D), (p.num_pages, p.kv_heads, 64, D)
    _check_all(here, ws, (("q", q, qs, T), ("k_new", k_new, kv, T), ("v_new", v_new, kv, T), ("out", out, qs, T),
                          ("positions", positions, (R,), i32), ("table", table, (R, p.pages_per_row), i32),
                          ("k_pool", k_pool, pool, T), ("v_pool", v_pool, pool, T),
                          ("group_pages", group_pages, (n,), i32), ("group_start", group_start, (n + 1,), i32)))
    _check(lib.pdattn_decode_shared(p, n, group_start.data_ptr(), group_pages.data_ptr(), q.data_ptr(), k_new.data_ptr(),
                                    v_new.data_ptr(), positions.data_ptr(), table.data_ptr(), k_pool.data_ptr(),
                                    v_pool.data_ptr(), out.data_ptr(), ws.data_ptr(), ws.nbytes, _stream_of(stream, here)))


class Pages:
    """The pools of a cache that share one page table, as pages_update and pages_compact take them."""

    def __init__(self, pools, num_pages):
        self.tensors, self.num_pages, self.device = tuple(pools), num_pages, pools[0].get_device()
        self.n = len(self.tensors)
        self.array = (Pool * self.n)()
        for i, t in enumerate(self.tensors):
            self.array[i] = Pool(t.data_ptr(), t.shape[1], t.element_size() * (t.shape[3] if t.dim() == 4 else 1))


def make_pages(p, pools):
    """Pools [num_pages, heads, 64, D] of any type (keys, values, codes) and [num_pages, heads, 64] (scales), of every
    layer that shares p's table; keeps the tensors alive."""
    pools = list(pools)
    if not pools:
        raise ValueError("at least one pool is needed")
    for i, t in enumerate(pools):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"pool {i} must be a torch tensor")
        if not t.is_cuda or not t.is_contiguous() or t.dim() not in (3, 4) or t.shape[0] != p.num_pages or t.shape[2] != 64:
            raise ValueError(f"pool {i} must be a contiguous CUDA tensor [{p.num_pages}, heads, 64(, D)], "
                             f"got {tuple(t.shape)}")
    _same_device(*pools)
    spans = sorted((t.data_ptr(), t.data_ptr() + t.nbytes) for t in pools)
    if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
        raise ValueError("the pools overlap")
    return Pages(pools, p.num_pages)


def pages_workspace_size(p):
    n = lib.pdattn_pages_workspace_size(ctypes.byref(p))
    if n == 0:
        raise PdattnError(EINVAL, lib.pdattn_last_error().decode() or "invalid parameters")
    return n


def new_pages_workspace(p, device="cuda"):
    return torch.zeros(pages_workspace_size(p), dtype=torch.uint8, device=device)


def _check_pages(p, pages, here):
    if not isinstance(pages, Pages):
        raise TypeError("pages must come from make_pages")
    if pages.num_pages != p.num_pages:
        raise ValueError(f"the pools have {pages.num_pages} pages, the parameters {p.num_pages}")
    if pages.device != here:
        _same_device(pages.tensors[0])


def pages_update(p, pages, table, lengths, refs, parents, new_lengths, ws, table_out=None, refs_out=None, stream=None):
    """Row r continues row parents[r] (-1: nothing) with room for new_lengths[r] positions; see pdattn_pages_update.
    table and refs are updated in place, or written to table_out and refs_out."""
    here, i32 = _here(), torch.int32
    _check_pages(p, pages, here)
    table_out, refs_out = table if table_out is None else table_out, refs if refs_out is None else refs_out
    tab, row, num = (p.rows, p.pages_per_row), (p.rows,), (p.num_pages,)
    _check_all(here, ws, (("table", table, tab, i32), ("lengths", lengths, row, i32), ("refs", refs, num, i32),
                          ("parents", parents, row, i32), ("new_lengths", new_lengths, row, i32),
                          ("table_out", table_out, tab, i32), ("refs_out", refs_out, num, i32)))
    _check(lib.pdattn_pages_update(p, pages.n, pages.array, table.data_ptr(), lengths.data_ptr(), refs.data_ptr(),
                                   parents.data_ptr(), new_lengths.data_ptr(), table_out.data_ptr(),
                                   refs_out.data_ptr(), ws.data_ptr(), ws.nbytes, _stream_of(stream, here)))


def pages_compact(p, pages, table, lengths, refs, page_map, ws, table_out=None, refs_out=None, stream=None):
    """Moves the pages in use to the lowest ids; page_map [num_pages] gets every page's new id or -1."""
    here, i32 = _here(), torch.int32
    _check_pages(p, pages, here)
    table_out, refs_out = table if table_out is None else table_out, refs if refs_out is None else refs_out
    tab, num = (p.rows, p.pages_per_row), (p.num_pages,)
    _check_all(here, ws, (("table", table, tab, i32), ("lengths", lengths, (p.rows,), i32), ("refs", refs, num, i32),
                          ("page_map", page_map, num, i32), ("table_out", table_out, tab, i32),
                          ("refs_out", refs_out, num, i32)))
    _check(lib.pdattn_pages_compact(p, pages.n, pages.array, table.data_ptr(), lengths.data_ptr(), refs.data_ptr(),
                                    table_out.data_ptr(), refs_out.data_ptr(), page_map.data_ptr(), ws.data_ptr(),
                                    ws.nbytes, _stream_of(stream, here)))


def check_status(ws, stream=None):
    """Synchronise, read and clear the device status; raise on a recorded error."""
    _check(lib.pdattn_check_status(_ptr(ws), _stream(stream)))


def last_launch_count():
    return int(lib.pdattn_last_launch_count())
