"""ctypes binding of libifq (include/ifq.h): argument marshalling only.

Each function takes torch tensors that already live on the GPU, passes their
device pointers and sizes to the C ABI function of the same name, and raises
IfqError on a non-OK status.  No arithmetic of the method happens here, and
there is no fallback: if libifq.so is missing, loading fails loudly.
"""
import ctypes
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libifq.so")

IFQ_MAX_STAGES = 8
IFQ_MAX_GEMV_BATCH = 16
IFQ_MAX_GROUP = 32
IFQ_QUANT_STATIC_SCRATCH_BYTES = 2 << 20
IFQ_DEV_NONFINITE = 0x1
IFQ_DEV_TIMEOUT = 0x2
IFQ_DEV_RANGE = 0x4
IFQ_KV4_MAX_NEW = 16
IFQ_KV4_MAX_APPEND = 1048544

EXPORTED = (
    "ifq_status_string",
    "ifq_widely_linear_from_real",
    "ifq_quantize_workspace_bytes",
    "ifq_quantize_pack",
    "ifq_quantize_pack_static",
    "ifq_quantize_stage",
    "ifq_quantize_finish",
    "ifq_widely_linear_quantize_workspace_bytes",
    "ifq_widely_linear_quantize_pack",
    "ifq_dequantize",
    "ifq_gemv_workspace_bytes",
    "ifq_gemv",
    "ifq_gemv_plan_bytes",
    "ifq_gemv_prepare",
    "ifq_gemv_run",
    "ifq_gemm",
    "ifq_gemm_wait_limit",
    "ifq_w4_quantize",
    "ifq_w4_dequantize",
    "ifq_w4_gemv",
    "ifq_kv4_append",
    "ifq_kv4_read",
    "ifq_kv4_attention_workspace_bytes",
    "ifq_kv4_attention",
)

STATUS_NAMES = {
    0: "IFQ_OK", 1: "IFQ_ERR_NULL", 2: "IFQ_ERR_SHAPE", 3: "IFQ_ERR_ALIGN", 4: "IFQ_ERR_STAGES",
    5: "IFQ_ERR_BATCH", 6: "IFQ_ERR_WORKSPACE", 7: "IFQ_ERR_CUDA", 8: "IFQ_ERR_UNSUPPORTED", 9: "IFQ_ERR_COUNT",
    10: "IFQ_ERR_STATIC_LIMIT",
}


class IfqError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class QTensor(ctypes.Structure):
    _fields_ = [("w_re", ctypes.c_void_p), ("w_im", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class QPartials(ctypes.Structure):
    _fields_ = [("partials", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("scales", ctypes.c_void_p)]


class DqTensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64), ("w_re", ctypes.c_void_p), ("w_im", ctypes.c_void_p)]


class WlLayer(ctypes.Structure):
    _fields_ = [("R", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("U_re", ctypes.c_void_p), ("U_im", ctypes.c_void_p), ("W_re", ctypes.c_void_p),
                ("W_im", ctypes.c_void_p), ("codes_u", ctypes.c_void_p), ("scales_u", ctypes.c_void_p),
                ("codes_w", ctypes.c_void_p), ("scales_w", ctypes.c_void_p)]


class Layer(ctypes.Structure):
    _fields_ = [("codes_u", ctypes.c_void_p), ("scales_u", ctypes.c_void_p), ("codes_w", ctypes.c_void_p),
                ("scales_w", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("x_re", ctypes.c_void_p), ("x_im", ctypes.c_void_p), ("y_re", ctypes.c_void_p),
                ("y_im", ctypes.c_void_p), ("rot_re", ctypes.c_void_p), ("rot_im", ctypes.c_void_p)]


class W4Tensor(ctypes.Structure):
    _fields_ = [("R", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class W4DqTensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("w", ctypes.c_void_p)]


class W4Layer(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("x_re", ctypes.c_void_p), ("x_im", ctypes.c_void_p),
                ("y_re", ctypes.c_void_p), ("y_im", ctypes.c_void_p)]


class Kv4CacheDesc(ctypes.Structure):
    _fields_ = [("records", ctypes.c_void_p), ("pages", ctypes.c_int64), ("page_tokens", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("dim", ctypes.c_int32), ("B", ctypes.c_int32),
                ("n_new", ctypes.c_int32), ("rows", ctypes.c_int64), ("page_table", ctypes.c_void_p),
                ("table_cols", ctypes.c_int64), ("kv_lens", ctypes.c_void_p), ("new_offsets", ctypes.c_void_p)]


_lib = None


def load():
    """Load libifq.so (built in-tree); raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with python -m bit_complex_quantized_b200.build")
    lib = ctypes.CDLL(LIB_PATH)
    i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    lib.ifq_status_string.restype = ctypes.c_char_p
    lib.ifq_status_string.argtypes = [i32]
    lib.ifq_widely_linear_from_real.restype = i32
    lib.ifq_widely_linear_from_real.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp]
    lib.ifq_quantize_workspace_bytes.restype = sz
    lib.ifq_quantize_workspace_bytes.argtypes = [ctypes.POINTER(QTensor), i32, i32]
    lib.ifq_quantize_pack.restype = i32
    lib.ifq_quantize_pack.argtypes = [ctypes.POINTER(QTensor), i32, i32, vp, sz, vp, vp]
    lib.ifq_quantize_pack_static.restype = i32
    lib.ifq_quantize_pack_static.argtypes = [ctypes.POINTER(QTensor), i32, i32, vp, vp]
    lib.ifq_quantize_stage.restype = i32
    lib.ifq_quantize_stage.argtypes = [ctypes.POINTER(QTensor), i32, i32, vp, sz, vp, vp]
    lib.ifq_quantize_finish.restype = i32
    lib.ifq_quantize_finish.argtypes = [ctypes.POINTER(QPartials), i32, i32, vp]
    lib.ifq_widely_linear_quantize_workspace_bytes.restype = sz
    lib.ifq_widely_linear_quantize_workspace_bytes.argtypes = [ctypes.POINTER(WlLayer), i32, i32]
    lib.ifq_widely_linear_quantize_pack.restype = i32
    lib.ifq_widely_linear_quantize_pack.argtypes = [ctypes.POINTER(WlLayer), i32, i32, vp, sz, vp, vp]
    lib.ifq_dequantize.restype = i32
    lib.ifq_dequantize.argtypes = [ctypes.POINTER(DqTensor), i32, i32, vp]
    lib.ifq_gemv_workspace_bytes.restype = sz
    lib.ifq_gemv_workspace_bytes.argtypes = [ctypes.POINTER(Layer), i32, i32, i32]
    lib.ifq_gemv.restype = i32
    lib.ifq_gemv.argtypes = [ctypes.POINTER(Layer), i32, i32, i32, vp, sz, vp, vp]
    lib.ifq_gemv_plan_bytes.restype = sz
    lib.ifq_gemv_plan_bytes.argtypes = []
    lib.ifq_gemv_prepare.restype = i32
    lib.ifq_gemv_prepare.argtypes = [ctypes.POINTER(Layer), i32, i32, i32, vp, sz, vp, vp, sz]
    lib.ifq_gemv_run.restype = i32
    lib.ifq_gemv_run.argtypes = [vp, vp]
    lib.ifq_gemm.restype = i32
    lib.ifq_gemm.argtypes = [ctypes.POINTER(Layer), i32, i32, i64, vp, vp]
    lib.ifq_gemm_wait_limit.restype = i32
    lib.ifq_gemm_wait_limit.argtypes = [ctypes.POINTER(Layer), i32, i32, i64, ctypes.c_uint64, vp, vp]
    lib.ifq_w4_quantize.restype = i32
    lib.ifq_w4_quantize.argtypes = [vp, i32, i32, vp, vp]
    lib.ifq_w4_dequantize.restype = i32
    lib.ifq_w4_dequantize.argtypes = [vp, i32, i32, vp]
    lib.ifq_w4_gemv.restype = i32
    lib.ifq_w4_gemv.argtypes = [vp, i32, i32, i32, vp, vp]
    kvp = ctypes.POINTER(Kv4CacheDesc)
    lib.ifq_kv4_append.restype = i32
    lib.ifq_kv4_append.argtypes = [kvp, vp, vp, vp, vp, i64, vp, vp]
    lib.ifq_kv4_read.restype = i32
    lib.ifq_kv4_read.argtypes = [kvp, vp, vp, vp, vp, i64, vp, vp]
    lib.ifq_kv4_attention_workspace_bytes.restype = sz
    lib.ifq_kv4_attention_workspace_bytes.argtypes = [kvp, i32]
    lib.ifq_kv4_attention.restype = i32
    lib.ifq_kv4_attention.argtypes = [kvp, i32, vp, vp, i64, ctypes.c_float, vp, vp, i64, vp, sz, vp, vp]
    _lib = lib
    return lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status):
    if status != 0:
        raise IfqError(status, load().ifq_status_string(status).decode())


def ifq_status_string(status):
    return load().ifq_status_string(int(status)).decode()


def ifq_widely_linear_from_real(R, U_re, U_im, W_re, W_im, stream=None):
    """R: float32 [2n][2m]; outputs float32 [n][m] (all on the device)."""
    rows, cols = R.shape
    _check(load().ifq_widely_linear_from_real(_ptr(R), rows, cols, _ptr(U_re), _ptr(U_im), _ptr(W_re), _ptr(W_im),
                                              _stream(stream)))


def _qtensors(tensors):
    arr = (QTensor * len(tensors))()
    for i, t in enumerate(tensors):
        w_re, w_im, codes, scales = t
        arr[i] = QTensor(w_re.data_ptr(), w_im.data_ptr(), w_re.shape[0], w_re.shape[1], codes.data_ptr(),
                         scales.data_ptr())
    return arr


def ifq_quantize_workspace_bytes(tensors, T):
    """tensors: list of (w_re, w_im, codes, scales)."""
    return int(load().ifq_quantize_workspace_bytes(_qtensors(tensors), len(tensors), T))


def ifq_quantize_pack(tensors, T, workspace, dev_status=None, stream=None, workspace_bytes=None):
    """tensors: list of (w_re [N][K] f32, w_im, codes u8 [T][N][K/4], scales f32 [T][2])."""
    arr = _qtensors(tensors)
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(load().ifq_quantize_pack(arr, len(tensors), T, _ptr(workspace), nbytes, _ptr(dev_status),
                                    _stream(stream)))


def ifq_quantize_pack_static(tensors, T, dev_status=None, stream=None):
    """As ifq_quantize_pack, with the library's fixed device scratch instead of a workspace."""
    arr = _qtensors(tensors)
    _check(load().ifq_quantize_pack_static(arr, len(tensors), T, _ptr(dev_status), _stream(stream)))


def ifq_quantize_stage(tensors, t, partials, dev_status=None, stream=None):
    """Stage t (1-based) of a row shard: codes of the shard and its tile partials in `partials`
    (a device buffer of ifq_quantize_workspace_bytes(tensors, t) bytes)."""
    arr = _qtensors(tensors)
    _check(load().ifq_quantize_stage(arr, len(tensors), t, _ptr(partials),
                                     partials.numel() * partials.element_size(), _ptr(dev_status), _stream(stream)))


def ifq_quantize_finish(parts, t, stream=None):
    """parts: list of (gathered partials of a whole tensor, N, K, scales [T][2]); writes stage t's scales."""
    arr = (QPartials * len(parts))()
    for i, (pt, N, K, sc) in enumerate(parts):
        arr[i] = QPartials(pt.data_ptr(), N, K, sc.data_ptr())
    _check(load().ifq_quantize_finish(arr, len(parts), t, _stream(stream)))


def ifq_dequantize(tensors, T, stream=None):
    """tensors: list of (codes u8 [T][N][K/4], scales f32 [T][2], w_re, w_im) with w_* bf16 [N][K]
    (written): the dequantized weights sum_t (s_re,t Re b_t + i s_im,t Im b_t)."""
    arr = (DqTensor * len(tensors))()
    for i, (codes, scales, w_re, w_im) in enumerate(tensors):
        arr[i] = DqTensor(codes.data_ptr(), scales.data_ptr(), w_re.shape[0], w_re.shape[1], w_re.data_ptr(),
                          w_im.data_ptr())
    _check(load().ifq_dequantize(arr, len(tensors), T, _stream(stream)))


def _wl_layers(layers):
    arr = (WlLayer * len(layers))()
    for i, d in enumerate(layers):
        R = d["R"]
        arr[i] = WlLayer(R.data_ptr(), R.shape[0], R.shape[1], _ptr(d["U_re"]), _ptr(d["U_im"]), _ptr(d["W_re"]),
                         _ptr(d["W_im"]), _ptr(d["codes_u"]), _ptr(d["scales_u"]), _ptr(d["codes_w"]),
                         _ptr(d["scales_w"]))
    return arr


def ifq_widely_linear_quantize_workspace_bytes(layers, T):
    """layers: list of dicts with R [2n][2m] f32, U_re, U_im, W_re, W_im [n][m] f32,
    codes_u, codes_w u8 [T][n][m/4], scales_u, scales_w f32 [T][2] (all on the device)."""
    return int(load().ifq_widely_linear_quantize_workspace_bytes(_wl_layers(layers), len(layers), T))


def ifq_widely_linear_quantize_pack(layers, T, workspace, dev_status=None, stream=None, workspace_bytes=None):
    """Conversion and T-stage quantization of each layer in one call, stage 1 fused with the conversion."""
    arr = _wl_layers(layers)
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(load().ifq_widely_linear_quantize_pack(arr, len(layers), T, _ptr(workspace), nbytes, _ptr(dev_status),
                                                  _stream(stream)))


def _layers(layers):
    arr = (Layer * len(layers))()
    for i, d in enumerate(layers):
        arr[i] = Layer(d["codes_u"].data_ptr(), d["scales_u"].data_ptr(),
                       None if d.get("codes_w") is None else d["codes_w"].data_ptr(),
                       None if d.get("scales_w") is None else d["scales_w"].data_ptr(),
                       d["N"], d["K"], d["x_re"].data_ptr(), d["x_im"].data_ptr(), d["y_re"].data_ptr(),
                       d["y_im"].data_ptr(),
                       None if d.get("rot_re") is None else d["rot_re"].data_ptr(),
                       None if d.get("rot_im") is None else d["rot_im"].data_ptr())
    return arr


class LayerSet:
    """Layer descriptors marshalled once, for a caller that repeats the same grouped call
    (the tensors must stay alive and in place).  Accepted wherever a list of layer dicts is."""

    def __init__(self, layers):
        self.layers = list(layers)
        self.array = _layers(self.layers)

    def __len__(self):
        return len(self.layers)


def _as_array(layers):
    return (layers.array, len(layers)) if isinstance(layers, LayerSet) else (_layers(layers), len(layers))


def ifq_gemv_workspace_bytes(layers, T, B):
    arr, n = _as_array(layers)
    return int(load().ifq_gemv_workspace_bytes(arr, n, T, B))


def ifq_gemv(layers, T, B, workspace=None, dev_status=None, stream=None, workspace_bytes=None):
    """layers: list of dicts with codes_u, scales_u, codes_w, scales_w (or None), N, K,
    x_re, x_im (bf16 [B][K]), y_re, y_im (float32 [B][N]), and optionally rot_re, rot_im
    (float32 [B][N]: each output is multiplied by rot_re + i rot_im).  workspace: a device
    buffer of ifq_gemv_workspace_bytes() bytes (no initial contents needed)."""
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if workspace_bytes is not None:
        nbytes = workspace_bytes
    arr, n = _as_array(layers)
    _check(load().ifq_gemv(arr, n, T, B, _ptr(workspace), nbytes, _ptr(dev_status), _stream(stream)))


class GemvPlan:
    """A prepared decode call (ifq_gemv_prepare) in a 64-byte aligned host buffer; run() launches it
    (ifq_gemv_run).  The layers' tensors, the workspace and dev_status must stay alive and in place."""

    def __init__(self, layers, T, B, workspace=None, dev_status=None, workspace_bytes=None):
        lib = load()
        n = int(lib.ifq_gemv_plan_bytes())
        self._buf = ctypes.create_string_buffer(n + 64)
        addr = ctypes.addressof(self._buf)
        self.ptr = ctypes.c_void_p((addr + 63) & ~63)
        self._keep = (layers, workspace, dev_status)
        nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        if workspace_bytes is not None:
            nbytes = workspace_bytes
        arr, cnt = _as_array(layers)
        self._arr = arr
        _check(lib.ifq_gemv_prepare(arr, cnt, T, B, _ptr(workspace), nbytes, _ptr(dev_status), self.ptr, n))

    def run(self, stream=None):
        _check(load().ifq_gemv_run(self.ptr, _stream(stream)))


def ifq_gemm(layers, T, M, dev_status=None, stream=None):
    """As ifq_gemv with x [M][K] and y [M][N]."""
    arr, n = _as_array(layers)
    _check(load().ifq_gemm(arr, n, T, M, _ptr(dev_status), _stream(stream)))


def ifq_gemm_wait_limit(layers, T, M, wait_limit_ns, dev_status=None, stream=None):
    """As ifq_gemm with each pipeline wait bounded by wait_limit_ns (IFQ_DEV_TIMEOUT when one runs out)."""
    arr, n = _as_array(layers)
    _check(load().ifq_gemm_wait_limit(arr, n, T, M, int(wait_limit_ns), _ptr(dev_status), _stream(stream)))


# ------------------------------------------------------------------ 4-bit layers and cache
# A decode step makes these calls every few microseconds of GPU time, so the checks build no message and no
# object unless they fail, and descriptors are packed as 64-bit words.
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)   # bf16 values or their bit patterns
_F32 = (torch.float32,)
_U8 = (torch.uint8,)
_I32 = (torch.int32,)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _enqueue(index, stream, fn, *args):
    """fn(*args, stream) with CUDA device `index` current; stream: that device's current one by default."""
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return _enqueue(index, stream, fn, *args)
    if stream is not None:
        raw = stream.cuda_stream
    elif _current_raw_stream is not None:
        raw = _current_raw_stream(index)
    else:
        raw = torch.cuda.current_stream().cuda_stream
    status = fn(*args, raw)
    if status != 0:
        _check(status)


def _plane(t, numel, dtypes, index, what):
    """Address of a contiguous tensor of `numel` elements and one of the types on CUDA device `index`."""
    if t.numel() == numel and t.dtype in dtypes and t.is_contiguous() and t.get_device() == index >= 0:
        return t.data_ptr()
    if t.get_device() != index or index < 0:
        raise ValueError(f"{what}: all tensors of a call must be on one CUDA device, got {t.device}")
    raise ValueError(f"{what}: needs a contiguous {dtypes[0]} tensor of {numel} elements, got {t.dtype} "
                     f"{tuple(t.shape)} with strides {t.stride()}")


def _words(words):
    """An array of descriptors made of 64-bit words."""
    return struct.pack(f"{len(words)}q", *words)


def _status_ptr(t, index):
    """Address of an optional device status word."""
    if t is None:
        return None
    if t.get_device() != index or t.element_size() != 4 or t.numel() < 1:
        raise ValueError("dev_status must be a 32-bit integer tensor on the call's device")
    return t.data_ptr()


def w4_shapes(rows, cols, group):
    """Shapes of the codes (uint8) and scales (bf16) of a 4-bit [rows][cols] layer."""
    tiles = (rows + 15) // 16
    return (tiles, cols // 64, 512), (tiles, cols // group, 16)


def _w4_buffers(codes, scales, rows, cols, group, index):
    if group not in (32, 64, 128) or cols < 1 or cols % 64 or cols % group or rows < 1:
        raise ValueError(f"a [{rows}][{cols}] layer in groups of {group}: cols must be a multiple of 64 and of the "
                         "group, which is 32, 64 or 128")
    entries = (rows + 15) // 16 * 16 * cols
    return (_plane(codes, entries // 2, _U8, index, "codes"),
            _plane(scales, entries // group, _BF16, index, "scales"))


def _some(items):
    if not items:
        _check(9)  # IFQ_ERR_COUNT
    return items


def ifq_w4_quantize(tensors, group, dev_status=None, stream=None):
    """tensors: list of (R float32 [rows][cols], codes uint8, scales bf16), the last two written, of w4_shapes()."""
    index, words = _some(tensors)[0][0].get_device(), []
    for R, codes, scales in tensors:
        rows, cols = R.shape
        c, s = _w4_buffers(codes, scales, rows, cols, group, index)
        words += (_plane(R, rows * cols, _F32, index, "R"), rows, cols, c, s)
    _enqueue(index, stream, load().ifq_w4_quantize, _words(words), len(tensors), group,
             _status_ptr(dev_status, index))


def ifq_w4_dequantize(tensors, group, stream=None):
    """tensors: list of (codes, scales, w bf16 [rows][cols]), w written."""
    index, words = _some(tensors)[0][0].get_device(), []
    for codes, scales, w in tensors:
        rows, cols = w.shape
        c, s = _w4_buffers(codes, scales, rows, cols, group, index)
        words += (c, s, rows, cols, _plane(w, rows * cols, _BF16, index, "w"))
    _enqueue(index, stream, load().ifq_w4_dequantize, _words(words), len(tensors), group)


def _w4_layers(layers, group, B):
    """(device index, descriptor words) of ifq_w4_gemv's layers."""
    index, words = _some(layers)[0]["codes"].get_device(), []
    for d in layers:
        rows, cols, codes, scales = d["rows"], d["cols"], d["codes"], d["scales"]
        x_re, x_im, y_re, y_im = d["x_re"], d.get("x_im"), d["y_re"], d.get("y_im")
        c, s = _w4_buffers(codes, scales, rows, cols, group, index)
        if y_im is not None and rows % 2:
            raise ValueError("planar outputs need an even number of rows")
        xs = B * (cols if x_im is None else cols // 2)
        ys = B * (rows if y_im is None else rows // 2)
        words += (c, s, rows, cols, _plane(x_re, xs, _BF16, index, "x_re"),
                  0 if x_im is None else _plane(x_im, xs, _BF16, index, "x_im"),
                  _plane(y_re, ys, _F32, index, "y_re"), 0 if y_im is None else _plane(y_im, ys, _F32, index, "y_im"))
    return index, _words(words)


class W4LayerSet:
    """Layers of ifq_w4_gemv checked and marshalled once for B tokens, for a caller that repeats the same call (the
    tensors must stay alive and in place).  Accepted by ifq_w4_gemv in place of the list."""

    def __init__(self, layers, group, B):
        self.layers, self.group, self.B = list(layers), group, B
        self.index, self.array = _w4_layers(self.layers, group, B)


def ifq_w4_gemv(layers, group, B, dev_status=None, stream=None):
    """layers: list of dicts with codes, scales, rows, cols, x_re, x_im (bf16 [B][cols/2]; x_im None: x_re is
    [B][cols]) and y_re, y_im (float32 [B][rows/2]; y_im None: y_re is [B][rows]), or a W4LayerSet of them."""
    if isinstance(layers, W4LayerSet):
        if layers.group != group or layers.B != B:
            raise ValueError(f"the layers were marshalled for group {layers.group} and {layers.B} tokens")
        index, arr, n = layers.index, layers.array, len(layers.layers)
    else:
        (index, arr), n = _w4_layers(layers, group, B), len(layers)
    _enqueue(index, stream, load().ifq_w4_gemv, arr, n, group, B, _status_ptr(dev_status, index))


class Kv4Cache:
    """A 4-bit key/value cache and the sequences of a step (ifq_kv4_cache), marshalled once: the tensors must
    stay alive and in place; new lengths, pages and offsets are written into the same tensors.

    records      uint8 [pages][kv_heads][page_tokens/16][32 dim + 256]
    page_table   int32 [B][table_cols]
    kv_lens      int32 [B], tokens of each sequence with its new ones
    n_new        new tokens per sequence: the number of each, or the most that new_offsets gives
    new_offsets  int32 [B+1] or None
    rows         rows of the q, k, v and o buffers (default B n_new)"""

    def __init__(self, records, page_table, kv_lens, dim, n_new=1, rows=None, new_offsets=None):
        if records.dim() != 4 or records.shape[3] != 32 * dim + 256 or page_table.dim() != 2:
            raise ValueError(f"needs records [pages][kv_heads][page_tokens/16][{32 * dim + 256}] and page_table "
                             f"[B][table_cols], got {tuple(records.shape)} and {tuple(page_table.shape)}")
        if not 1 <= n_new < 1 << 31:
            _check(5)  # IFQ_ERR_BATCH
        pages, kv_heads, tiles = records.shape[:3]
        B = kv_lens.shape[0]
        self.dim, self.kv_heads, self.B, self.n_new = dim, kv_heads, B, n_new
        self.rows = B * n_new if rows is None else rows
        self._keep = (records, page_table, kv_lens, new_offsets)
        self.index = i = records.get_device()
        self.desc = Kv4CacheDesc(
            _plane(records, records.numel(), _U8, i, "records"), pages, 16 * tiles, kv_heads, dim, B, n_new,
            self.rows, _plane(page_table, B * page_table.shape[1], _I32, i, "page_table"), page_table.shape[1],
            _plane(kv_lens, B, _I32, i, "kv_lens"),
            None if new_offsets is None else _plane(new_offsets, B + 1, _I32, i, "new_offsets"))
        self._ref = ctypes.byref(self.desc)

    @staticmethod
    def records_shape(pages, kv_heads, page_tokens, dim):
        return pages, kv_heads, page_tokens // 16, 32 * dim + 256


def _row_planes(cache, planes, width, dtypes, what):
    """Addresses and the common row stride of [rows][width] planes whose rows may be slices of wider ones."""
    rows, index = cache.rows, cache.index
    numel = rows * width
    for t in planes:
        if not (t.numel() == numel and t.dtype in dtypes and t.is_contiguous() and t.get_device() == index):
            break
    else:
        return [t.data_ptr() for t in planes], width
    ld = None
    for t in planes:
        if t.dim() != 2 or t.shape[0] < rows or t.shape[1] != width or t.dtype not in dtypes or t.stride(1) != 1:
            raise ValueError(f"{what}: needs {dtypes[0]} planes [{rows}][{width}], rows contiguous; got {t.dtype} "
                             f"{tuple(t.shape)} with strides {t.stride()}")
        if t.get_device() != index:
            raise ValueError(f"{what}: on {t.device}, the cache on cuda:{index}")
        step = t.stride(0) if t.shape[0] > 1 else width   # a single row's stride says nothing
        if ld is not None and step != ld:
            raise ValueError(f"{what}: the planes' row strides differ ({ld} and {step})")
        ld = step
    return [t.data_ptr() for t in planes], ld


def ifq_kv4_append(cache, k_re, k_im, v_re, v_im, dev_status=None, stream=None):
    """Quantizes the new tokens' keys and values (float32 [rows][kv_heads dim], or column slices of wider
    buffers with one row stride) into the cache."""
    p, ld = _row_planes(cache, (k_re, k_im, v_re, v_im), cache.kv_heads * cache.dim, _F32, "k, v")
    _enqueue(cache.index, stream, load().ifq_kv4_append, cache._ref, *p, ld, _status_ptr(dev_status, cache.index))


def ifq_kv4_read(cache, k_re, k_im, v_re, v_im, dev_status=None, stream=None):
    """Writes the stored values of the new tokens (float32, laid out as for ifq_kv4_append)."""
    p, ld = _row_planes(cache, (k_re, k_im, v_re, v_im), cache.kv_heads * cache.dim, _F32, "k, v")
    _enqueue(cache.index, stream, load().ifq_kv4_read, cache._ref, *p, ld, _status_ptr(dev_status, cache.index))


def ifq_kv4_attention_workspace_bytes(cache, q_heads):
    return int(load().ifq_kv4_attention_workspace_bytes(cache._ref, q_heads))


def ifq_kv4_attention(cache, q_re, q_im, o_re, o_im, scale, workspace=None, dev_status=None, stream=None,
                      workspace_bytes=None):
    """q_re, q_im: float32 [rows][q_heads dim]; o_re, o_im: bf16, the same shape, written.  workspace: a device
    buffer of ifq_kv4_attention_workspace_bytes(cache, q_heads) bytes (no initial contents needed)."""
    width, index = q_re.shape[-1], cache.index
    if width % cache.dim:
        raise ValueError("q's row must be a whole number of heads")
    q, ldq = _row_planes(cache, (q_re, q_im), width, _F32, "q")
    o, ldo = _row_planes(cache, (o_re, o_im), width, _BF16, "o")
    nbytes, ws = 0, None
    if workspace is not None:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("the workspace must be contiguous and on the cache's device")
        nbytes, ws = workspace.numel() * workspace.element_size(), workspace.data_ptr()
    if workspace_bytes is not None:
        nbytes = workspace_bytes
    _enqueue(index, stream, load().ifq_kv4_attention, cache._ref, width // cache.dim, *q, ldq, scale, *o, ldo, ws,
             nbytes, _status_ptr(dev_status, index))


# Raw entry point for callers that build ctypes descriptors themselves.
def raw():
    return load()
