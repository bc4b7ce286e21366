"""ctypes binding of libmla_decode.so: argument marshalling only.

Every function here forwards to the C ABI in include/mla_decode.h with device
pointers taken from torch tensors and the current torch CUDA stream.  There is
no fallback: if the shared library cannot be loaded, importing the binding
raises.
"""
import ctypes
import os

import torch

from . import build as _build

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmla_decode.so")

STATUS = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "WORKSPACE_TOO_SMALL", 4: "CUDA_ERROR",
          5: "DEVICE_BOUNDS", 6: "TIMEOUT"}

ENTRY_POINTS = (
    "mla_decode_workspace_size", "mla_decode_workspace_size_ex", "mla_decode_plan",
    "mla_decode_plan_ex", "mla_decode_run", "mla_decode_absorb", "mla_decode_attend",
    "mla_decode_combine", "mla_decode_up_project", "mla_decode_check", "mla_decode_status_string",
    "mla_decode_workspace_offsets", "mla_decode_kernels_per_run",
    "mla_decode_run_static_scratch", "mla_decode_selftest_wait_timeout",
    "mla_decode_run_fp8w", "mla_decode_absorb_fp8w", "mla_decode_up_project_fp8w",
    "mla_decode_append_fp8kv", "mla_decode_plan_fp8kv", "mla_decode_run_fp8kv",
    "mla_decode_attend_fp8kv", "mla_decode_page_keys", "mla_decode_page_keys_fp8kv",
    "mla_decode_score_pages", "mla_decode_select_pages")


class Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "q_len", "num_heads", "qk_nope", "qk_rope", "kv_lora", "v_head", "page_size",
        "num_pages", "max_pages_per_seq")]


class MlaDecodeError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__("%s failed: %s (%d) %s" % (where, STATUS.get(code, "?"), code,
                                                   lib().mla_decode_status_string(code).decode()))


_lib = None


def lib():
    """Load (building first if sources are newer) the CUDA library; raises if unavailable."""
    global _lib
    if _lib is None:
        if not _build.up_to_date():
            _build.build()
        L = ctypes.CDLL(LIB_PATH)
        P, D, S = ctypes.c_void_p, ctypes.POINTER(Dims), ctypes.c_size_t
        sz = ctypes.POINTER(ctypes.c_size_t)
        i32 = ctypes.c_int32
        L.mla_decode_workspace_size.argtypes = [D, sz]
        L.mla_decode_workspace_size_ex.argtypes = [D, i32, sz]
        L.mla_decode_plan.argtypes = [D, P, P, S, P]
        L.mla_decode_plan_ex.argtypes = [D, P, i32, P, S, P]
        L.mla_decode_run.argtypes = [D, P, P, P, P, P, P, ctypes.c_float, P, P, P, S, P]
        L.mla_decode_absorb.argtypes = [D, P, P, P, S, P]
        L.mla_decode_attend.argtypes = [D, P, P, P, ctypes.c_float, P, P, S, P]
        L.mla_decode_combine.argtypes = [D, ctypes.c_float, P, P, S, P]
        L.mla_decode_up_project.argtypes = [D, P, P, P, S, P]
        L.mla_decode_check.argtypes = [P, P]
        L.mla_decode_status_string.argtypes = [ctypes.c_int]
        L.mla_decode_status_string.restype = ctypes.c_char_p
        L.mla_decode_workspace_offsets.argtypes = [D, i32, ctypes.POINTER(ctypes.c_int64), i32]
        L.mla_decode_run_static_scratch.argtypes = [D, P, P, P, P, P, P, ctypes.c_float, P, P, P]
        L.mla_decode_selftest_wait_timeout.argtypes = [P, P]
        L.mla_decode_kernels_per_run.argtypes = [D, i32, ctypes.POINTER(ctypes.c_int32)]
        L.mla_decode_run_fp8w.argtypes = [D, P, P, P, P, P, P, P, P, ctypes.c_float, P, P, P, S, P]
        L.mla_decode_absorb_fp8w.argtypes = [D, P, P, P, P, S, P]
        L.mla_decode_up_project_fp8w.argtypes = [D, P, P, P, P, S, P]
        L.mla_decode_append_fp8kv.argtypes = [D, P, i32, P, P, P, P, P, P, P]
        L.mla_decode_plan_fp8kv.argtypes = [D, P, i32, P, S, P]
        L.mla_decode_run_fp8kv.argtypes = [D, P, P, P, P, P, P, P, ctypes.c_float, P, P, P, S, P]
        L.mla_decode_attend_fp8kv.argtypes = [D, P, P, P, P, ctypes.c_float, P, P, S, P]
        L.mla_decode_page_keys.argtypes = [D, P, P, P, i32, P, P, P, P]
        L.mla_decode_page_keys_fp8kv.argtypes = [D, P, P, P, P, i32, P, P, P, P]
        L.mla_decode_score_pages.argtypes = [D, P, P, P, P, P, P, P]
        L.mla_decode_select_pages.argtypes = [D, P, P, P, i32, i32, i32, P, P, P, P, P]
        for n in ENTRY_POINTS:
            if n != "mla_decode_status_string":
                getattr(L, n).restype = ctypes.c_int
        _lib = L
    return _lib


def dims_for(q, cache, block_table) -> Dims:
    B, T, H, dq = q.shape
    return Dims(B, T, H, 128, dq - 128, cache.shape[2] - (dq - 128), 128, cache.shape[1],
                cache.shape[0], block_table.shape[1])


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _public_raw_stream(device):
    return torch.cuda.current_stream(device).cuda_stream


# The current device and its current stream's handle.  torch.cuda.current_stream()
# builds a Stream object, 2.9 us a call; these take 0.2, but are torch's own: a
# torch without them serves the same through its public calls.
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_raw_stream)


def _stream():
    return _raw_stream(_device())


def _ok(code, where):
    if code != 0:
        raise MlaDecodeError(code, where)


def workspace_size(d: Dims, num_ranges: int = 0) -> int:
    n = ctypes.c_size_t(0)
    _ok(lib().mla_decode_workspace_size_ex(ctypes.byref(d), num_ranges, ctypes.byref(n)),
        "mla_decode_workspace_size_ex")
    return n.value


def workspace_offsets(d: Dims, num_ranges: int = 0):
    arr = (ctypes.c_int64 * 4)()
    _ok(lib().mla_decode_workspace_offsets(ctypes.byref(d), num_ranges, arr, 4),
        "mla_decode_workspace_offsets")
    return dict(qlat=arr[0], qlo=arr[1], olat=arr[2], header=arr[3])


def kernels_per_run(d: Dims, fp8_weights: bool = False) -> int:
    """Kernels one whole run enqueues on the current device (plan not counted)."""
    n = ctypes.c_int32(0)
    _ok(lib().mla_decode_kernels_per_run(ctypes.byref(d), int(fp8_weights), ctypes.byref(n)),
        "mla_decode_kernels_per_run")
    return n.value


class MlaDecode:
    """Owns a device workspace for one set of dims; plan() once per decode step,
    run() or run_fp8kv() once per layer.  All tensors must be CUDA, contiguous.
    With fp8_kv plan() balances the work for the 8-bit cache (a plan of either
    kind serves both)."""

    def __init__(self, d: Dims, device=None, num_ranges: int = 0, fp8_kv: bool = False):
        self.dims = d
        self.num_ranges = num_ranges
        self.ws_bytes = workspace_size(d, num_ranges)
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8,
                                     device=device or torch.device("cuda"))
        self.fp8_kv = fp8_kv
        # What the calls over the 8-bit cache take.  (Query, out and lse by their
        # number of elements: [B, T, ...] serves a handle of B * T sequences.)
        B, pages, H = d.batch, d.num_pages, d.num_heads
        n = B * d.q_len * H
        self._attend_spec = (
            ("kv8", torch.uint8, (pages, 64, 576)), ("kv_scale", torch.float32, (pages,)),
            ("block_table", torch.int32, (B, d.max_pages_per_seq)),
            ("seq_lens", torch.int32, (B,)), ("lse", torch.float32, n))
        self._run_spec = self._attend_spec + (
            ("q", torch.bfloat16, n * 192), ("w_uk", torch.bfloat16, (H, 128, 512)),
            ("w_uv", torch.bfloat16, (H, 512, 128)), ("out", torch.bfloat16, n * 128))

    def plan(self, seq_lens):
        if self.fp8_kv:
            _ok(lib().mla_decode_plan_fp8kv(ctypes.byref(self.dims), _ptr(seq_lens),
                                            self.num_ranges, _ptr(self.workspace), self.ws_bytes,
                                            _stream()),
                "mla_decode_plan_fp8kv")
            return
        _ok(lib().mla_decode_plan_ex(ctypes.byref(self.dims), _ptr(seq_lens), self.num_ranges,
                                     _ptr(self.workspace), self.ws_bytes, _stream()),
            "mla_decode_plan_ex")

    def run(self, q, cache, block_table, seq_lens, w_uk, w_uv, scale, out, lse):
        _ok(lib().mla_decode_run(ctypes.byref(self.dims), _ptr(q), _ptr(cache), _ptr(block_table),
                                 _ptr(seq_lens), _ptr(w_uk), _ptr(w_uv), float(scale), _ptr(out),
                                 _ptr(lse), _ptr(self.workspace), self.ws_bytes, _stream()),
            "mla_decode_run")

    def run_fp8w(self, q, cache, block_table, seq_lens, w_uk8, w_uk_scale, w_uv8, w_uv_scale,
                 scale, out, lse):
        _ok(lib().mla_decode_run_fp8w(ctypes.byref(self.dims), _ptr(q), _ptr(cache),
                                      _ptr(block_table), _ptr(seq_lens), _ptr(w_uk8),
                                      _ptr(w_uk_scale), _ptr(w_uv8), _ptr(w_uv_scale),
                                      float(scale), _ptr(out), _ptr(lse), _ptr(self.workspace),
                                      self.ws_bytes, _stream()),
            "mla_decode_run_fp8w")

    def run_fp8kv(self, q, kv8, kv_scale, block_table, seq_lens, w_uk, w_uv, scale, out, lse):
        stream = _checked_as(self._run_spec, self.workspace, kv8, kv_scale, block_table, seq_lens,
                             lse, q, w_uk, w_uv, out)
        _ok(lib().mla_decode_run_fp8kv(ctypes.byref(self.dims), q.data_ptr(), kv8.data_ptr(),
                                       kv_scale.data_ptr(), block_table.data_ptr(),
                                       seq_lens.data_ptr(), w_uk.data_ptr(), w_uv.data_ptr(),
                                       float(scale), out.data_ptr(), lse.data_ptr(),
                                       self.workspace.data_ptr(), self.ws_bytes, stream),
            "mla_decode_run_fp8kv")

    def attend_fp8kv(self, kv8, kv_scale, block_table, seq_lens, scale, lse):
        stream = _checked_as(self._attend_spec, self.workspace, kv8, kv_scale, block_table,
                             seq_lens, lse)
        _ok(lib().mla_decode_attend_fp8kv(ctypes.byref(self.dims), kv8.data_ptr(),
                                          kv_scale.data_ptr(), block_table.data_ptr(),
                                          seq_lens.data_ptr(), float(scale), lse.data_ptr(),
                                          self.workspace.data_ptr(), self.ws_bytes, stream),
            "mla_decode_attend_fp8kv")

    def absorb_fp8w(self, q, w_uk8, w_uk_scale):
        _ok(lib().mla_decode_absorb_fp8w(ctypes.byref(self.dims), _ptr(q), _ptr(w_uk8),
                                         _ptr(w_uk_scale), _ptr(self.workspace), self.ws_bytes,
                                         _stream()),
            "mla_decode_absorb_fp8w")

    def up_project_fp8w(self, w_uv8, w_uv_scale, out):
        _ok(lib().mla_decode_up_project_fp8w(ctypes.byref(self.dims), _ptr(w_uv8),
                                             _ptr(w_uv_scale), _ptr(out), _ptr(self.workspace),
                                             self.ws_bytes, _stream()),
            "mla_decode_up_project_fp8w")

    def absorb(self, q, w_uk):
        _ok(lib().mla_decode_absorb(ctypes.byref(self.dims), _ptr(q), _ptr(w_uk),
                                    _ptr(self.workspace), self.ws_bytes, _stream()),
            "mla_decode_absorb")

    def attend(self, cache, block_table, seq_lens, scale, lse):
        _ok(lib().mla_decode_attend(ctypes.byref(self.dims), _ptr(cache), _ptr(block_table),
                                    _ptr(seq_lens), float(scale), _ptr(lse), _ptr(self.workspace),
                                    self.ws_bytes, _stream()),
            "mla_decode_attend")

    def combine(self, scale, lse):
        _ok(lib().mla_decode_combine(ctypes.byref(self.dims), float(scale), _ptr(lse),
                                     _ptr(self.workspace), self.ws_bytes, _stream()),
            "mla_decode_combine")

    def up_project(self, w_uv, out):
        _ok(lib().mla_decode_up_project(ctypes.byref(self.dims), _ptr(w_uv), _ptr(out),
                                        _ptr(self.workspace), self.ws_bytes, _stream()),
            "mla_decode_up_project")

    def check(self) -> int:
        """Synchronise the stream; return the device status code (0 = OK)."""
        return lib().mla_decode_check(_ptr(self.workspace), _stream())

    # -- views of intermediates (tests / profiling)
    def _view(self, key, cols, dtype=torch.bfloat16):
        off = workspace_offsets(self.dims, self.num_ranges)[key]
        rows = self.dims.batch * self.dims.q_len * self.dims.num_heads
        n = rows * cols * torch.empty(0, dtype=dtype).element_size()
        return self.workspace[off:off + n].view(dtype).view(rows, cols)

    def q_lat(self):
        return self._view("qlat", 576)

    def q_lo(self):
        """The residual q_lat - bf16(q_lat), times 2^10, as raw E4M3 bytes."""
        return self._view("qlo", 512, torch.uint8)

    def o_lat(self):
        return self._view("olat", 512)

    def plan_header(self):
        off = workspace_offsets(self.dims, self.num_ranges)["header"]
        return self.workspace[off:off + 16].view(torch.int32).tolist()


def decode(q, cache, block_table, seq_lens, w_uk, w_uv, scale, num_ranges: int = 0):
    """One-shot convenience: plan + run, returns (out bf16 [B,T,H,128], lse fp32 [B,T,H])."""
    d = dims_for(q, cache, block_table)
    m = MlaDecode(d, q.device, num_ranges)
    out = torch.empty(q.shape[0], q.shape[1], q.shape[2], 128, dtype=torch.bfloat16,
                      device=q.device)
    lse = torch.empty(q.shape[0], q.shape[1], q.shape[2], dtype=torch.float32, device=q.device)
    m.plan(seq_lens)
    m.run(q, cache, block_table, seq_lens, w_uk, w_uv, scale, out, lse)
    return out, lse


# ---------------------------------------------------------------- 8-bit cache, sparse decode
def _refuse(name, t, dtype, shape):
    got = None if t is None else (t.dtype, tuple(t.shape), t.is_contiguous(), str(t.device))
    size = "shape %s" % (shape,) if type(shape) is tuple else "%d elements" % shape
    raise ValueError("%s: expected a contiguous %s tensor of %s on the current CUDA device, "
                     "with the other tensors, got %s" % (name, dtype, size, got))


def _checked(*tensors):
    """The current stream, once every (name, tensor, dtype, shape) is what it should
    be: the C ABI sees pointers only.  (One loop without helpers: the checks are
    most of a small call's time on the host.)"""
    device = tensors[0][1].get_device() if tensors[0][1] is not None else -1
    for name, t, dtype, shape in tensors:
        if (t is None or t.dtype is not dtype or t.shape != shape or not t.is_contiguous()
                or t.get_device() != device):
            _refuse(name, t, dtype, shape)
    if device < 0 or device != _device():
        _refuse(*tensors[0])
    return _raw_stream(device)


def _checked_as(spec, workspace, *tensors):
    """The same for (name, dtype, shape or number of elements), made once, on the
    workspace's device: nine tensors in the time that four take above."""
    device = workspace.get_device()
    for t, (name, dtype, shape) in zip(tensors, spec):
        if (t is None or t.dtype is not dtype
                or (t.shape if type(shape) is tuple else t.numel()) != shape
                or not t.is_contiguous() or t.get_device() != device):
            _refuse(name, t, dtype, shape)
    if device < 0 or device != _device():
        _refuse(spec[0][0], tensors[0], *spec[0][1:])
    return _raw_stream(device)


def _lines(d, block_table, seq_lens, new_lens=None, status=None):
    B = d.batch
    lines = [("block_table", block_table, torch.int32, (B, d.max_pages_per_seq)),
             ("seq_lens", seq_lens, torch.int32, (B,))]
    if new_lens is not None:
        lines.append(("new_lens", new_lens, torch.int32, (B,)))
    if status is not None:
        lines.append(("status", status, torch.int32, (1,)))
    return lines


def append_fp8kv(d: Dims, rows, kv8, kv_scale, block_table, seq_lens, new_lens=None,
                 status=None):
    """Quantise new rows (bf16 [B, max_new, 576]) into the 8-bit cache, in place.

    Row i < new_lens[b] (default: every row) goes to position
    seq_lens[b] - new_lens[b] + i.  status: optional int32 [1] on the device
    that receives the first error found there."""
    B, pages = d.batch, d.num_pages
    max_new = rows.shape[1] if rows is not None and rows.dim() == 3 else 0
    stream = _checked(("rows", rows, torch.bfloat16, (B, max_new, 576)),
                      ("kv8", kv8, torch.uint8, (pages, 64, 576)),
                      ("kv_scale", kv_scale, torch.float32, (pages,)),
                      *_lines(d, block_table, seq_lens, new_lens, status))
    _ok(lib().mla_decode_append_fp8kv(ctypes.byref(d), rows.data_ptr(), max_new, _ptr(new_lens),
                                      block_table.data_ptr(), seq_lens.data_ptr(), kv8.data_ptr(),
                                      kv_scale.data_ptr(), _ptr(status), stream),
        "mla_decode_append_fp8kv")


def page_keys(d: Dims, cache, block_table, seq_lens, max_new, keys, new_lens=None, status=None):
    """Mean keys (bf16 [num_pages, 576], in place) of the pages that hold each
    sequence's newest new_lens[b] <= max_new tokens (default: max_new), from the
    bf16 cache."""
    pages = d.num_pages
    stream = _checked(("cache", cache, torch.bfloat16, (pages, 64, 576)),
                      ("keys", keys, torch.bfloat16, (pages, 576)),
                      *_lines(d, block_table, seq_lens, new_lens, status))
    _ok(lib().mla_decode_page_keys(ctypes.byref(d), cache.data_ptr(), block_table.data_ptr(),
                                   seq_lens.data_ptr(), max_new, _ptr(new_lens), keys.data_ptr(),
                                   _ptr(status), stream),
        "mla_decode_page_keys")


def page_keys_fp8kv(d: Dims, kv8, kv_scale, block_table, seq_lens, max_new, keys, new_lens=None,
                    status=None):
    """page_keys() from the 8-bit cache."""
    pages = d.num_pages
    stream = _checked(("kv8", kv8, torch.uint8, (pages, 64, 576)),
                      ("kv_scale", kv_scale, torch.float32, (pages,)),
                      ("keys", keys, torch.bfloat16, (pages, 576)),
                      *_lines(d, block_table, seq_lens, new_lens, status))
    _ok(lib().mla_decode_page_keys_fp8kv(ctypes.byref(d), kv8.data_ptr(), kv_scale.data_ptr(),
                                         block_table.data_ptr(), seq_lens.data_ptr(), max_new,
                                         _ptr(new_lens), keys.data_ptr(), _ptr(status), stream),
        "mla_decode_page_keys_fp8kv")


def score_pages(d: Dims, query, keys, block_table, seq_lens, scores, status=None):
    """scores (fp32 [B, T, max_pages_per_seq], written): each query token's
    largest head product (query: bf16 [B, T, H, 576]) with every page's key."""
    B, T = d.batch, d.q_len
    stream = _checked(("query", query, torch.bfloat16, (B, T, d.num_heads, 576)),
                      ("keys", keys, torch.bfloat16, (d.num_pages, 576)),
                      ("scores", scores, torch.float32, (B, T, d.max_pages_per_seq)),
                      *_lines(d, block_table, seq_lens, None, status))
    _ok(lib().mla_decode_score_pages(ctypes.byref(d), query.data_ptr(), keys.data_ptr(),
                                     block_table.data_ptr(), seq_lens.data_ptr(),
                                     scores.data_ptr(), _ptr(status), stream),
        "mla_decode_score_pages")


def select_pages(d: Dims, scores, block_table, seq_lens, top_k, keep_first, keep_last, sel_table,
                 sel_lens, sel_pages=None, status=None):
    """The top_k pages of every query token, as a block table (int32 [B * T, top_k])
    and lengths (int32 [B * T]) to decode on with one query token per line."""
    lines = d.batch * d.q_len
    tensors = [("scores", scores, torch.float32, (d.batch, d.q_len, d.max_pages_per_seq)),
               ("sel_table", sel_table, torch.int32, (lines, top_k)),
               ("sel_lens", sel_lens, torch.int32, (lines,))]
    if sel_pages is not None:
        tensors.append(("sel_pages", sel_pages, torch.int32, (lines, top_k)))
    stream = _checked(*tensors, *_lines(d, block_table, seq_lens, None, status))
    _ok(lib().mla_decode_select_pages(ctypes.byref(d), scores.data_ptr(), block_table.data_ptr(),
                                      seq_lens.data_ptr(), top_k, keep_first, keep_last,
                                      sel_table.data_ptr(), _ptr(sel_pages), sel_lens.data_ptr(),
                                      _ptr(status), stream),
        "mla_decode_select_pages")
