"""PyTorch-facing binding of libw4a16: one function per C entry point, same names.

Argument marshalling only: shapes, dtypes and devices are checked, outputs are allocated with
torch when the caller does not pass them, and the C function runs on the current (or given)
CUDA stream.  Every step of the computation happens in the library's kernels.

Tensor conventions: bf16 values travel as ``torch.bfloat16`` tensors, packed int4 words as
``torch.int32`` tensors holding the uint32 bit patterns (layout L1, see include/w4a16.h).
"""
from __future__ import annotations

import ctypes as C
import functools

import torch

from . import _lib

W4_EPI_NONE = _lib.W4_EPI_NONE
W4_EPI_GELU_GATE = _lib.W4_EPI_GELU_GATE


def _p(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _s(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _need(name, t, dtype, shape=None, dev=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name}: expected device {dev}, got {t.device}")


_WS: dict = {}


def workspace(nbytes: int, device, stream=None) -> torch.Tensor | None:
    """A scratch buffer of at least nbytes for calls on (device, stream).

    One buffer per stream: calls on one stream run in order, so they may share it (the library
    clears what it relies on, so contents left by earlier calls do not matter), while calls on
    different streams never do.  A buffer that is outgrown is kept alive, not freed, so a CUDA
    graph captured with it stays valid; a capture on its own stream gets its own buffer.
    """
    if nbytes == 0:
        return None
    dev = torch.device(device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    key = (dev, s.cuda_stream)
    bufs = _WS.setdefault(key, [])
    if not bufs or bufs[-1].numel() < nbytes:
        bufs.append(torch.zeros((nbytes + 255) // 256 * 256, dtype=torch.uint8, device=dev))
    return bufs[-1]


def w4_workspace_bytes(op: int, m_or_t: int, n: int, k_dim: int, e: int, k: int) -> int:
    return int(_lib.load().w4_workspace_bytes(op, m_or_t, n, k_dim, e, k))


def w4_repack(w, codes=None, scales=None, group_m=None, off_grid_count=None, stream=None):
    """bf16 weights [rows, K] -> (codes int32 [rows, K/8], scales bf16 [rows, K/32],
    group_m uint8 [rows, K/32], off_grid_count int64 [1])."""
    lib = _lib.load()
    rows, K = w.shape
    _need("w", w, torch.bfloat16)
    dev = w.device
    codes = torch.empty((rows, K // 8), dtype=torch.int32, device=dev) if codes is None else codes
    scales = torch.empty((rows, K // 32), dtype=torch.bfloat16, device=dev) if scales is None else scales
    group_m = torch.empty((rows, K // 32), dtype=torch.uint8, device=dev) if group_m is None else group_m
    if off_grid_count is None:
        off_grid_count = torch.empty(1, dtype=torch.int64, device=dev)
    _need("codes", codes, torch.int32, (rows, K // 8), dev)
    _need("scales", scales, torch.bfloat16, (rows, K // 32), dev)
    _need("group_m", group_m, torch.uint8, (rows, K // 32), dev)
    _need("off_grid_count", off_grid_count, torch.int64, (1,), dev)
    _lib.check("w4_repack", lib.w4_repack(_p(w), rows, K, _p(codes), _p(scales), _p(group_m),
                                          _p(off_grid_count), _s(stream)))
    return codes, scales, group_m, off_grid_count


def w4a16_linear(x, codes, scales, y=None, ws=None, stream=None):
    """y [M, N] = x [M, K] @ dequant(codes, scales)^T, bf16 out."""
    lib = _lib.load()
    M, K = x.shape
    N = codes.shape[0]
    dev = x.device
    _need("x", x, torch.bfloat16)
    _need("codes", codes, torch.int32, (N, K // 8), dev)
    _need("scales", scales, torch.bfloat16, (N, K // 32), dev)
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    _need("y", y, torch.bfloat16, (M, N), dev)
    nbytes = w4_workspace_bytes(_lib.W4_OP_LINEAR, M, N, K, 1, 1)
    if ws is None:
        ws = workspace(nbytes, dev, stream)
    _lib.check("w4a16_linear", lib.w4a16_linear(_p(x), _p(codes), _p(scales), _p(y), M, N, K,
                                                _p(ws), 0 if ws is None else ws.numel(), _s(stream)))
    return y


def w4a16_linear_g(x, codes, scales, group: int, zeros=None, y=None, ws=None, stream=None):
    """The linear on the weight-format variants: scales [N, K/group] bf16, zeros [N, K/group]
    uint8 zero-points (or None: z = 8); W = s * (u - z)."""
    lib = _lib.load()
    M, K = x.shape
    N = codes.shape[0]
    dev = x.device
    _need("x", x, torch.bfloat16)
    _need("codes", codes, torch.int32, (N, K // 8), dev)
    _need("scales", scales, torch.bfloat16, (N, K // group), dev)
    if zeros is not None:
        _need("zeros", zeros, torch.uint8, (N, K // group), dev)
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    _need("y", y, torch.bfloat16, (M, N), dev)
    if ws is None:
        ws = workspace(w4_workspace_bytes(_lib.W4_OP_LINEAR_G, M, N, K, 1, 1), dev, stream)
    _lib.check("w4a16_linear_g", lib.w4a16_linear_g(_p(x), _p(codes), _p(scales), _p(zeros), group, _p(y),
                                                    M, N, K, _p(ws), 0 if ws is None else ws.numel(),
                                                    _s(stream)))
    return y


NOALLOC_SCRATCH_BYTES = 8 << 20


def w4a16_linear_noalloc(x, codes, scales, y=None, stream=None):
    """Like w4a16_linear, but never needs a workspace: split-K scratch comes from the library's
    fixed 8 MiB device array (for callers that cannot allocate device memory).  Calls that
    overlap on the GPU share that array and must be ordered by the caller."""
    lib = _lib.load()
    M, K = x.shape
    N = codes.shape[0]
    dev = x.device
    _need("x", x, torch.bfloat16)
    _need("codes", codes, torch.int32, (N, K // 8), dev)
    _need("scales", scales, torch.bfloat16, (N, K // 32), dev)
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    _need("y", y, torch.bfloat16, (M, N), dev)
    _lib.check("w4a16_linear_noalloc", lib.w4a16_linear_noalloc(_p(x), _p(codes), _p(scales), _p(y),
                                                                M, N, K, _s(stream)))
    return y


class Routing:
    __slots__ = ("topk_ids", "topk_w", "expert_offsets", "sorted_pair", "pair_pos")

    def __init__(self, topk_ids, topk_w, expert_offsets, sorted_pair, pair_pos):
        self.topk_ids = topk_ids
        self.topk_w = topk_w
        self.expert_offsets = expert_offsets
        self.sorted_pair = sorted_pair
        self.pair_pos = pair_pos


def moe_route_permute(logits, k: int, out: Routing | None = None, ws=None, stream=None) -> Routing:
    """Top-k routing of float32 logits [T, E] and the expert-major permutation."""
    lib = _lib.load()
    T, E = logits.shape
    dev = logits.device
    _need("logits", logits, torch.float32)
    if out is None:
        out = Routing(torch.empty((T, k), dtype=torch.int32, device=dev),
                      torch.empty((T, k), dtype=torch.float32, device=dev),
                      torch.empty(E + 1, dtype=torch.int32, device=dev),
                      torch.empty(T * k, dtype=torch.int32, device=dev),
                      torch.empty(T * k, dtype=torch.int32, device=dev))
    _need("topk_ids", out.topk_ids, torch.int32, (T, k), dev)
    _need("topk_w", out.topk_w, torch.float32, (T, k), dev)
    _need("expert_offsets", out.expert_offsets, torch.int32, (E + 1,), dev)
    _need("sorted_pair", out.sorted_pair, torch.int32, (T * k,), dev)
    _need("pair_pos", out.pair_pos, torch.int32, (T * k,), dev)
    nbytes = w4_workspace_bytes(_lib.W4_OP_ROUTE, T, 0, 0, E, k)
    if ws is None:
        ws = workspace(nbytes, dev, stream)
    _lib.check("moe_route_permute", lib.moe_route_permute(
        _p(logits), T, E, k, _p(out.topk_ids), _p(out.topk_w), _p(out.expert_offsets),
        _p(out.sorted_pair), _p(out.pair_pos), _p(ws), 0 if ws is None else ws.numel(), _s(stream)))
    return out


def moe_w4a16_gmm(a, a_row_of_pair, k: int, codes, scales, expert_offsets, rows: int,
                  epilogue: int = W4_EPI_NONE, out=None, ws=None, dev_status=None, stream=None):
    """Grouped W4A16 GEMM: codes [E, N, K/8], scales [E, N, K/32]; out [rows, N or N/2] bf16."""
    lib = _lib.load()
    E, N, Kw = codes.shape
    K = Kw * 8
    dev = a.device
    _need("a", a, torch.bfloat16)
    if a.shape[1] != K:
        raise ValueError("a: wrong number of columns")
    if a_row_of_pair is not None:
        _need("a_row_of_pair", a_row_of_pair, torch.int32, (rows,), dev)
    _need("codes", codes, torch.int32, (E, N, K // 8), dev)
    _need("scales", scales, torch.bfloat16, (E, N, K // 32), dev)
    _need("expert_offsets", expert_offsets, torch.int32, (E + 1,), dev)
    n_out = N // 2 if epilogue == W4_EPI_GELU_GATE else N
    out = torch.empty((rows, n_out), dtype=torch.bfloat16, device=dev) if out is None else out
    _need("out", out, torch.bfloat16, (rows, n_out), dev)
    nbytes = w4_workspace_bytes(_lib.W4_OP_GMM, rows, N, K, E, k)
    if ws is None:
        ws = workspace(nbytes, dev, stream)
    if dev_status is not None:
        _need("dev_status", dev_status, torch.int32, (1,), dev)
    _lib.check("moe_w4a16_gmm", lib.moe_w4a16_gmm(
        _p(a), _p(a_row_of_pair), k, _p(codes), _p(scales), _p(expert_offsets), E, rows, N, K,
        epilogue, _p(out), _p(ws), 0 if ws is None else ws.numel(), _p(dev_status), _s(stream)))
    return out


def moe_combine(o, topk_w, pair_pos, y=None, stream=None):
    """y [T, H] = sum_j topk_w[t, j] * o[pair_pos[t*k + j]] (bf16 out)."""
    lib = _lib.load()
    T, k = topk_w.shape
    H = o.shape[1]
    dev = o.device
    _need("o", o, torch.bfloat16, (T * k, H), dev)
    _need("topk_w", topk_w, torch.float32, (T, k), dev)
    _need("pair_pos", pair_pos, torch.int32, (T * k,), dev)
    y = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if y is None else y
    _need("y", y, torch.bfloat16, (T, H), dev)
    _lib.check("moe_combine", lib.moe_combine(_p(o), _p(topk_w), _p(pair_pos), T, k, H, _p(y),
                                              _s(stream)))
    return y


RMS_EPS = 1e-6


def moe_rms_chain(y, x_next=None, eps: float = RMS_EPS, stream=None):
    """x_next [T, H] = bf16(y / sqrt(mean over each row of y^2 + eps)): the input of the next
    layer of a stack (bf16 in and out)."""
    lib = _lib.load()
    T, H = y.shape
    dev = y.device
    _need("y", y, torch.bfloat16, (T, H), dev)
    x_next = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if x_next is None else x_next
    _need("x_next", x_next, torch.bfloat16, (T, H), dev)
    _lib.check("moe_rms_chain", lib.moe_rms_chain(_p(y), T, H, eps, _p(x_next), _s(stream)))
    return x_next


def moe_w4a16_gmm_g(a, a_row_of_pair, k: int, codes, scales, expert_offsets, rows: int, group: int,
                    zeros=None, epilogue: int = W4_EPI_NONE, out=None, ws=None, dev_status=None,
                    stream=None):
    """The grouped GEMM on the weight-format variants: scales [E, N, K/group], zeros
    [E, N, K/group] uint8 or None."""
    lib = _lib.load()
    E, N, Kw = codes.shape
    K = Kw * 8
    dev = a.device
    _need("a", a, torch.bfloat16)
    if a.shape[1] != K:
        raise ValueError("a: wrong number of columns")
    if a_row_of_pair is not None:
        _need("a_row_of_pair", a_row_of_pair, torch.int32, (rows,), dev)
    _need("codes", codes, torch.int32, (E, N, K // 8), dev)
    _need("scales", scales, torch.bfloat16, (E, N, K // group), dev)
    if zeros is not None:
        _need("zeros", zeros, torch.uint8, (E, N, K // group), dev)
    _need("expert_offsets", expert_offsets, torch.int32, (E + 1,), dev)
    n_out = N // 2 if epilogue == W4_EPI_GELU_GATE else N
    out = torch.empty((rows, n_out), dtype=torch.bfloat16, device=dev) if out is None else out
    _need("out", out, torch.bfloat16, (rows, n_out), dev)
    if ws is None:
        ws = workspace(w4_workspace_bytes(_lib.W4_OP_GMM_G, rows, N, K, E, k), dev, stream)
    if dev_status is not None:
        _need("dev_status", dev_status, torch.int32, (1,), dev)
    _lib.check("moe_w4a16_gmm_g", lib.moe_w4a16_gmm_g(
        _p(a), _p(a_row_of_pair), k, _p(codes), _p(scales), _p(zeros), group, _p(expert_offsets), E,
        rows, N, K, epilogue, _p(out), _p(ws), 0 if ws is None else ws.numel(), _p(dev_status),
        _s(stream)))
    return out


def moe_layer_fusable(T: int, E: int, k: int, H: int, I: int) -> bool:
    """Whether moe_w4a16_layer accepts these sizes (1 <= T <= 128, T k <= 6 E, E <= 576)."""
    return T >= 1 and w4_workspace_bytes(_lib.W4_OP_LAYER, T, H, I, E, k) > 0


def layer_workspace(T: int, E: int, k: int, H: int, I: int, device) -> torch.Tensor:
    """A private workspace for moe_w4a16_layer, zero-filled (its control area must start at
    zero; every call leaves it so).  Not shared with other calls."""
    nbytes = w4_workspace_bytes(_lib.W4_OP_LAYER, T, H, I, E, k)
    if nbytes == 0:
        raise _lib.W4Error("moe_w4a16_layer", _lib.W4_ERR_UNSUPPORTED)
    return torch.zeros((nbytes + 255) // 256 * 256, dtype=torch.uint8, device=device)


def moe_w4a16_layer(x, logits, k: int, gu_codes, gu_scales, dn_codes, dn_scales, y=None, ws=None,
                    dev_status=None, stream=None):
    """One MoE decode layer in one kernel launch: x bf16 [T, H], logits f32 [T, E], gate/up
    codes [E, 2I, H/8] / scales [E, 2I, H/32], down codes [E, H, I/8] / scales [E, H, I/32]
    -> y bf16 [T, H].  ws: a workspace from layer_workspace (allocated here when None)."""
    lib = _lib.load()
    T, H = x.shape
    E, N2, _ = gu_codes.shape
    I = N2 // 2
    dev = x.device
    _need("x", x, torch.bfloat16, (T, H), dev)
    _need("logits", logits, torch.float32, (T, E), dev)
    _need("gu_codes", gu_codes, torch.int32, (E, 2 * I, H // 8), dev)
    _need("gu_scales", gu_scales, torch.bfloat16, (E, 2 * I, H // 32), dev)
    _need("dn_codes", dn_codes, torch.int32, (E, H, I // 8), dev)
    _need("dn_scales", dn_scales, torch.bfloat16, (E, H, I // 32), dev)
    y = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if y is None else y
    _need("y", y, torch.bfloat16, (T, H), dev)
    if ws is None:
        ws = layer_workspace(T, E, k, H, I, dev)
    _need("ws", ws, torch.uint8, None, dev)
    if dev_status is not None:
        _need("dev_status", dev_status, torch.int32, (1,), dev)
    _lib.check("moe_w4a16_layer", lib.moe_w4a16_layer(
        _p(x), _p(logits), T, E, k, _p(gu_codes), _p(gu_scales), _p(dn_codes), _p(dn_scales), H, I,
        _p(y), _p(ws), ws.numel(), _p(dev_status), _s(stream)))
    return y


class MoELayer:
    """One mixture-of-experts layer on the device: the four entry points composed on one stream
    (route -> gate/up GEMM with the GELU gate -> down GEMM -> combine), with every buffer
    allocated once so that a step launches kernels only.  fused=True runs the same layer as one
    moe_w4a16_layer launch (decode sizes only; its routing, h and o then stay in the layer's
    private workspace)."""

    def __init__(self, gu_codes, gu_scales, dn_codes, dn_scales, T: int, k: int, fused: bool = False):
        self.E, self.N2, _ = gu_codes.shape
        self.H = gu_codes.shape[2] * 8
        self.I = self.N2 // 2
        self.T, self.k = T, k
        dev = gu_codes.device
        self.w = (gu_codes, gu_scales, dn_codes, dn_scales)
        self.fused = fused
        if fused:
            self.layer_ws = layer_workspace(T, self.E, k, self.H, self.I, dev)
            self.y = torch.empty((T, self.H), dtype=torch.bfloat16, device=dev)
            return
        self.rt = Routing(torch.empty((T, k), dtype=torch.int32, device=dev),
                          torch.empty((T, k), dtype=torch.float32, device=dev),
                          torch.empty(self.E + 1, dtype=torch.int32, device=dev),
                          torch.empty(T * k, dtype=torch.int32, device=dev),
                          torch.empty(T * k, dtype=torch.int32, device=dev))
        self.h = torch.empty((T * k, self.I), dtype=torch.bfloat16, device=dev)
        self.o = torch.empty((T * k, self.H), dtype=torch.bfloat16, device=dev)
        self.y = torch.empty((T, self.H), dtype=torch.bfloat16, device=dev)
        nr = w4_workspace_bytes(_lib.W4_OP_ROUTE, T, 0, 0, self.E, k)
        # private: the routing outputs of layers that run back to back must not share scratch
        self.route_ws = torch.zeros(nr, dtype=torch.uint8, device=dev) if nr else None

    def __call__(self, x, logits, stream=None):
        gu_c, gu_s, dn_c, dn_s = self.w
        if self.fused:
            return moe_w4a16_layer(x, logits, self.k, gu_c, gu_s, dn_c, dn_s, y=self.y,
                                   ws=self.layer_ws, stream=stream)
        moe_route_permute(logits, self.k, out=self.rt, ws=self.route_ws, stream=stream)
        moe_w4a16_gmm(x, self.rt.sorted_pair, self.k, gu_c, gu_s, self.rt.expert_offsets,
                      self.T * self.k, W4_EPI_GELU_GATE, out=self.h, stream=stream)
        moe_w4a16_gmm(self.h, None, 1, dn_c, dn_s, self.rt.expert_offsets, self.T * self.k,
                      W4_EPI_NONE, out=self.o, stream=stream)
        moe_combine(self.o, self.rt.topk_w, self.rt.pair_pos, y=self.y, stream=stream)
        return self.y


# ---------------------------------------------------------------------------------------------
# the steps around the expert layers: norm, 8-bit linear, key/value cache and its attention
# ---------------------------------------------------------------------------------------------

def _device_call(fn):
    """Runs fn with the current device and stream set as its arguments ask: on `stream` when one is
    given (allocations included, so that a returned tensor belongs to that stream), otherwise on
    the current stream of the first tensor's device, whichever device is current."""
    name = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        first = args[0] if args else kw.get(name)
        if not isinstance(first, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor")
        if not first.is_cuda:
            raise ValueError(f"{name}: must live on a CUDA device")
        dev = first.device
        if stream is not None:
            if stream.device != dev:
                raise ValueError(f"stream: expected device {dev}, got {stream.device}")
            with torch.cuda.stream(stream):
                return fn(*args, **kw)
        if dev.index != _current_device():
            with torch.cuda.device(dev):
                return fn(*args, **kw)
        return fn(*args, **kw)
    return call


def _cur(dev) -> int:
    """The raw handle of dev's current stream (without building a Stream object, where torch allows)."""
    if _RAW_STREAM is not None:
        return _RAW_STREAM(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# (a CUDA tensor is at hand where this is called, so CUDA is up)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _fits(name, t, dtype, shape, dev):
    """_need's checks in one cheap expression; the details only when it fails."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev
            and t.is_contiguous()):
        _need(name, t, dtype, shape, dev)


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _rows3(name, t, heads, dim, dev):
    """A bf16 [T, heads, dim] tensor whose rows may be columns of a wider one; its row stride."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name}: expected {torch.bfloat16}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name}: expected device {dev}, got {t.device}")
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name}: expected shape [rows, {heads}, {dim}], got {tuple(shape)}")
    s = t.stride()
    if s[2] != 1 or (heads > 1 and s[1] != dim):
        raise ValueError(f"{name}: heads and elements of a row must be contiguous")
    return s[0] if shape[0] > 1 else heads * dim


@functools.lru_cache(maxsize=4096)
def _bytes_needed(op, m, n, k, e, index):
    """w4_workspace_bytes on the current device (whose index only keys the cache)."""
    return int(_lib.load().w4_workspace_bytes(op, m, n, k, e, 0))


def _scratch(ws, nbytes: int, dev):
    """(pointer, size, tensor to keep) of a call's scratch: ws, or one from torch's stream-ordered
    allocator, so that calls on different streams never share it and a call captured into a CUDA
    graph keeps it in that graph's own pool."""
    if ws is None:
        if not nbytes:
            return 0, 0, None
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        return ws.data_ptr(), nbytes, ws
    _need("ws", ws, torch.uint8, None, dev)
    return ws.data_ptr(), ws.numel(), ws


def linear_scratch(M: int, N: int, words: int, dev) -> torch.Tensor | None:
    """Scratch for one w4a16_linear call on codes [N, words] from torch's stream-ordered allocator (None when it
    needs none): unlike workspace()'s buffers, two captured graphs never share it."""
    n = _bytes_needed(_lib.W4_OP_LINEAR, M, N, 8 * words, 1, dev.index)
    return torch.empty(n, dtype=torch.uint8, device=dev) if n else None


def _rms_args(x, residual, weight, h):
    if x.dtype is not torch.bfloat16 or not x.is_contiguous():
        _need("x", x, torch.bfloat16)
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x: expected two dimensions")
    dev = x.device
    if residual is not None:
        _fits("residual", residual, torch.bfloat16, shape, dev)
        if h is None:
            h = torch.empty_like(x)
        else:
            _fits("h", h, torch.bfloat16, shape, dev)
    elif h is not None:
        raise ValueError("h: only written when a residual is given")
    if weight is not None:
        _fits("weight", weight, torch.bfloat16, shape[1:], dev)
    return shape, dev, h


@_device_call
def w4_rms_add(x, residual=None, weight=None, eps: float = RMS_EPS, h=None, y=None):
    """h = bf16(x + residual), y = bf16(h * weight / sqrt(mean over each row of h^2 + eps)); bf16
    [T, H] -> (y, h).  h is x itself without a residual; h may be passed as the residual's own
    buffer to update it in place."""
    shape, dev, h = _rms_args(x, residual, weight, h)
    if y is None:
        y = torch.empty_like(x)
    else:
        _fits("y", y, torch.bfloat16, shape, dev)
    _lib.rms_add(x.data_ptr(), _ptr(residual), _ptr(weight), shape[0], shape[1], eps, _ptr(h), y.data_ptr(), _cur(dev))
    return y, x if h is None else h


@_device_call
def w4_rms_add_q8(x, residual=None, weight=None, eps: float = RMS_EPS, h=None, q=None, q_scale=None):
    """w4_rms_add with 8-bit rows: (q int8 [T, H], q_scale f32 [T], h), y = q_scale * q."""
    shape, dev, h = _rms_args(x, residual, weight, h)
    if q is None:
        q = torch.empty_like(x, dtype=torch.int8)
    else:
        _fits("q", q, torch.int8, shape, dev)
    if q_scale is None:
        q_scale = torch.empty(shape[0], dtype=torch.float32, device=dev)
    else:
        _fits("q_scale", q_scale, torch.float32, shape[:1], dev)
    _lib.rms_add_q8(x.data_ptr(), _ptr(residual), _ptr(weight), shape[0], shape[1], eps, _ptr(h), q.data_ptr(),
                    q_scale.data_ptr(), _cur(dev))
    return q, q_scale, x if h is None else h


@_device_call
def w4a8_linear(xq, xs, codes, scales, y=None, ws=None, dev_status=None):
    """y [M, N] = xs * (xq [M, K] int8 @ dequant(codes, scales)^T), bf16 out.  dev_status: int32 [1], set where a
    bounded wait inside the kernels runs out (outputs lost to that are NaN)."""
    if xq.dim() != 2 or codes.dim() != 2:
        raise ValueError("xq, codes: expected two dimensions")
    M, K = xq.shape
    N = codes.shape[0]
    dev = xq.device
    _fits("xq", xq, torch.int8, (M, K), dev)
    _fits("xs", xs, torch.float32, (M,), dev)
    _fits("codes", codes, torch.int32, (N, K // 8), dev)
    _fits("scales", scales, torch.bfloat16, (N, K // 32), dev)
    if y is None:
        y = torch.empty_strided((M, N), (N, 1), dtype=torch.bfloat16, device=dev)   # (torch.empty: 0.9 us more)
    else:
        _fits("y", y, torch.bfloat16, (M, N), dev)
    if dev_status is not None:
        _fits("dev_status", dev_status, torch.int32, (1,), dev)
    p, n, ws = _scratch(ws, _bytes_needed(_lib.W4_OP_LINEAR_8, M, N, K, 1, dev.index), dev)
    _lib.linear_8(xq.data_ptr(), xs.data_ptr(), codes.data_ptr(), scales.data_ptr(), y.data_ptr(), M, N, K, p, n,
                  _ptr(dev_status), _cur(dev))
    return y


_KV_KINDS = {torch.bfloat16: (_lib.W4_KV_BF16, 1), torch.int8: (_lib.W4_KV_INT8, 1), torch.int32: (_lib.W4_KV_INT4, 8)}


def _cache_args(k_cache, v_cache, k_scales, v_scales, dev):
    """(kind, kv_heads, head_dim, pages, page_size) of a cache, its tensors checked."""
    if not isinstance(k_cache, torch.Tensor):
        raise TypeError("k_cache: expected a torch.Tensor")
    dtype, shape = k_cache.dtype, k_cache.shape
    if dtype not in _KV_KINDS:
        raise TypeError(f"k_cache: expected bfloat16, int8 or int32 words, got {dtype}")
    kind, per = _KV_KINDS[dtype]
    if len(shape) != 4:
        raise ValueError("k_cache: expected [pages, kv_heads, page_size, head_dim]")
    _fits("k_cache", k_cache, dtype, shape, dev)
    _fits("v_cache", v_cache, dtype, shape, dev)
    pages, heads, page_size, dim = shape
    dim *= per
    if kind == _lib.W4_KV_BF16:
        if k_scales is not None or v_scales is not None:
            raise ValueError("k_scales, v_scales: a bfloat16 cache has none")
    else:
        want = (pages, heads, page_size, dim // 32)
        _fits("k_scales", k_scales, torch.bfloat16, want, dev)
        _fits("v_scales", v_scales, torch.bfloat16, want, dev)
    return kind, heads, dim, pages, page_size


@_device_call
def kv_cache_write(k, v, slots, k_cache, v_cache, k_scales=None, v_scales=None, dev_status=None):
    """Rows k, v bf16 [T, kv_heads, head_dim] (rows may be strided) into the cache's slots int64 [T]
    (page * page_size + offset, negative: padded), quantised to the cache's kind: bfloat16, int8,
    or int4 (int32 words)."""
    dev = k.device
    kind, heads, dim, pages, page_size = _cache_args(k_cache, v_cache, k_scales, v_scales, dev)
    ks, vs = _rows3("k", k, heads, dim, dev), _rows3("v", v, heads, dim, dev)
    T = k.shape[0]
    if v.shape[0] != T:
        raise ValueError(f"v: expected {T} rows, got {v.shape[0]}")
    _fits("slots", slots, torch.int64, (T,), dev)
    if dev_status is not None:
        _fits("dev_status", dev_status, torch.int32, (1,), dev)
    _lib.kv_write(k.data_ptr(), v.data_ptr(), ks, vs, slots.data_ptr(), T, kind, heads, dim, pages, page_size,
                  k_cache.data_ptr(), v_cache.data_ptr(), _ptr(k_scales), _ptr(v_scales), _ptr(dev_status), _cur(dev))


@_device_call
def kv_cache_read(slots, k_cache, v_cache, k_scales=None, v_scales=None, k=None, v=None, dev_status=None):
    """The rows of slots int64 [T] as (k, v) bf16 [T, kv_heads, head_dim]; zeros for negative slots."""
    dev = slots.device
    kind, heads, dim, pages, page_size = _cache_args(k_cache, v_cache, k_scales, v_scales, dev)
    T = slots.shape[0]
    _fits("slots", slots, torch.int64, (T,), dev)
    want = (T, heads, dim)
    if k is None:
        k = torch.empty_strided(want, (heads * dim, dim, 1), dtype=torch.bfloat16, device=dev)
    else:
        _fits("k", k, torch.bfloat16, want, dev)
    if v is None:
        v = torch.empty_like(k)
    else:
        _fits("v", v, torch.bfloat16, want, dev)
    if dev_status is not None:
        _fits("dev_status", dev_status, torch.int32, (1,), dev)
    _lib.kv_read(slots.data_ptr(), T, kind, heads, dim, pages, page_size, k_cache.data_ptr(), v_cache.data_ptr(),
                 _ptr(k_scales), _ptr(v_scales), k.data_ptr(), v.data_ptr(), _ptr(dev_status), _cur(dev))
    return k, v


@_device_call
def kv_cache_attend(q, k_cache, v_cache, page_table, seq_lens, k_scales=None, v_scales=None, scale=None,
                    softcap: float = 0.0, window: int = 0, out=None, lse=None, ws=None, dev_status=None):
    """Attention of one query row per sequence, q bf16 [B, q_heads, head_dim] (rows may be strided),
    over the cached tokens named by page_table int32 [B, width] and seq_lens int32 [B] -> out bf16
    [B, q_heads, head_dim].  scale: 1 / sqrt(head_dim) when None; softcap, window: 0 for none;
    lse: float32 [B, q_heads] to receive log sum exp(score)."""
    dev = q.device
    kind, heads, dim, pages, page_size = _cache_args(k_cache, v_cache, k_scales, v_scales, dev)
    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q: expected [B, q_heads, head_dim]")
    B, q_heads, _ = shape
    qs = _rows3("q", q, q_heads, dim, dev)
    if page_table.dim() != 2:
        raise ValueError("page_table: expected [B, width]")
    width = page_table.shape[1]
    _fits("page_table", page_table, torch.int32, (B, width), dev)
    _fits("seq_lens", seq_lens, torch.int32, (B,), dev)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _fits("out", out, torch.bfloat16, shape, dev)
    if lse is not None:
        _fits("lse", lse, torch.float32, (B, q_heads), dev)
    if dev_status is not None:
        _fits("dev_status", dev_status, torch.int32, (1,), dev)
    p, n, ws = _scratch(ws, _bytes_needed(_lib.W4_OP_ATTEND, B, q_heads, dim, heads, dev.index), dev)
    _lib.kv_attend(
        q.data_ptr(), qs, k_cache.data_ptr(), v_cache.data_ptr(), _ptr(k_scales), _ptr(v_scales), kind,
        page_table.data_ptr(), width, seq_lens.data_ptr(), B, q_heads, heads, dim, pages, page_size,
        dim ** -0.5 if scale is None else scale, softcap, window, out.data_ptr(), _ptr(lse), p, n, _ptr(dev_status),
        _cur(dev))
    return out


class KVCache:
    """One layer's paged key/value cache and the calls on it.  kind: "bf16", "int8" or "int4" (codes
    with one bf16 scale per 32 elements of head_dim).  Freshly made it is zero throughout.  Rows of every head_dim that
    is a multiple of 32, up to 1024, are written and read; attention takes 64, 128, 192 and 256."""

    def __init__(self, pages: int, kv_heads: int, page_size: int, head_dim: int, kind: str = "int8", device="cuda"):
        if kind not in ("bf16", "int8", "int4"):
            raise ValueError(f"kind: expected bf16, int8 or int4, got {kind}")
        if head_dim % 32:
            raise ValueError("head_dim: expected a multiple of 32")
        dtype, per = {"bf16": (torch.bfloat16, 1), "int8": (torch.int8, 1), "int4": (torch.int32, 8)}[kind]
        shape = (pages, kv_heads, page_size)
        # int4 codes are stored as q + 8
        fill = -0x77777778 if kind == "int4" else 0
        self.k = torch.full((*shape, head_dim // per), fill, dtype=dtype, device=device)
        self.v = torch.full((*shape, head_dim // per), fill, dtype=dtype, device=device)
        self.k_scales = self.v_scales = None
        if kind != "bf16":
            self.k_scales = torch.zeros((*shape, head_dim // 32), dtype=torch.bfloat16, device=device)
            self.v_scales = torch.zeros_like(self.k_scales)
        self.kind, self.page_size = kind, page_size

    def write(self, k, v, slots, **kw):
        """kv_cache_write into this cache."""
        kv_cache_write(k, v, slots, self.k, self.v, self.k_scales, self.v_scales, **kw)

    def read(self, slots, **kw):
        """kv_cache_read from this cache."""
        return kv_cache_read(slots, self.k, self.v, self.k_scales, self.v_scales, **kw)

    def attend(self, q, page_table, seq_lens, **kw):
        """kv_cache_attend over this cache."""
        return kv_cache_attend(q, self.k, self.v, page_table, seq_lens, self.k_scales, self.v_scales, **kw)

    def slots(self, page_table, positions):
        """Slots int64 [B] of one position per sequence (int tensor [B]; negative positions stay
        padded): where a decode step writes its new rows.  A position on a negative page stays padded too;
        one that the table does not cover gets a slot past the cache, which a write reports and drops."""
        if page_table.dim() != 2 or page_table.shape[1] < 1:
            raise ValueError("page_table: expected [B, width], width at least 1")
        if positions.shape != page_table.shape[:1]:
            raise ValueError(f"positions: expected shape [{page_table.shape[0]}], got {tuple(positions.shape)}")
        pos = positions.long()
        at = pos.clamp(min=0)
        column = at // self.page_size
        page = torch.gather(page_table.long(), 1, column.clamp(max=page_table.shape[1] - 1)[:, None])[:, 0]
        slot = page * self.page_size + at % self.page_size
        past = self.k.shape[0] * self.page_size
        slot = torch.where(column >= page_table.shape[1], past, slot)
        return torch.where(pos < 0, -1, slot)

    def nbytes(self) -> int:
        """Device bytes of codes and scales."""
        return sum(t.numel() * t.element_size() for t in (self.k, self.v, self.k_scales, self.v_scales) if t is not None)
