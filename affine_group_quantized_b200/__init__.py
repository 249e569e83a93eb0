"""Python binding of libqmv, the B200 (sm_100a) affine group-quantized GEMV.

Argument marshalling only: every function here forwards to the C entry point
of the same name in ``libqmv.so`` (declared in ``include/qmv.h``) and every
step of the computation runs in that library's CUDA kernels.  There is no
CPU path: if ``libqmv.so`` is missing or no CUDA device is usable, calls
raise.

Arguments may be ``torch.Tensor`` (CUDA, contiguous; the data pointer is
passed) or plain integer device addresses.  bf16 buffers are ``torch.bfloat16``
tensors (or any 2-byte dtype holding bf16 bit patterns), packed weights are
``torch.int32``/``torch.uint32`` tensors.  ``stream`` defaults to the current
torch CUDA stream.  The ``kv_*`` calls refuse tensors of other types (float16 for
bf16, int64 or float32 for int32, ...); the others look at sizes alone.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqmv.so")

QMV_OK = 0
QMV_ERR_NULL = 1
QMV_ERR_SHAPE = 2
QMV_ERR_UNSUPPORTED = 3
QMV_ERR_ALIGN = 4
QMV_ERR_CUDA = 5

_STATUS_NAMES = {0: "QMV_OK", 1: "QMV_ERR_NULL", 2: "QMV_ERR_SHAPE",
                 3: "QMV_ERR_UNSUPPORTED", 4: "QMV_ERR_ALIGN", 5: "QMV_ERR_CUDA"}


class QmvError(RuntimeError):
    """A libqmv entry point returned a nonzero status."""

    def __init__(self, func: str, status: int, message: str):
        self.status = status
        super().__init__(f"{func}: {_STATUS_NAMES.get(status, status)}: {message}")


class _KVCacheStruct(ctypes.Structure):
    """qmv_kv_cache of include/qmv.h."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "k_scales", "k_biases", "v_scales",
                                                "v_biases")]
                + [(n, ctypes.c_int) for n in ("num_pages", "num_kv_heads", "page_size",
                                               "head_dim", "bits", "group_size")])


_lib = None


def lib() -> ctypes.CDLL:
    """Load libqmv.so (built in-tree by ``affine_group_quantized_b200.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m affine_group_quantized_b200.build` (nvcc, sm_100a)")
        L = ctypes.CDLL(LIB_PATH)
        P, I = ctypes.c_void_p, ctypes.c_int
        L.qmv.argtypes = [P, P, P, P, P, I, I, I, I, I, P]
        L.qmv_noalloc.argtypes = [P, P, P, P, P, I, I, I, I, I, P]
        L.qmv_gate_up.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, P]
        L.qmv_silu_gate_resid.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, P]
        L.gather_qmv.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I,
                                 P, P]
        for f in (L.qmv, L.qmv_noalloc, L.qmv_gate_up, L.qmv_silu_gate_resid, L.gather_qmv):
            f.restype = I
        L.qmv_last_error.restype = ctypes.c_char_p
        L.qmv_last_error.argtypes = []
        L.qmv_abi_version.restype = I
        L.qmv_abi_version.argtypes = []
        L.qvm.argtypes = [P, P, P, P, P, I, I, I, I, I, P]
        L.qmv_trellis.argtypes = [P, P, P, P, I, I, I, I, P]
        L.qmv_trellis.restype = I
        L.qvm.restype = I
        L.qmv_device_status.argtypes = [P, I, P]
        L.qmv_device_status.restype = I
        L.affine_quantize.argtypes = [P, P, P, P, I, I, I, I, P]
        L.affine_dequantize.argtypes = [P, P, P, P, I, I, I, I, P]
        L.affine_quantize.restype = I
        L.affine_dequantize.restype = I
        L.qmv_quant_last_error.restype = ctypes.c_char_p
        L.qmv_quant_last_error.argtypes = []
        Q, C = ctypes.c_longlong, ctypes.POINTER(_KVCacheStruct)
        L.kv_append.argtypes = [C, P, P, Q, Q, P, P, P, I, I, I, P, P, P, I, P, P]
        L.kv_read.argtypes = [C, P, P, Q, Q, P, P, P, I, I, I, P, P]
        L.kv_attention.argtypes = [C, P, Q, P, P, P, I, I, I, ctypes.c_float, P, I, P,
                                   ctypes.c_size_t, P, P]
        L.kv_attention_workspace.argtypes = [C, I, I, I, I, ctypes.POINTER(ctypes.c_size_t)]
        L.kv_evict.argtypes = [C] + [P] * 8 + [I] * 6 + [P, P]
        for f in (L.kv_append, L.kv_read, L.kv_attention, L.kv_attention_workspace, L.kv_evict):
            f.restype = I
        L.qmv_kv_last_error.restype = ctypes.c_char_p
        L.qmv_kv_last_error.argtypes = []
        _lib = L
    return _lib


EXPORTED = ("qmv", "qmv_noalloc", "qvm", "qmv_trellis", "qmv_gate_up", "qmv_silu_gate_resid", "gather_qmv",
            "qmv_last_error", "qmv_abi_version", "qmv_device_status", "affine_quantize",
            "affine_dequantize", "qmv_quant_last_error", "kv_append", "kv_read", "kv_attention",
            "kv_attention_workspace", "kv_evict", "qmv_kv_last_error")


def _ptr(a):
    if a is None:
        return None
    if isinstance(a, int):
        return a
    return a.data_ptr()


def _need(name, t, nbytes):
    """A tensor argument must hold at least the bytes the call reads or
    writes (plain integer addresses are the caller's responsibility)."""
    if t is None or isinstance(t, int):
        return
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{name}: {have} bytes, the call needs {nbytes}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _need_qmv(rows, codes, bits, gs, **arrays):
    """Sizes of a packed weight set: w [rows, codes*bits/32] uint32, scales
    and biases [rows, codes/gs] bf16."""
    _need("w", arrays.get("w"), rows * codes * bits // 8)
    for k in ("scales", "biases"):
        _need(k, arrays.get(k), 2 * rows * (codes // max(gs, 1)))


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(func: str, rc: int):
    if rc != QMV_OK:
        raise QmvError(func, rc, lib().qmv_last_error().decode())


def _check_quant(func: str, rc: int):
    if rc != QMV_OK:
        raise QmvError(func, rc, lib().qmv_quant_last_error().decode())


def last_error() -> str:
    return lib().qmv_last_error().decode()


def abi_version() -> int:
    return lib().qmv_abi_version()


def device_status(reset=False, stream=None) -> int:
    """The current device's kernel status word (0, or 2 if a bounded wait in
    some kernel gave up since the last reset); synchronizes `stream`."""
    out = ctypes.c_int(-1)
    _check("qmv_device_status", lib().qmv_device_status(ctypes.byref(out), 1 if reset else 0,
                                                        _stream(stream)))
    return out.value


def qmv(x, w, scales, biases, y, M, N, K, bits, group_size, stream=None):
    """y[M,N] = x[M,K] @ dequant(w).T  (see include/qmv.h)."""
    _need("x", x, 2 * M * K); _need("y", y, 2 * M * N)
    _need_qmv(N, K, bits, group_size, w=w, scales=scales, biases=biases)
    _check("qmv", lib().qmv(_ptr(x), _ptr(w), _ptr(scales), _ptr(biases),
                            _ptr(y), M, N, K, bits, group_size, _stream(stream)))


def qmv_noalloc(x, w, scales, biases, y, M, N, K, bits, group_size, stream=None):
    """qmv without device allocation by the library (see include/qmv.h)."""
    _need("x", x, 2 * M * K); _need("y", y, 2 * M * N)
    _need_qmv(N, K, bits, group_size, w=w, scales=scales, biases=biases)
    _check("qmv_noalloc", lib().qmv_noalloc(_ptr(x), _ptr(w), _ptr(scales), _ptr(biases),
                                            _ptr(y), M, N, K, bits, group_size,
                                            _stream(stream)))


def qvm(x, w, scales, biases, y, M, K, N, bits, group_size, stream=None):
    """y[M,N] = x[M,K] @ dequant(w) for w of K rows of N codes (see include/qmv.h)."""
    _need("x", x, 2 * M * K); _need("y", y, 2 * M * N)
    _need_qmv(K, N, bits, group_size, w=w, scales=scales, biases=biases)
    _check("qvm", lib().qvm(_ptr(x), _ptr(w), _ptr(scales), _ptr(biases), _ptr(y),
                            M, K, N, bits, group_size, _stream(stream)))


def qmv_trellis(x, w, scales, y, M, N, K, bits, stream=None):
    """Trellis-mode y[M,N] = scales[0] * x @ V.T (see include/qmv.h)."""
    _need("x", x, 2 * M * K); _need("y", y, 2 * M * N)
    _need("w", w, N * K * bits // 8); _need("scales", scales, 2)
    _check("qmv_trellis", lib().qmv_trellis(_ptr(x), _ptr(w), _ptr(scales), _ptr(y),
                                            M, N, K, bits, _stream(stream)))


def qmv_gate_up(x, w_gate, s_gate, b_gate, w_up, s_up, b_up, y_gate, y_up,
                M, N, K, bits, group_size, stream=None):
    """y_gate = x @ dequant(w_gate).T and y_up = x @ dequant(w_up).T, one launch."""
    _need("x", x, 2 * M * K); _need("y_gate", y_gate, 2 * M * N); _need("y_up", y_up, 2 * M * N)
    _need_qmv(N, K, bits, group_size, w=w_gate, scales=s_gate, biases=b_gate)
    _need_qmv(N, K, bits, group_size, w=w_up, scales=s_up, biases=b_up)
    _check("qmv_gate_up", lib().qmv_gate_up(
        _ptr(x), _ptr(w_gate), _ptr(s_gate), _ptr(b_gate), _ptr(w_up),
        _ptr(s_up), _ptr(b_up), _ptr(y_gate), _ptr(y_up), M, N, K, bits,
        group_size, _stream(stream)))


def qmv_silu_gate_resid(gate, up, x_resid, w, scales, biases, y, M, N, K,
                        bits, group_size, stream=None):
    """y = x_resid + dequant(w) @ (silu(gate) * up); x_resid may be None."""
    _need("gate", gate, 2 * M * K); _need("up", up, 2 * M * K); _need("y", y, 2 * M * N)
    _need("x_resid", x_resid, 2 * M * N)
    _need_qmv(N, K, bits, group_size, w=w, scales=scales, biases=biases)
    _check("qmv_silu_gate_resid", lib().qmv_silu_gate_resid(
        _ptr(gate), _ptr(up), _ptr(x_resid), _ptr(w), _ptr(scales),
        _ptr(biases), _ptr(y), M, N, K, bits, group_size, _stream(stream)))


def gather_qmv(x, w, scales, biases, lhs_indices, rhs_indices, y, num_pairs,
               num_x_rows, num_experts, N, K, bits, group_size,
               sorted_indices=False, d_status=None, stream=None):
    """y[p] = x[lhs[p]] @ dequant(w[rhs[p]]).T for every pair p."""
    _need("x", x, 2 * num_x_rows * K); _need("y", y, 2 * num_pairs * N)
    _need("lhs_indices", lhs_indices, 4 * num_pairs); _need("rhs_indices", rhs_indices, 4 * num_pairs)
    _need_qmv(num_experts * N, K, bits, group_size, w=w, scales=scales, biases=biases)
    _check("gather_qmv", lib().gather_qmv(
        _ptr(x), _ptr(w), _ptr(scales), _ptr(biases), _ptr(lhs_indices),
        _ptr(rhs_indices), _ptr(y), num_pairs, num_x_rows, num_experts, N, K,
        bits, group_size, 1 if sorted_indices else 0, _ptr(d_status),
        _stream(stream)))


def affine_quantize(w, w_q, scales, biases, N, K, bits, group_size, stream=None):
    """Quantize bf16 w[N,K] into packed w_q and bf16 scales/biases [N,K/gs]."""
    _need("w", w, 2 * N * K)
    _need_qmv(N, K, bits, group_size, w=w_q, scales=scales, biases=biases)
    _check_quant("affine_quantize", lib().affine_quantize(
        _ptr(w), _ptr(w_q), _ptr(scales), _ptr(biases), N, K, bits, group_size,
        _stream(stream)))


def affine_dequantize(w_q, scales, biases, w_hat, N, K, bits, group_size,
                      stream=None):
    """w_hat[N,K] = bf16(scale * q + bias) from the packed format."""
    _need("w_hat", w_hat, 2 * N * K)
    _need_qmv(N, K, bits, group_size, w=w_q, scales=scales, biases=biases)
    _check_quant("affine_dequantize", lib().affine_dequantize(
        _ptr(w_q), _ptr(scales), _ptr(biases), _ptr(w_hat), N, K, bits,
        group_size, _stream(stream)))


# ---------------------------------------------------------------------------
# The paged key-value cache
# ---------------------------------------------------------------------------


def _kv_error(func: str, rc: int):
    raise QmvError(func, rc, _kv().last_error())


class KVCache:
    """A paged key-value cache: the buffers and shape that every ``kv_*`` call
    takes (``qmv_kv_cache`` of include/qmv.h).  Rows (page, kv head, slot) of
    ``head_dim`` elements, packed codes with bf16 scales and biases for
    ``bits`` 4 or 8, bf16 rows (no scales; ``group_size`` ignored) for 16.
    The object keeps the buffers alive and holds nothing else.
    """

    def __init__(self, k, v, k_scales, k_biases, v_scales, v_biases, num_pages, num_kv_heads,
                 page_size, head_dim, bits, group_size):
        rows = num_pages * num_kv_heads * page_size
        for name, t in (("k", k), ("v", v)):
            _need(name, t, rows * head_dim * bits // 8)
            _of_type(name, t, bits == 16)
        if bits != 16:
            for name, t in (("k_scales", k_scales), ("k_biases", k_biases),
                            ("v_scales", v_scales), ("v_biases", v_biases)):
                _need(name, t, 2 * rows * (head_dim // max(group_size, 1)))
                _of_type(name, t, True)
        self.buffers = (k, v, k_scales, k_biases, v_scales, v_biases)
        self.num_pages, self.num_kv_heads, self.page_size = num_pages, num_kv_heads, page_size
        self.head_dim, self.bits, self.group_size = head_dim, bits, group_size
        self._struct = _KVCacheStruct(*(_ptr(t) for t in self.buffers), num_pages, num_kv_heads,
                                      page_size, head_dim, bits, group_size)
        self._address = ctypes.addressof(self._struct)
        self._device = None
        names = ("k", "v", "k_scales", "k_biases", "v_scales", "v_biases")
        for name, t in zip(names[:2 if bits == 16 else 6], self.buffers):
            d = _device_of(t)
            if self._device is None:
                self._device = d
            elif d not in (None, self._device):
                raise ValueError(f"{name}: on device {d}, the buffers before it on device "
                                 f"{self._device}")


def _bf16_types():
    """bf16, and the 2-byte integers that hold its bit patterns."""
    import torch
    return (torch.bfloat16, torch.int16, torch.uint16)


def _of_type(name, t, bf16):
    """A cache buffer holds bf16 values, or packed codes (any integers)."""
    if t is None or isinstance(t, int):
        return
    if bf16 and t.dtype not in _bf16_types():
        raise ValueError(f"{name}: must hold bf16 values, not {t.dtype}")
    if not bf16 and (t.dtype.is_floating_point or t.dtype.is_complex):
        raise ValueError(f"{name}: must hold packed codes (integers), not {t.dtype}")


def _device_of(t):
    """A tensor's CUDA device, or None for a plain address."""
    if t is None or isinstance(t, int):
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    return t.device.index


_native = None


def _kv():
    """The module with the kv_* calls' argument checks (csrc/kv_native.c)."""
    global _native
    if _native is None:
        lib()  # the library it calls
        try:
            from . import _kv_native
        except ImportError as e:
            raise RuntimeError(
                f"the binding's _kv_native module is missing ({e}): build it with "
                "`python -m affine_group_quantized_b200.build`") from e
        _setup(_kv_native)
        _native = _kv_native
    return _native


def _setup(native, current_device=None, current_stream=None):
    """Hands the module torch's types and functions (or a test's)."""
    import torch
    native.setup(
        current_device or getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
        current_stream or getattr(torch._C, "_cuda_getCurrentRawStream",
                                  lambda d: torch.cuda.current_stream(d).cuda_stream),
        _bf16_types(), (torch.int32, torch.uint32), (torch.float32,))


def kv_append(cache, k, v, block_table, lens, token_starts, batch, num_tokens, table_width,
              seen=None, positions=None, weights=None, state_width=0, k_stride=None,
              v_stride=None, d_status=None, stream=None):
    """Write num_tokens new tokens' keys and values into the cache: sequence b's
    tokens token_starts[b] .. token_starts[b+1]-1 (one token each without
    token_starts) fill its slots from lens[b] on (see include/qmv.h)."""
    rc = (_native or _kv()).append(
        cache._address, cache._device, k, v, block_table, lens, token_starts, batch, num_tokens,
        table_width, seen, positions, weights, state_width, k_stride, v_stride, d_status, stream)
    if rc:
        _kv_error("kv_append", rc)


def kv_read(cache, k, v, block_table, lens, token_starts, batch, num_tokens, table_width,
            k_stride=None, v_stride=None, d_status=None, stream=None):
    """Slots lens[b] .. of sequence b as dense bf16 rows token_starts[b] ..
    token_starts[b+1]-1 of k and v: the reverse of kv_append."""
    rc = (_native or _kv()).read(
        cache._address, cache._device, k, v, block_table, lens, token_starts, batch, num_tokens,
        table_width, k_stride, v_stride, d_status, stream)
    if rc:
        _kv_error("kv_read", rc)


def kv_attention_workspace(cache, batch, num_q_heads, table_width, with_weights=False) -> int:
    """Bytes of workspace kv_attention needs for these sizes, whatever the lengths."""
    n = ctypes.c_size_t(0)
    rc = lib().kv_attention_workspace(ctypes.byref(cache._struct), batch, num_q_heads, table_width,
                                      1 if with_weights else 0, ctypes.byref(n))
    if rc:
        raise QmvError("kv_attention_workspace", rc, lib().qmv_kv_last_error().decode())
    return n.value


def kv_attention(cache, q, block_table, lens, out, batch, num_q_heads, table_width, scale,
                 workspace, weights=None, state_width=0, q_stride=None, d_status=None,
                 stream=None):
    """Attention of one new token per sequence over its lens[b] slots; with
    weights, each slot's probabilities are added to them (see include/qmv.h).
    workspace: a tensor of kv_attention_workspace's bytes."""
    rc = (_native or _kv()).attention(
        cache._address, cache._device, q, block_table, lens, out, batch, num_q_heads,
        table_width, scale, workspace, weights, state_width, q_stride, d_status, stream)
    if rc:
        _kv_error("kv_attention", rc)


def kv_evict(cache, block_table, lens, seen, weights, positions, new_lens, new_weights,
             new_positions, batch, table_width, state_width, budget, recent=0, sinks=0,
             d_status=None, stream=None):
    """Keep the `budget` slots of every (sequence, kv head) with the largest
    weights, the newest `recent` and first `sinks` positions before all
    others, and move them below budget (see include/qmv.h)."""
    rc = (_native or _kv()).evict(
        cache._address, cache._device, block_table, lens, seen, weights, positions, new_lens,
        new_weights, new_positions, batch, table_width, state_width, budget, recent, sinks,
        d_status, stream)
    if rc:
        _kv_error("kv_evict", rc)
