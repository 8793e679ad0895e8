"""Python binding of libzn.so (include/zn.h): argument marshalling only.

Every step of setup, compression and decompression runs in the library's HIP
kernels; this module turns torch tensors into device pointers and streams,
and raises ZnError on a non-zero status.  There is no fallback: if libzn.so
is missing, every call raises.
"""
from __future__ import annotations

import ctypes as C
import functools
import math
import os
from typing import Sequence

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libzn.so")

BF16, FP32, FP8_E4M3, FP4X2_E2M1 = 0, 1, 2, 3
CODER_HUFFMAN, CODER_TANS = 0, 1
SETUP_PAIRS = 1
# FP4 E2M1 pairs travel as uint8 tensors (two values per byte, low nibble first)
TORCH_DTYPE = {BF16: torch.bfloat16, FP32: torch.float32, FP8_E4M3: torch.float8_e4m3fn,
               FP4X2_E2M1: torch.uint8}
ZN_DTYPE = {v: k for k, v in TORCH_DTYPE.items()}
STATUS = {0: "ok", -1: "invalid argument", -2: "corrupt container", -3: "buffer too small",
          -4: "tableset mismatch", -5: "HIP runtime error", -6: "out of memory"}
ROUNDS = 8


class ZnError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {STATUS.get(code, 'status %d' % code)}")
        self.code = code


_lib = None


def lib() -> C.CDLL:
    """Loads libzn.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ZnError(-1, f"libzn.so not built at {LIB_PATH} (run python lossless_float_weight_amd/build.py)")
        L = C.CDLL(LIB_PATH)
        P, U64, I, U32 = C.c_void_p, C.c_uint64, C.c_int, C.c_uint32
        PU64 = C.POINTER(C.c_uint64)
        L.zn_setup.argtypes = [I, C.POINTER(P), PU64, I, U32, I, P, C.POINTER(P)]
        L.zn_setup2.argtypes = [I, C.POINTER(P), PU64, I, U32, I, I, P, C.POINTER(P)]
        L.zn_tableset_pairs.argtypes = [P, I, C.POINTER(I), C.POINTER(I), C.POINTER(I), P, P]
        L.zn_setup_transfer.argtypes = [P, C.POINTER(P), PU64, I, P, C.POINTER(P)]
        L.zn_plan_from_container.argtypes = [P, U64, P, C.POINTER(P)]
        L.zn_header_info.argtypes = [P, U64, C.POINTER(I), C.POINTER(I), PU64, C.POINTER(U32),
                                     C.POINTER(U32), PU64, PU64]
        L.zn_tableset_info.argtypes = [P, C.POINTER(I), C.POINTER(I), PU64, C.POINTER(U32),
                                       C.POINTER(U32), C.POINTER(I), PU64]
        L.zn_compress_bound.argtypes = [P, PU64]
        L.zn_scratch_bytes.argtypes = [P, PU64]
        L.zn_compress.argtypes = [P, P, P, U64, PU64, P, U64, P]
        L.zn_compress2.argtypes = [P, I, P, P, U64, PU64, P, U64, P]
        L.zn_decompress.argtypes = [P, P, U64, P, P, U64, I, P]
        L.zn_decompress_noalloc.argtypes = [P, P, U64, P, P, I, P]
        L.zn_tableset_save.argtypes = [P, P, U64, PU64]
        L.zn_tableset_load.argtypes = [P, U64, C.POINTER(P)]
        L.zn_tableset_lengths.argtypes = [P, I, P]
        L.zn_tableset_map.argtypes = [P, P]
        L.zn_tableset_cost_history.argtypes = [P, PU64]
        L.zn_tableset_free.argtypes = [P]
        L.zn_status_str.restype = C.c_char_p
        L.zn_debug_histograms.argtypes = [P, P, P, P]
        L.zn_debug_code_lengths.argtypes = [P, I, I, I, P, P]
        L.zn_debug_kernel_events.argtypes = [C.c_char_p, P, P]
        L.zn_mx_quantize.argtypes = [I, P, U64, U64, U64, I, P, P, P]
        L.zn_mx_dequantize.argtypes = [I, P, P, U64, U64, I, P, U64, P]
        L.zn_mx_rms_norm.argtypes = [I, P, U64, P, U64, P, C.c_float, U64, U64, P, U64, I, P, P, P]
        L.zn_mx_matmul_scratch_bytes.argtypes = [I, I, U64, U64, U64, PU64]
        L.zn_mx_matmul.argtypes = [I, P, P, I, P, P, U64, U64, U64, I, P, U64, P, U64, P]
        L.zn_mx_matmul2.argtypes = [I, P, P, I, P, P, U64, U64, U64, U32, I, P, U64, P, U64, P]
        for f in ("zn_setup", "zn_setup_transfer", "zn_plan_from_container", "zn_header_info",
                  "zn_tableset_info", "zn_compress_bound",
                  "zn_scratch_bytes", "zn_compress", "zn_decompress", "zn_decompress_noalloc",
                  "zn_tableset_save",
                  "zn_tableset_load", "zn_tableset_lengths", "zn_tableset_map",
                  "zn_tableset_cost_history", "zn_debug_histograms", "zn_debug_code_lengths",
                  "zn_debug_kernel_events", "zn_mx_quantize", "zn_mx_dequantize", "zn_mx_rms_norm",
                  "zn_mx_matmul_scratch_bytes", "zn_mx_matmul", "zn_mx_matmul2"):
            getattr(L, f).restype = C.c_int
        _lib = L
    return _lib


def _check(rc: int, where: str) -> None:
    if rc != 0:
        raise ZnError(rc, where)


def _stream(stream) -> C.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _ptr_array(tensors: Sequence[torch.Tensor], device, stream=None) -> torch.Tensor:
    """Device array of the tensors' data pointers (the ABI's d_*_ptrs), its
    copy ordered on the stream the call runs on."""
    vals = torch.tensor([t.data_ptr() for t in tensors], dtype=torch.int64)
    if stream is None:
        return vals.to(device)
    with torch.cuda.stream(stream):
        return vals.to(device)


def _u64(vals):
    return (C.c_uint64 * len(vals))(*[int(v) for v in vals])


class Tableset:
    """Owns a zn_tableset handle (the plan and optional group tables)."""

    def __init__(self, handle: C.c_void_p):
        self.handle = handle

    def __del__(self):
        h = getattr(self, "handle", None)
        if h and _lib is not None:
            _lib.zn_tableset_free(h)
            self.handle = None

    def info(self) -> dict:
        """Plan facts (fixed for the handle's lifetime, so read once)."""
        if getattr(self, "_info", None) is None:
            self._info = self._read_info()
        return dict(self._info)

    def _read_info(self) -> dict:
        dt, T, nc, K = C.c_int(), C.c_int(), C.c_uint32(), C.c_int()
        cb, h = C.c_uint32(), C.c_uint64()
        _check(lib().zn_tableset_info(self.handle, C.byref(dt), C.byref(T), None, C.byref(cb),
                                      C.byref(nc), C.byref(K), C.byref(h)), "tableset_info")
        n = (C.c_uint64 * T.value)()
        _check(lib().zn_tableset_info(self.handle, None, None, n, None, None, None, None),
               "tableset_info")
        return {"dtype": dt.value, "n_tensors": T.value, "n_elems": [int(v) for v in n],
                "chunk_bytes": cb.value, "n_chunks": nc.value, "n_groups": K.value,
                "hash": h.value}

    @property
    def dtype(self) -> int:
        return self.info()["dtype"]

    @property
    def n_groups(self) -> int:
        return self.info()["n_groups"]

    @property
    def hash(self) -> int:
        return self.info()["hash"]

    def lengths(self, g: int) -> list:
        A = 16 if self.dtype in (FP8_E4M3, FP4X2_E2M1) else 256
        buf = (C.c_uint8 * A)()
        _check(lib().zn_tableset_lengths(self.handle, g, buf), "tableset_lengths")
        return list(buf)

    def pairs(self, g: int):
        """Group g's packed-pair code: (packs, F as a list, token lengths as a
        list of 512), or None when the setup has no pair codes."""
        has, packed, nf = C.c_int(), C.c_int(), C.c_int()
        F = (C.c_uint8 * 16)()
        tl = (C.c_uint8 * 512)()
        _check(lib().zn_tableset_pairs(self.handle, g, C.byref(has), C.byref(packed), C.byref(nf), F, tl),
               "tableset_pairs")
        if not has.value:
            return None
        return bool(packed.value), list(F)[: nf.value], list(tl)

    def group_map(self) -> list:
        buf = (C.c_uint8 * max(1, self.info()["n_chunks"]))()
        _check(lib().zn_tableset_map(self.handle, buf), "tableset_map")
        return list(buf)[: self.info()["n_chunks"]]

    def cost_history(self) -> list:
        buf = (C.c_uint64 * (ROUNDS + 1))()
        _check(lib().zn_tableset_cost_history(self.handle, buf), "cost_history")
        return [int(v) for v in buf]

    def save(self) -> bytes:
        n = C.c_uint64()
        _check(lib().zn_tableset_save(self.handle, None, 0, C.byref(n)), "tableset_save")
        buf = (C.c_uint8 * n.value)()
        _check(lib().zn_tableset_save(self.handle, buf, n.value, C.byref(n)), "tableset_save")
        return bytes(buf)

    @classmethod
    def load(cls, data: bytes) -> "Tableset":
        buf = (C.c_uint8 * len(data)).from_buffer_copy(data)
        h = C.c_void_p()
        _check(lib().zn_tableset_load(buf, len(data), C.byref(h)), "tableset_load")
        return cls(h)


def setup(tensors: Sequence[torch.Tensor] | None = None, *, dtype=None, n_elems=None,
          chunk_bytes: int = 262144, n_groups: int = 0, pairs: bool = False, stream=None) -> Tableset:
    """zn_setup (zn_setup2 with pairs): a plan for these tensor sizes; with
    n_groups > 0 the chunks of `tensors` are grouped and share code tables;
    pairs adds packed exponent pairs (BF16)."""
    if tensors is not None:
        tensors = [t.contiguous() for t in tensors]
        dtype = ZN_DTYPE[tensors[0].dtype]
        n_elems = [t.numel() for t in tensors]
        ptrs = (C.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])
    else:
        ptrs = None
        dtype = ZN_DTYPE.get(dtype, dtype)
    h = C.c_void_p()
    # the tableset lives on the tensors' device (else on the current one)
    with torch.cuda.device(tensors[0].device if tensors else None):
        _check(lib().zn_setup2(int(dtype), ptrs, _u64(n_elems), len(n_elems), chunk_bytes, n_groups,
                               SETUP_PAIRS if pairs else 0, _stream(stream), C.byref(h)), "setup")
    return Tableset(h)


def setup_transfer(src: Tableset, tensors: Sequence[torch.Tensor], stream=None) -> Tableset:
    """zn_setup_transfer: src's group codes for these tensors (same dtype and
    chunk size), each chunk assigned by content to its cheapest group code."""
    want = TORCH_DTYPE[src.info()["dtype"]]
    if any(t.dtype != want for t in tensors):
        raise ZnError(-1, f"setup_transfer: the source tableset codes {want}, got "
                          f"{sorted(set(str(t.dtype) for t in tensors))}")
    tensors = [t.contiguous() for t in tensors]
    ptrs = (C.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])
    h = C.c_void_p()
    with torch.cuda.device(tensors[0].device):
        _check(lib().zn_setup_transfer(src.handle, ptrs, _u64([t.numel() for t in tensors]), len(tensors),
                                       _stream(stream), C.byref(h)), "setup_transfer")
    return Tableset(h)


def plan_from_container(blob: torch.Tensor, stream=None) -> Tableset:
    h = C.c_void_p()
    with torch.cuda.device(blob.device):
        _check(lib().zn_plan_from_container(C.c_void_p(blob.data_ptr()), blob.numel(), _stream(stream),
                                            C.byref(h)), "plan_from_container")
    return Tableset(h)


def header_info(hdr) -> dict:
    """zn_header_info on the first 64 bytes of a container (host bytes, a
    numpy array or a tensor on any device)."""
    if isinstance(hdr, torch.Tensor):
        hdr = hdr[:64].cpu().numpy().tobytes()
    elif not isinstance(hdr, (bytes, bytearray)):
        hdr = bytes(memoryview(hdr)[:64])
    buf = (C.c_uint8 * max(1, len(hdr))).from_buffer_copy(bytes(hdr) or b"\0")
    dt, T = C.c_int(), C.c_int()
    n, tot, h = C.c_uint64(), C.c_uint64(), C.c_uint64()
    cb, nc = C.c_uint32(), C.c_uint32()
    _check(lib().zn_header_info(buf, len(hdr), C.byref(dt), C.byref(T), C.byref(n), C.byref(cb),
                                C.byref(nc), C.byref(tot), C.byref(h)), "header_info")
    return {"dtype": dt.value, "n_tensors": T.value, "n_elems": n.value, "chunk_bytes": cb.value,
            "n_chunks": nc.value, "total_bytes": tot.value, "tableset_hash": h.value}


def _check_tensors(ts: Tableset, tensors, where: str, exact: bool) -> None:
    """The tensors must be the plan's: count, dtype, one CUDA device,
    contiguous storage, and exactly (inputs) or at least (outputs) the
    plan's element counts.  Raises ZnError(-1) before any launch."""
    info = ts.info()
    want = TORCH_DTYPE[info["dtype"]]
    if len(tensors) != info["n_tensors"]:
        raise ZnError(-1, f"{where}: plan has {info['n_tensors']} tensors, got {len(tensors)}")
    dev = None
    for i, (t, n) in enumerate(zip(tensors, info["n_elems"])):
        if t.dtype != want:
            raise ZnError(-1, f"{where}: tensor {i} is {t.dtype}, the plan codes {want}")
        if not t.is_cuda or (dev is not None and t.device != dev):
            raise ZnError(-1, f"{where}: tensor {i} is not on the plan's CUDA device")
        dev = t.device
        if not t.is_contiguous():
            raise ZnError(-1, f"{where}: tensor {i} is not contiguous (pass .contiguous())")
        if (t.numel() != n) if exact else (t.numel() < n):
            raise ZnError(-1, f"{where}: tensor {i} has {t.numel()} elements, the plan {n}")


def _keep_alive(stream, *tensors) -> None:
    """Temporaries of an asynchronous call on a stream other than the current
    one stay allocated until that stream's work is done."""
    if stream is None:
        return
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def compress_bound(ts: Tableset) -> int:
    b = C.c_uint64()
    _check(lib().zn_compress_bound(ts.handle, C.byref(b)), "compress_bound")
    return b.value


def scratch_bytes(ts: Tableset) -> int:
    b = C.c_uint64()
    _check(lib().zn_scratch_bytes(ts.handle, C.byref(b)), "scratch_bytes")
    return b.value


def new_scratch(ts: Tableset, device="cuda") -> torch.Tensor:
    return torch.empty(scratch_bytes(ts), dtype=torch.uint8, device=device)


def compress(ts: Tableset, tensors: Sequence[torch.Tensor], out: torch.Tensor | None = None,
             scratch: torch.Tensor | None = None, ptrs: torch.Tensor | None = None,
             sync: bool = True, stream=None):
    """zn_compress.  Returns the container (a view of `out`) when sync, else
    `out` itself (size at byte 56 once the stream has run)."""
    return compress2(ts, CODER_HUFFMAN, tensors, out, scratch, ptrs, sync, stream)


def compress2(ts: Tableset, coder: int, tensors: Sequence[torch.Tensor], out: torch.Tensor | None = None,
              scratch: torch.Tensor | None = None, ptrs: torch.Tensor | None = None,
              sync: bool = True, stream=None):
    """zn_compress2: compress with the exponent stream's coder chosen
    (CODER_HUFFMAN or CODER_TANS)."""
    _check_tensors(ts, tensors, "compress", exact=True)
    dev = tensors[0].device
    tmp = []
    if out is None:
        out = torch.empty(compress_bound(ts), dtype=torch.uint8, device=dev)
    if scratch is None:
        scratch = new_scratch(ts, dev)
        tmp.append(scratch)
    if ptrs is None:
        ptrs = _ptr_array(tensors, dev, stream)
        tmp.append(ptrs)
    for name, b in (("out", out), ("scratch", scratch)):
        if b.device != dev or not b.is_contiguous() or b.dtype != torch.uint8:
            raise ZnError(-1, f"compress: {name} must be a contiguous uint8 tensor on {dev}")
    if not sync:
        _keep_alive(stream, *tmp)
    nb = C.c_uint64()
    with torch.cuda.device(dev):   # the tableset must live on the tensors' device
        _check(lib().zn_compress2(ts.handle, int(coder), C.c_void_p(ptrs.data_ptr()),
                                  C.c_void_p(out.data_ptr()), out.numel(), C.byref(nb) if sync else None,
                                  C.c_void_p(scratch.data_ptr()), scratch.numel(), _stream(stream)),
               "compress")
    return out[: nb.value] if sync else out


def decompress(ts: Tableset, blob: torch.Tensor, outs: Sequence[torch.Tensor] | None = None,
               scratch: torch.Tensor | None = None, ptrs: torch.Tensor | None = None,
               sync: bool = True, stream=None):
    """zn_decompress into `outs` (allocated from the plan when None)."""
    if not blob.is_cuda or not blob.is_contiguous() or blob.dtype != torch.uint8:
        raise ZnError(-1, "decompress: the container must be a contiguous uint8 CUDA tensor")
    if outs is None:
        info = ts.info()
        outs = [torch.empty(n, dtype=TORCH_DTYPE[info["dtype"]], device=blob.device)
                for n in info["n_elems"]]
    _check_tensors(ts, outs, "decompress", exact=False)
    if outs and outs[0].device != blob.device:
        raise ZnError(-1, "decompress: outputs and container on different devices")
    tmp = []
    if scratch is None:
        scratch = torch.empty(256, dtype=torch.uint8, device=blob.device)
        tmp.append(scratch)
    if ptrs is None:
        ptrs = _ptr_array(outs, blob.device, stream)
        tmp.append(ptrs)
    if not sync:
        _keep_alive(stream, *tmp)
    with torch.cuda.device(blob.device):
        _check(lib().zn_decompress(ts.handle, C.c_void_p(blob.data_ptr()), blob.numel(),
                                   C.c_void_p(ptrs.data_ptr()), C.c_void_p(scratch.data_ptr()),
                                   scratch.numel(), 1 if sync else 0, _stream(stream)), "decompress")
    return outs


def decompress_noalloc(ts: Tableset, blob: torch.Tensor, outs: Sequence[torch.Tensor],
                       ptrs: torch.Tensor, status: torch.Tensor | None = None, sync: bool = True,
                       stream=None):
    """zn_decompress_noalloc: the library allocates nothing; the caller
    passes the outputs, their device pointer array and optionally a device
    int32 `status` that receives the error word."""
    if not blob.is_cuda or not blob.is_contiguous() or blob.dtype != torch.uint8:
        raise ZnError(-1, "decompress_noalloc: the container must be a contiguous uint8 CUDA tensor")
    _check_tensors(ts, outs, "decompress_noalloc", exact=False)
    if ptrs.device != blob.device or ptrs.dtype != torch.int64 or ptrs.numel() != len(outs):
        raise ZnError(-1, "decompress_noalloc: ptrs must be the outputs' int64 device pointers")
    if status is not None and (status.device != blob.device or status.dtype != torch.int32):
        raise ZnError(-1, "decompress_noalloc: status must be an int32 tensor on the container's device")
    with torch.cuda.device(blob.device):
        _check(lib().zn_decompress_noalloc(ts.handle, C.c_void_p(blob.data_ptr()), blob.numel(),
                                           C.c_void_p(ptrs.data_ptr()),
                                           C.c_void_p(status.data_ptr()) if status is not None else None,
                                           1 if sync else 0, _stream(stream)), "decompress_noalloc")
    return outs


# ------------------------------------------------------- microscaled numbers --
# Rows of FP8 E4M3 codes (torch.float8_e4m3fn) or FP4 E2M1 pairs (torch.uint8)
# with one E8M0 scale byte (torch.float8_e8m0fnu, or the same as uint8) for
# every 32 values; the last axis is the row, filled up to whole blocks.
MX_BLOCK = 32
MX_FAST_SUMS = 1
_MX_FMT = {torch.float8_e4m3fn: FP8_E4M3, torch.uint8: FP4X2_E2M1}
_MX_PLAIN = {torch.bfloat16: BF16, torch.float32: FP32}
_MX_SCALE = (torch.float8_e8m0fnu, torch.uint8)


def _mx_device(where: str, stream, first: torch.Tensor, *others) -> torch.device:
    """The one CUDA device of the call's tensors (and of its stream)."""
    i = first.get_device()
    for t in others:
        if t is not None and t.get_device() != i:
            raise ZnError(-1, f"{where}: tensors on {first.device} and {t.device}")
    if i < 0:
        raise ZnError(-1, f"{where}: the tensors are on {first.device}, not on a CUDA device")
    if stream is not None and stream.device.index != i:
        raise ZnError(-1, f"{where}: the stream is on {stream.device}, the tensors on {first.device}")
    return first.device


def _torch_c(name: str, public):
    """A function of torch's own module that saves microseconds a call, or the
    public one where this torch has none of the name."""
    return getattr(torch._C, name, None) or public


_current_device = _torch_c("_cuda_getDevice", lambda: torch.cuda.current_device())
_current_raw_stream = _torch_c("_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)


def _mx_call(where: str, dev: torch.device, stream, function, *args) -> None:
    """The library call on the tensors' device and the stream (its current one when None)."""
    if _current_device() != dev.index:
        with torch.cuda.device(dev):
            return _mx_call(where, dev, stream, function, *args)
    # the handle alone: making a Stream object takes longer than the launch
    raw = stream.cuda_stream if stream is not None else _current_raw_stream(dev.index)
    rc = function(*args, raw)
    if rc:
        raise ZnError(rc, where)


def _mx_rows(where: str, name: str, t: torch.Tensor, write: bool = False):
    """(rows, k, row stride) of a plain tensor whose last axis is dense and
    whose other axes are evenly spaced rows."""
    if t.dim() == 0:
        raise ZnError(-1, f"{where}: {name} has no axis")
    k = t.shape[-1]
    if t.is_contiguous():
        n = t.numel()
        return (n // k if n else math.prod(t.shape[:-1])), k, k
    stride, rows = None, 1
    for n, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if stride is None:
            stride = st
        elif st != stride * rows:
            stride = -1
        rows *= n
    if rows == 0:
        return 0, k, k
    if stride is None:
        stride = k
    if (k > 1 and t.stride(-1) != 1) or stride < 0 or (write and rows > 1 and stride < k):
        raise ZnError(-1, f"{where}: {name} is not made of evenly spaced dense rows (pass .contiguous())")
    return rows, k, stride


def _mx_new(dtype, dev, stream, *shape) -> torch.Tensor:
    """An output on the stream that writes it; it may be used on the current
    stream too (once that has waited for the call's)."""
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        t = torch.empty(*shape, dtype=dtype, device=dev)
    t.record_stream(torch.cuda.current_stream(dev))
    return t


def _mx_given(where: str, name: str, t: torch.Tensor, shape, dtypes) -> None:
    """A packed tensor of the call: type, shape and dense rows."""
    if t.dtype not in dtypes or t.shape != shape:
        raise ZnError(-1, f"{where}: {name} is {t.dtype} {tuple(t.shape)}, wanted {dtypes[0]} {tuple(shape)}")
    if not t.is_contiguous():
        raise ZnError(-1, f"{where}: {name} is not contiguous (pass .contiguous())")


def _mx_packed(where: str, name: str, codes: torch.Tensor, scales: torch.Tensor):
    """(fmt, stored row length, leading shape) of codes and their scales, checked."""
    fmt = _MX_FMT.get(codes.dtype)
    shape = codes.shape
    if fmt is None or not shape:
        raise ZnError(-1, f"{where}: {name} is {codes.dtype}, wanted float8_e4m3fn, or uint8 pairs of E2M1, in rows")
    lead, kp = shape[:-1], shape[-1] if fmt == FP8_E4M3 else shape[-1] * 2
    if kp == 0 or kp % MX_BLOCK:
        raise ZnError(-1, f"{where}: {name} has rows of {kp} values, wanted whole blocks of {MX_BLOCK}")
    if not codes.is_contiguous():
        raise ZnError(-1, f"{where}: {name} is not contiguous (pass .contiguous())")
    _mx_given(where, name + "'s scales", scales, (*lead, kp // MX_BLOCK), _MX_SCALE)
    return fmt, kp, lead


def _mx_use(stream, *tensors) -> None:
    """Tensors of a call on another stream than the current one stay
    allocated until that stream's work is done."""
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _mx_no_grad(where: str, **tensors) -> None:
    """The operators have no gradient: a plain output whose graph would end
    here, or a given one that autograd watches, is refused."""
    if torch.is_grad_enabled():
        for name, t in tensors.items():
            if t is not None and t.requires_grad:
                raise ZnError(-1, f"{where}: {name} requires a gradient, which the operator has not "
                                  "(pass .detach(), or call under torch.no_grad())")


def _mx_codes(where, lead, k, fmt, codes, scales, dev, stream):
    """The output pair, given or made."""
    if fmt == FP8_E4M3:
        dt, width = torch.float8_e4m3fn, MX_BLOCK
    elif fmt == FP4X2_E2M1:
        dt, width = torch.uint8, MX_BLOCK // 2
    else:
        raise ZnError(-1, f"{where}: fmt is {fmt!r}, wanted FP8_E4M3 or FP4X2_E2M1")
    if k == 0:
        raise ZnError(-1, f"{where}: rows of no values")
    nb = -(-k // MX_BLOCK)
    if codes is None:
        codes = _mx_new(dt, dev, stream, *lead, nb * width)
    else:
        _mx_given(where, "codes", codes, (*lead, nb * width), (dt,))
    if scales is None:
        scales = _mx_new(torch.float8_e8m0fnu, dev, stream, *lead, nb)
    else:
        _mx_given(where, "scales", scales, (*lead, nb), _MX_SCALE)
    return codes, scales


def _mx_plain(where: str, name: str, dtype) -> int:
    if dtype not in _MX_PLAIN:
        raise ZnError(-1, f"{where}: {name} is {dtype}, wanted bfloat16 or float32")
    return _MX_PLAIN[dtype]


def _mx_out(where, lead, n, dtype, out, dev, stream):
    """(tensor, type, rows, row stride) of a plain output, given or made."""
    if out is None:
        dt = _mx_plain(where, "dtype", dtype)
        return _mx_new(dtype, dev, stream, *lead, n), dt, math.prod(lead), n
    if out.shape != (*lead, n):
        raise ZnError(-1, f"{where}: out is {tuple(out.shape)}, wanted {(*lead, n)}")
    dt = _mx_plain(where, "out", out.dtype)
    rows, _, stride = _mx_rows(where, "out", out, write=True)
    return out, dt, rows, stride


def mx_quantize(x: torch.Tensor, fmt: int = FP8_E4M3, codes: torch.Tensor | None = None,
                scales: torch.Tensor | None = None, stream=None):
    """zn_mx_quantize: rows of x (last axis; BF16 or FP32) to (codes, scales).
    The codes are the tensors that a FP8_E4M3 or FP4X2_E2M1 plan compresses."""
    where = "mx_quantize"
    dt = _mx_plain(where, "x", x.dtype)
    dev = _mx_device(where, stream, x, codes, scales)
    rows, k, stride = _mx_rows(where, "x", x)
    codes, scales = _mx_codes(where, x.shape[:-1], k, fmt, codes, scales, dev, stream)
    _mx_call(where, dev, stream, lib().zn_mx_quantize, dt, x.data_ptr(), stride, rows, k, fmt, codes.data_ptr(),
             scales.data_ptr())
    if stream is not None:
        _mx_use(stream, x, codes, scales)
    return codes, scales


def mx_dequantize(codes: torch.Tensor, scales: torch.Tensor, k: int | None = None, dtype=torch.bfloat16,
                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """zn_mx_dequantize: the values of the first k of every row (all stored
    ones when None), in BF16 or FP32."""
    where = "mx_dequantize"
    _mx_no_grad(where, out=out)
    fmt, kp, lead = _mx_packed(where, "codes", codes, scales)
    if k is None:
        k = kp
    if not kp - MX_BLOCK < k <= kp:
        raise ZnError(-1, f"{where}: {k} values do not fill rows of {kp}")
    dev = _mx_device(where, stream, codes, scales, out)
    out, dt, rows, stride = _mx_out(where, lead, k, dtype, out, dev, stream)
    _mx_call(where, dev, stream, lib().zn_mx_dequantize, fmt, codes.data_ptr(), scales.data_ptr(), rows, k, dt,
             out.data_ptr(), stride)
    if stream is not None:
        _mx_use(stream, codes, scales, out)
    return out


def mx_rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-5,
                fmt: int = FP8_E4M3, codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                residual_out: torch.Tensor | None = None, stream=None):
    """zn_mx_rms_norm: (codes, scales, h) of h = x + residual normed and
    quantised; h is stored in residual_out (x or residual itself is fine).
    Without a residual h is x.  No gradient: with a residual, an x or residual
    that requires one is refused while gradients are recorded."""
    where = "mx_rms_norm"
    if residual is not None:  # without one h is x itself
        _mx_no_grad(where, x=x, residual=residual, residual_out=residual_out)
    dt = _mx_plain(where, "x", x.dtype)
    dev = _mx_device(where, stream, x, weight, residual, residual_out, codes, scales)
    rows, k, stride = _mx_rows(where, "x", x)
    if weight.dtype != x.dtype or weight.shape != (k,) or not weight.is_contiguous():
        raise ZnError(-1, f"{where}: weight is {weight.dtype} {tuple(weight.shape)}, wanted dense {x.dtype} {(k,)}")
    if residual is None and residual_out is not None:
        raise ZnError(-1, f"{where}: residual_out without a residual")
    if not math.isfinite(eps) or eps < 0:
        raise ZnError(-1, f"{where}: eps is {eps}")
    rs = hs = 0
    if residual is not None:
        if residual.dtype != x.dtype or residual.shape != x.shape:
            raise ZnError(-1, f"{where}: residual is {residual.dtype} {tuple(residual.shape)}, x {x.dtype} {tuple(x.shape)}")
        rs = _mx_rows(where, "residual", residual)[2]
        if residual_out is None:
            residual_out, hs = _mx_new(x.dtype, dev, stream, *x.shape), k
        elif residual_out.dtype != x.dtype or residual_out.shape != x.shape:
            raise ZnError(-1, f"{where}: residual_out is {residual_out.dtype} {tuple(residual_out.shape)}, "
                              f"x {x.dtype} {tuple(x.shape)}")
        else:
            hs = _mx_rows(where, "residual_out", residual_out, write=True)[2]
    codes, scales = _mx_codes(where, x.shape[:-1], k, fmt, codes, scales, dev, stream)
    _mx_call(where, dev, stream, lib().zn_mx_rms_norm, dt, x.data_ptr(), stride,
             residual.data_ptr() if residual is not None else None, rs, weight.data_ptr(), eps, rows, k,
             residual_out.data_ptr() if residual is not None else None, hs, fmt, codes.data_ptr(), scales.data_ptr())
    if stream is not None:
        _mx_use(stream, x, weight, residual, residual_out, codes, scales)
    return codes, scales, (x if residual is None else residual_out)


@functools.lru_cache(maxsize=4096)
def mx_matmul_scratch_bytes(a_fmt: int, w_fmt: int, m: int, n: int, k: int) -> int:
    """zn_mx_matmul_scratch_bytes: device scratch of a product of m rows with
    n rows of stored length k."""
    b = C.c_uint64()
    _check(lib().zn_mx_matmul_scratch_bytes(a_fmt, w_fmt, m, n, k, C.byref(b)), "mx_matmul_scratch_bytes")
    return b.value


def mx_matmul(a: torch.Tensor, a_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
              dtype=torch.bfloat16, out: torch.Tensor | None = None, scratch: torch.Tensor | None = None,
              stream=None, fast_sums: bool = False) -> torch.Tensor:
    """zn_mx_matmul: a [..., k] by the rows of w [n, k], both microscaled (FP8
    or FP4 each), as BF16 or FP32 [..., n], summed in FP32.  fast_sums
    (zn_mx_matmul2 with ZN_MX_FAST_SUMS, BF16 only) adds FP8 products by the
    scaled matrix instruction: faster, with fewer bits."""
    where = "mx_matmul"
    _mx_no_grad(where, out=out)
    fa, k, lead = _mx_packed(where, "a", a, a_scales)
    fw, kw, wlead = _mx_packed(where, "w", w, w_scales)
    if len(wlead) != 1 or kw != k:
        raise ZnError(-1, f"{where}: w has rows of {kw} values and {w.dim()} axes, wanted {k} and 2")
    dev = _mx_device(where, stream, a, a_scales, w, w_scales, out, scratch)
    n = wlead[0]
    out, dt, m, stride = _mx_out(where, lead, n, dtype, out, dev, stream)
    if fast_sums and dt != BF16:
        raise ZnError(-1, f"{where}: fast_sums is for bfloat16 results, not {out.dtype}")
    need = mx_matmul_scratch_bytes(fa, fw, m, n, k)
    sa, sw = a_scales.data_ptr(), w_scales.data_ptr()
    if scratch is None:
        if (sa | sw) % 16 and k % 512 == 0 and m > 16:
            need += (m + n) * k // MX_BLOCK  # room to lay the scales out
        scratch = _mx_new(torch.uint8, dev, stream, need) if need else None
    elif scratch.dtype != torch.uint8 or not scratch.is_contiguous() or scratch.numel() < need:
        raise ZnError(-1, f"{where}: scratch must be a contiguous uint8 tensor of at least {need} bytes")
    _mx_call(where, dev, stream, lib().zn_mx_matmul2, fa, a.data_ptr(), sa, fw, w.data_ptr(), sw,
             m, n, k, MX_FAST_SUMS if fast_sums else 0, dt, out.data_ptr(), stride,
             scratch.data_ptr() if scratch is not None else None, scratch.numel() if scratch is not None else 0)
    if stream is not None:
        _mx_use(stream, a, a_scales, w, w_scales, out, scratch)
    return out


def debug_histograms(ts: Tableset, tensors: Sequence[torch.Tensor], stream=None) -> torch.Tensor:
    info = ts.info()
    nc = {BF16: 1, FP32: 4, FP8_E4M3: 2, FP4X2_E2M1: 2}[info["dtype"]]
    hist = torch.zeros((info["n_chunks"], nc, 256), dtype=torch.int32, device=tensors[0].device)
    ptrs = _ptr_array(tensors, tensors[0].device)
    _check(lib().zn_debug_histograms(ts.handle, C.c_void_p(ptrs.data_ptr()),
                                     C.c_void_p(hist.data_ptr()), _stream(stream)), "histograms")
    torch.cuda.synchronize()
    return hist


def debug_code_lengths(hist: torch.Tensor, alphabet: int = 256, group_rule: bool = False,
                       stream=None) -> torch.Tensor:
    """Device package-merge of n histograms (int64 [n, 256] on the GPU)."""
    hist = hist.to(torch.int64).contiguous()
    out = torch.zeros(hist.shape, dtype=torch.uint8, device=hist.device)
    _check(lib().zn_debug_code_lengths(C.c_void_p(hist.data_ptr()), hist.shape[0], alphabet,
                                       1 if group_rule else 0, C.c_void_p(out.data_ptr()),
                                       _stream(stream)), "code_lengths")
    torch.cuda.synchronize()
    return out


def debug_kernel_events(kernel: str, before=None, after=None) -> None:
    """zn_debug_kernel_events with torch.cuda.Event objects (None stops the
    recording for that kernel).  Events not yet created are created here."""
    def handle(e):
        if e is None:
            return None
        if not e.cuda_event:
            e.record()
        return C.c_void_p(e.cuda_event)
    _check(lib().zn_debug_kernel_events(kernel.encode(), handle(before), handle(after)),
           "kernel_events")
