"""Thin ctypes binding of the C ABI in include/eva_vq.h.

Functions carry the C names and only marshal arguments: every step of the
layer runs in the CUDA library.  PyTorch is used for device memory and
streams only (``VQLinear``).  There is no CPU fallback: if the library cannot
be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build

EVA_OK, EVA_ERR_INVALID_ARG, EVA_ERR_UNSUPPORTED, EVA_ERR_CUDA, EVA_ERR_OOM, \
    EVA_ERR_DEVICE_TIMEOUT, EVA_ERR_NO_DEVICE, EVA_ERR_DEVICE_CHECK, EVA_ERR_SCRATCH_TOO_SMALL, \
    EVA_ERR_BAD_INDEX = range(10)
EVA_F16, EVA_F32 = 0, 1
EVA_ROPE_HALF, EVA_ROPE_INTERLEAVED = 0, 1
EVA_ROPE_UNSCALED, EVA_ROPE_LINEAR, EVA_ROPE_NTK, EVA_ROPE_YARN, EVA_ROPE_BANDS = range(5)
EVA_CACHE_INT8, EVA_CACHE_E4M3 = 0, 1
EVA_PATH_AUTO, EVA_PATH_OC_LOOKUP, EVA_PATH_DEQUANT_MMA, EVA_PATH_TCGEN05 = 0, 1, 2, 3

# Every function the header declares; the CPU tests check the library exports them.
EVA_RUN_INDEPENDENT = 1

ABI_FUNCTIONS = (
    "eva_vq_linear_create", "eva_vq_linear_run", "eva_vq_linear_run_ex", "eva_vq_linear_run_host",
    "eva_vq_linear_destroy", "eva_vq_unpack_indices", "eva_vq_sync_status",
    "eva_vq_status_string", "eva_vq_linear_info", "eva_vq_device_check_record",
    "eva_vq_debug_timeline", "eva_vq_linear_run_noalloc",
    "eva_vq_quantize", "eva_vq_kmeans_assign", "eva_vq_kmeans_update", "eva_vq_residual",
    "eva_vq_linear_run_group", "eva_vq_debug_inject_wait_timeout",
    "eva_rope_create", "eva_rope_run", "eva_rope_destroy",
    "eva_kv_create", "eva_kv_append", "eva_kv_read", "eva_kv_attend", "eva_kv_sync_status",
    "eva_kv_debug_inject_wait_timeout", "eva_kv_cache_info", "eva_kv_destroy",
)


class EvaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = eva_vq_status_string(status) if _lib is not None else str(status)
        super().__init__(f"{fn} failed: {msg} ({status})")


class eva_vq_desc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("K", ctypes.c_int32), ("d", ctypes.c_int32),
                ("index_bits", ctypes.c_int32), ("codebook_rows", ctypes.c_int32),
                ("residual_group", ctypes.c_int32), ("hadamard_block", ctypes.c_int32),
                ("max_batch", ctypes.c_int32), ("out_dtype", ctypes.c_int),
                ("path", ctypes.c_int)]


class eva_quant_desc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("K", ctypes.c_int32), ("d", ctypes.c_int32),
                ("index_bits", ctypes.c_int32), ("codebook_rows", ctypes.c_int32),
                ("residual_group", ctypes.c_int32), ("hadamard_block", ctypes.c_int32),
                ("iters", ctypes.c_int32)]


class eva_vq_info(ctypes.Structure):
    _fields_ = [("stream_bytes", ctypes.c_int64), ("wi_bytes", ctypes.c_int64),
                ("sign_bytes", ctypes.c_int64), ("alpha_bytes", ctypes.c_int64),
                ("codebook_bytes", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
                ("slices", ctypes.c_int32), ("row_tiles", ctypes.c_int32),
                ("grid", ctypes.c_int32), ("kernels_per_run", ctypes.c_int32),
                ("path", ctypes.c_int32), ("sm_count", ctypes.c_int32),
                ("staged_units", ctypes.c_int32)]


class eva_rope_desc(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("norm", ctypes.c_int32),
                ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("scaling", ctypes.c_int32),
                ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float), ("theta", ctypes.c_double),
                ("factor", ctypes.c_double), ("original", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("magnitude", ctypes.c_double)]


class eva_kv_desc(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("max_seqs", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("cache_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int),
                ("window", ctypes.c_int32), ("softcap", ctypes.c_float), ("scale", ctypes.c_float)]


class eva_kv_info(ctypes.Structure):
    _fields_ = [("workspace_bytes", ctypes.c_int64), ("sm_count", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("grid", ctypes.c_int32), ("stages", ctypes.c_int32)]


_lib = None


def library_path() -> str:
    """The regular library; EVA_VQ_CHECKED=1 selects the device-check build,
    EVA_VQ_TIMELINE=1 the phase-timeline build, EVA_VQ_NAIVE=1 the build with
    the naive image layout (all three diagnostics only), and
    EVA_VQ_LIBRARY=<path> any other build of the same C ABI."""
    if os.environ.get("EVA_VQ_LIBRARY"):
        return os.environ["EVA_VQ_LIBRARY"]
    if os.environ.get("EVA_VQ_CHECKED") == "1":
        return _build.CHECKED_LIB
    if os.environ.get("EVA_VQ_TIMELINE") == "1":
        return _build.TIMELINE_LIB
    if os.environ.get("EVA_VQ_NAIVE") == "1":
        return _build.NAIVE_LIB
    return _build.LIB


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libeva_vq.so (building it with nvcc if it is absent)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        if not build_if_missing:
            raise RuntimeError(f"{path} is missing; build it with vector_quantized_weight_b200.build")
        _build.build(checked=path == _build.CHECKED_LIB, timeline=path == _build.TIMELINE_LIB,
                     naive=path == _build.NAIVE_LIB)
    lib = ctypes.CDLL(path)
    P, I32, H = ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p
    lib.eva_vq_linear_create.argtypes = [ctypes.POINTER(H), ctypes.POINTER(eva_vq_desc), P, P, P, P, P, P]
    lib.eva_vq_linear_run.argtypes = [H, P, I32, P, P]
    lib.eva_vq_linear_run_ex.argtypes = [H, P, I32, P, P, ctypes.c_uint32]
    lib.eva_vq_linear_run_noalloc.argtypes = [H, P, I32, P, P]
    lib.eva_vq_linear_run_group.argtypes = [P, P, P, I32, I32, P, ctypes.c_uint32]
    lib.eva_vq_linear_run_host.argtypes = [H, P, I32, P, P]
    lib.eva_vq_linear_destroy.argtypes = [H]
    lib.eva_vq_unpack_indices.argtypes = [H, P, P]
    lib.eva_vq_sync_status.argtypes = [H]
    lib.eva_vq_status_string.argtypes = [ctypes.c_int]
    lib.eva_vq_status_string.restype = ctypes.c_char_p
    lib.eva_vq_linear_info.argtypes = [H, ctypes.POINTER(eva_vq_info)]
    lib.eva_vq_device_check_record.argtypes = [H, P]
    lib.eva_vq_debug_inject_wait_timeout.argtypes = [H, I32]
    lib.eva_vq_debug_timeline.argtypes = [H, P, I32, ctypes.POINTER(I32)]
    I64 = ctypes.c_int64
    lib.eva_vq_quantize.argtypes = [ctypes.POINTER(eva_quant_desc), P, P, P, P, P, P, P, P, P, P]
    lib.eva_vq_kmeans_assign.argtypes = [P, I64, I32, P, I32, I64, P, P]
    lib.eva_vq_kmeans_update.argtypes = [P, I64, I32, P, I32, I64, P, P, P, P]
    lib.eva_vq_residual.argtypes = [P, I32, I32, P, I32, P, I32, I32, P, P, P]
    lib.eva_rope_create.argtypes = [ctypes.POINTER(H), ctypes.POINTER(eva_rope_desc), P, P, P]
    lib.eva_rope_run.argtypes = [H, P, I64, P, I64, P, I32, P, I64, P, I64, P]
    lib.eva_rope_destroy.argtypes = [H]
    lib.eva_kv_create.argtypes = [ctypes.POINTER(H), ctypes.POINTER(eva_kv_desc), P, P, P, P, P]
    lib.eva_kv_append.argtypes = [H, P, I64, P, I64, ctypes.c_int, P, P, P, I32, I32, P]
    lib.eva_kv_read.argtypes = [H, P, P, P, I32, I32, ctypes.c_int, P, P, P]
    lib.eva_kv_attend.argtypes = [H, P, I64, P, P, P, I32, I32, P, P, P]
    lib.eva_kv_sync_status.argtypes = [H]
    lib.eva_kv_debug_inject_wait_timeout.argtypes = [H, I32]
    lib.eva_kv_cache_info.argtypes = [H, ctypes.POINTER(eva_kv_info)]
    lib.eva_kv_destroy.argtypes = [H]
    for fn in ABI_FUNCTIONS:
        if fn != "eva_vq_status_string":
            getattr(lib, fn).restype = ctypes.c_int
    _lib = lib
    return lib


def _check(fn: str, rc: int):
    if rc != EVA_OK:
        raise EvaError(fn, rc)


# ------------------------------------------------------------ the C names

def eva_vq_status_string(status: int) -> str:
    return load().eva_vq_status_string(int(status)).decode()


def eva_vq_linear_create(desc: eva_vq_desc, wc: int, wi: int, signs: int | None, alpha: int | None,
                         hsign: int | None, stream: int | None) -> int:
    h = ctypes.c_void_p()
    rc = load().eva_vq_linear_create(ctypes.byref(h), ctypes.byref(desc), wc, wi, signs, alpha,
                                     hsign, stream)
    _check("eva_vq_linear_create", rc)
    return h.value


def eva_vq_linear_run(h: int, x: int, B: int, y: int, stream: int | None) -> None:
    _check("eva_vq_linear_run", load().eva_vq_linear_run(h, x, int(B), y, stream))


def eva_vq_linear_run_ex(h: int, x: int, B: int, y: int, stream: int | None, flags: int) -> None:
    _check("eva_vq_linear_run_ex", load().eva_vq_linear_run_ex(h, x, int(B), y, stream, int(flags)))


def eva_vq_linear_run_noalloc(h: int, x: int, B: int, y: int, stream: int | None) -> None:
    """eva_vq_linear_run without any device allocation: a rotated layer's
    scratch comes from the library's 4 MiB static device array (see the
    header for who needs this and the sharing rules)."""
    _check("eva_vq_linear_run_noalloc", load().eva_vq_linear_run_noalloc(h, x, int(B), y, stream))


def eva_vq_linear_run_group(hs: list, xs: list, ys: list, B: int, stream: int | None, flags: int = 0) -> None:
    """Independent layers in one launch where their shapes and formats allow
    (see the header); hs, xs, ys are lists of handles and device pointers."""
    n = len(hs)
    ha = (ctypes.c_void_p * n)(*hs)
    xa = (ctypes.c_void_p * n)(*xs)
    ya = (ctypes.c_void_p * n)(*ys)
    _check("eva_vq_linear_run_group", load().eva_vq_linear_run_group(ha, xa, ya, n, int(B), stream, int(flags)))


def eva_vq_linear_run_host(h: int, x_host: int, B: int, y_host: int, stream: int | None) -> None:
    _check("eva_vq_linear_run_host", load().eva_vq_linear_run_host(h, x_host, int(B), y_host, stream))


def eva_vq_linear_destroy(h: int | None) -> None:
    _check("eva_vq_linear_destroy", load().eva_vq_linear_destroy(h))


def eva_vq_unpack_indices(h: int, wi_out: int, stream: int | None) -> None:
    _check("eva_vq_unpack_indices", load().eva_vq_unpack_indices(h, wi_out, stream))


def eva_vq_sync_status(h: int) -> int:
    return int(load().eva_vq_sync_status(h))


def eva_vq_debug_inject_wait_timeout(h: int, rounds: int) -> None:
    _check("eva_vq_debug_inject_wait_timeout", load().eva_vq_debug_inject_wait_timeout(h, rounds))


def eva_vq_device_check_record(h: int) -> list:
    rec = (ctypes.c_int32 * 8)()
    _check("eva_vq_device_check_record", load().eva_vq_device_check_record(h, rec))
    return list(rec)


def eva_vq_debug_timeline(h: int, max_entries: int = 1 << 16) -> list:
    buf = (ctypes.c_uint64 * max_entries)()
    n = ctypes.c_int32()
    _check("eva_vq_debug_timeline", load().eva_vq_debug_timeline(h, buf, max_entries, ctypes.byref(n)))
    return list(buf[:n.value])


def eva_vq_linear_info(h: int) -> eva_vq_info:
    info = eva_vq_info()
    _check("eva_vq_linear_info", load().eva_vq_linear_info(h, ctypes.byref(info)))
    return info


def eva_vq_quantize(desc: eva_quant_desc, w: int, hsign: int | None, init_index: int, wc_out: int, wi_out: int,
                    signs_out: int | None, alpha_out: int | None, wrot_out: int | None, cent_out: int | None,
                    stream: int | None) -> None:
    _check("eva_vq_quantize", load().eva_vq_quantize(ctypes.byref(desc), w, hsign, init_index, wc_out, wi_out,
                                                     signs_out, alpha_out, wrot_out, cent_out, stream))


def eva_vq_kmeans_assign(v: int, M: int, d: int, centroids: int, ncent: int, vecs_per_cb: int, idx_out: int,
                         stream: int | None) -> None:
    _check("eva_vq_kmeans_assign", load().eva_vq_kmeans_assign(v, int(M), int(d), centroids, int(ncent),
                                                               int(vecs_per_cb), idx_out, stream))


def eva_vq_kmeans_update(v: int, M: int, d: int, idx: int, ncent: int, vecs_per_cb: int, old: int, new_out: int,
                         counts_out: int | None, stream: int | None) -> None:
    _check("eva_vq_kmeans_update", load().eva_vq_kmeans_update(v, int(M), int(d), idx, int(ncent),
                                                               int(vecs_per_cb), old, new_out, counts_out, stream))


def eva_vq_residual(wrot: int, N: int, K: int, wc: int, ncent: int, wi: int, codebook_rows: int, group: int,
                    signs_out: int, alpha_out: int, stream: int | None) -> None:
    _check("eva_vq_residual", load().eva_vq_residual(wrot, int(N), int(K), wc, int(ncent), wi,
                                                     int(codebook_rows), int(group), signs_out, alpha_out, stream))


def eva_rope_create(desc: eva_rope_desc, q_weight: int | None, k_weight: int | None, stream: int | None) -> int:
    h = ctypes.c_void_p()
    _check("eva_rope_create", load().eva_rope_create(ctypes.byref(h), ctypes.byref(desc), q_weight, k_weight, stream))
    return h.value


def eva_rope_run(h: int, q: int | None, ldq: int, k: int | None, ldk: int, positions: int | None, T: int,
                 q_out: int | None, ldqo: int, k_out: int | None, ldko: int, stream: int | None) -> None:
    _check("eva_rope_run", load().eva_rope_run(h, q, ldq, k, ldk, positions, T, q_out, ldqo, k_out, ldko, stream))


def eva_rope_destroy(h: int | None) -> None:
    _check("eva_rope_destroy", load().eva_rope_destroy(h))


def eva_kv_create(desc: eva_kv_desc, k_pages: int, v_pages: int, k_scale: int, v_scale: int,
                  stream: int | None) -> int:
    h = ctypes.c_void_p()
    _check("eva_kv_create", load().eva_kv_create(ctypes.byref(h), ctypes.byref(desc), k_pages, v_pages, k_scale,
                                                 v_scale, stream))
    return h.value


def eva_kv_append(h: int, k: int, ldk: int, v: int, ldv: int, in_dtype: int, starts: int, lens: int,
                  page_table: int, B: int, T: int, stream: int | None) -> None:
    _check("eva_kv_append", load().eva_kv_append(h, k, ldk, v, ldv, in_dtype, starts, lens, page_table, B, T, stream))


def eva_kv_read(h: int, starts: int, begins: int, page_table: int, B: int, T: int, out_dtype: int,
                k_out: int | None, v_out: int | None, stream: int | None) -> None:
    _check("eva_kv_read", load().eva_kv_read(h, starts, begins, page_table, B, T, out_dtype, k_out, v_out, stream))


def eva_kv_attend(h: int, q: int, ldq: int, starts: int, lens: int, page_table: int, B: int, T: int, out: int,
                  lse: int | None, stream: int | None) -> None:
    _check("eva_kv_attend", load().eva_kv_attend(h, q, ldq, starts, lens, page_table, B, T, out, lse, stream))


def eva_kv_sync_status(h: int) -> int:
    return int(load().eva_kv_sync_status(h))


def eva_kv_debug_inject_wait_timeout(h: int, rounds: int) -> None:
    _check("eva_kv_debug_inject_wait_timeout", load().eva_kv_debug_inject_wait_timeout(h, rounds))


def eva_kv_cache_info(h: int) -> eva_kv_info:
    info = eva_kv_info()
    _check("eva_kv_cache_info", load().eva_kv_cache_info(h, ctypes.byref(info)))
    return info


def eva_kv_destroy(h: int | None) -> None:
    _check("eva_kv_destroy", load().eva_kv_destroy(h))


# ------------------------------------------------------- torch convenience

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


class VQLinear:
    """One layer held on the device.  Weights are torch CUDA tensors in the
    canonical layouts (see synth.py); they are copied and repacked by the
    library, so the caller may drop them after construction."""

    def __init__(self, wc, wi, *, signs=None, alpha=None, hsign=None, codebook_rows=0,
                 residual_group=0, hadamard_block=0, max_batch=1, out_dtype="float16",
                 path=EVA_PATH_AUTO, index_bits=8, stream=None):
        import torch
        N, J = wi.shape
        if index_bits == 4:          # two indices per byte
            J *= 2
        self.index_bits = int(index_bits)
        self.N, self.K = int(N), int(J) * 4
        self.out_dtype = torch.float32 if out_dtype in ("float32", torch.float32) else torch.float16
        self.max_batch = int(max_batch)
        self.desc = eva_vq_desc(self.N, self.K, 4, self.index_bits, int(codebook_rows), int(residual_group),
                                int(hadamard_block), self.max_batch,
                                EVA_F32 if self.out_dtype == torch.float32 else EVA_F16, int(path))
        tensors = [wc, wi, signs, alpha, hsign]
        for t in tensors:
            if t is not None and (not t.is_cuda or not t.is_contiguous()):
                raise ValueError("weights must be contiguous CUDA tensors")
        self.handle = None
        self.handle = eva_vq_linear_create(self.desc, _ptr(wc), _ptr(wi), _ptr(signs), _ptr(alpha),
                                           _ptr(hsign), _stream_handle(stream))

    def __call__(self, x, out=None, stream=None, independent=False):
        """y = layer(x) on `stream`.  independent=True passes EVA_RUN_INDEPENDENT:
        the caller promises the preceding kernel on the stream neither writes x
        nor touches y; the call then overlaps it and takes the overlap grid."""
        import torch
        if x.dtype != torch.float16 or not x.is_cuda or not x.is_contiguous():
            raise ValueError("x must be a contiguous CUDA float16 tensor [B, K]")
        x2 = x.view(-1, self.K)
        B = x2.shape[0]
        y = out if out is not None else torch.empty((B, self.N), dtype=self.out_dtype, device=x.device)
        eva_vq_linear_run_ex(self.handle, _ptr(x2), B, _ptr(y), _stream_handle(stream),
                             EVA_RUN_INDEPENDENT if independent else 0)
        return y

    def run_host(self, x_host, y_host, stream=None):
        """Host buffers in and out (torch CPU tensors, ideally pinned)."""
        B = x_host.shape[0]
        eva_vq_linear_run_host(self.handle, _ptr(x_host), B, _ptr(y_host), _stream_handle(stream))
        return y_host

    def unpack_indices(self, stream=None):
        """The canonical index matrix back: [N][K/4], or [N][K/8] packed for 4-bit indices."""
        import torch
        cols = self.K // 4 if self.index_bits == 8 else self.K // 8
        out = torch.empty((self.N, cols), dtype=torch.uint8, device="cuda")
        eva_vq_unpack_indices(self.handle, _ptr(out), _stream_handle(stream))
        return out

    def info(self) -> eva_vq_info:
        return eva_vq_linear_info(self.handle)

    def close(self):
        if self.handle is not None:
            eva_vq_linear_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def from_layer(layer, *, max_batch=1, out_dtype="float16", path=EVA_PATH_AUTO, device="cuda"):
    """Build a VQLinear from a synth.LayerData (numpy arrays)."""
    import torch

    def dev(a):
        return None if a is None else torch.from_numpy(a).to(device)
    s = layer.shape
    return VQLinear(dev(layer.wc), dev(layer.wi), signs=dev(layer.signs), alpha=dev(layer.alpha),
                    hsign=dev(layer.hsign), codebook_rows=s.codebook_rows,
                    residual_group=s.residual_group, hadamard_block=s.hadamard_block,
                    max_batch=max_batch, out_dtype=out_dtype, path=path, index_bits=s.index_bits)


def quantize(w, init_index, iters: int, *, hsign=None, hadamard_block: int = 0, codebook_rows: int = 0,
             residual_group: int = 128, index_bits: int = 8, keep_wrot: bool = False, keep_centroids: bool = False,
             stream=None) -> dict:
    """The offline quantizer on the GPU (eva_vq_quantize).  w: CUDA fp16
    [N][K]; init_index: CUDA int32 [G][2^index_bits] starting blocks (see the
    header).  Returns CUDA tensors wc, wi (and signs, alpha with a residual;
    wrot, centroids on request) ready for VQLinear."""
    import torch
    N, K = w.shape
    dev = w.device
    G = N // codebook_rows if codebook_rows else 1
    ncent = 1 << index_bits
    # 4-bit pointers come packed two per byte (the layout VQLinear(index_bits=4) takes)
    out = {"wc": torch.empty((G, ncent, 4), dtype=torch.float16, device=dev),
           "wi": torch.empty((N, K // 8 if index_bits == 4 else K // 4), dtype=torch.uint8, device=dev)}
    if residual_group:
        out["signs"] = torch.empty((N, K // 8), dtype=torch.uint8, device=dev)
        out["alpha"] = torch.empty((N, K // residual_group), dtype=torch.float16, device=dev)
    if keep_wrot:
        out["wrot"] = torch.empty((N, K), dtype=torch.float32, device=dev)
    if keep_centroids:
        out["centroids"] = torch.empty((G, ncent, 4), dtype=torch.float32, device=dev)
    desc = eva_quant_desc(N, K, 4, index_bits, codebook_rows, residual_group, hadamard_block, iters)
    eva_vq_quantize(desc, _ptr(w.contiguous()), _ptr(hsign), _ptr(init_index.contiguous()), _ptr(out["wc"]),
                    _ptr(out["wi"]), _ptr(out.get("signs")), _ptr(out.get("alpha")), _ptr(out.get("wrot")),
                    _ptr(out.get("centroids")), _stream_handle(stream))
    return out


def run_group(layers, xs, outs=None, stream=None, independent=False):
    """Run VQLinear layers on their inputs (CUDA fp16 [B][K] tensors, one B)
    as one grouped call; returns the outputs."""
    import torch
    B = xs[0].shape[0]
    if outs is None:
        outs = [torch.empty((B, l.N), dtype=l.out_dtype, device=x.device) for l, x in zip(layers, xs)]
    eva_vq_linear_run_group([l.handle for l in layers], [x.data_ptr() for x in xs], [y.data_ptr() for y in outs],
                            B, _stream_handle(stream), EVA_RUN_INDEPENDENT if independent else 0)
    return outs


# ------------------------------- between a block's q, k, v layers and its o layer

_DTYPES = {}      # torch dtype or its name -> (torch dtype, eva_dtype_t); filled on first use
_INT32 = None


def _dtype(t):
    global _INT32
    if not _DTYPES:
        import torch
        _INT32 = torch.int32
        for d, code in ((torch.float16, EVA_F16), (torch.float32, EVA_F32)):
            _DTYPES[d] = _DTYPES[str(d).removeprefix("torch.")] = (d, code)
    if t not in _DTYPES:
        raise ValueError(f"dtype must be float16 or float32, not {t}")
    return _DTYPES[t]


def _rows(name, x, heads, head_dim, dtype, device):
    """Checks a [T][heads][head_dim] (or [T][heads * head_dim]) tensor whose rows may lie apart; (T, row stride)."""
    shape, stride = x.shape, x.stride()
    if x.dtype != dtype or x.device != device:
        raise ValueError(f"{name} must be a {dtype} tensor on {device}, not {x.dtype} on {x.device}")
    if len(shape) == 3:
        ok = shape[1] == heads and shape[2] == head_dim and (
            (stride[2] == 1 or head_dim == 1) and (stride[1] == head_dim or heads == 1) or 0 in shape)
    else:
        ok = len(shape) == 2 and shape[1] == heads * head_dim and (stride[1] == 1 or shape[1] <= 1 or 0 in shape)
    if not ok:
        raise ValueError(f"{name} must be [T][{heads}][{head_dim}] with contiguous rows, not {tuple(shape)} "
                         f"with strides {stride}")
    return shape[0], (stride[0] if shape[0] > 1 else heads * head_dim)


def _indices(name, x, shape, device):
    if x.dtype != _INT32 or x.device != device or x.shape != shape or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {tuple(shape)} on {device}, "
                         f"not {x.dtype} {tuple(x.shape)} on {x.device}")


def _cuda_device(device):
    """A CUDA device with its number: the current one for None and for "cuda"."""
    import torch
    d = torch.device("cuda" if device is None else device)
    if d.type != "cuda":
        raise ValueError(f"the device must be a CUDA device, not {d}")
    return d if d.index is not None else torch.device("cuda", torch.cuda.current_device())


class _OnDevice:
    """A handle on one device: its stream, and outputs that belong to the stream of the call.  A decode step's calls
    are a few microseconds of device time, so what a call needs of torch is looked up once."""

    def _prepare(self):
        import torch
        self._raw_stream = torch._C._cuda_getCurrentRawStream
        self._empty_like, self._half, self._single = torch.empty_like, torch.float16, torch.float32
        self._like = {d: torch.empty(0, dtype=d, device=self.device) for d in (torch.float16, torch.float32)}

    def _stream(self, stream):
        if stream is None:
            return self._raw_stream(self.device.index)
        if stream.device != self.device:
            raise ValueError(f"the stream is on {stream.device}, the handle on {self.device}")
        return stream.cuda_stream

    def _empty(self, shape, dtype, stream, x=None):
        """An output of the call's stream; x: an input that may have its shape and type (copying those is cheapest)."""
        if stream is None:
            if x is not None and x.dtype == dtype and x.shape == shape and x.is_contiguous():
                return self._empty_like(x)
            return self._like[dtype].new_empty(shape)
        import torch
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class HeadRope(_OnDevice):
    """Rotary positions for a block's queries and keys, with the per-head RMS norm in the same pass (norm=True).

    layout: "half" (dimensions i and i + rotary_dim / 2 turn together) or "interleaved" (2i and 2i + 1);
    rotary_dim (default head_dim): the first dimensions of a head, the others pass through.
    scaling: None or {"type": "linear" | "ntk" | "yarn" | "bands", "factor": f, ...}; yarn takes "original", "low"
    (1) and "high" (32), bands "original", "low" (1) and "high" (4); "magnitude" replaces the type's own (see the
    header for the formulas).  q_weight, k_weight: CUDA fp16 [head_dim], copied; weight_offset is added to them."""

    _SCALING = {"linear": EVA_ROPE_LINEAR, "ntk": EVA_ROPE_NTK, "yarn": EVA_ROPE_YARN, "bands": EVA_ROPE_BANDS}

    def __init__(self, q_heads, kv_heads, head_dim, *, rotary_dim=None, layout="half", theta=10000.0, scaling=None,
                 norm=False, q_weight=None, k_weight=None, eps=1e-6, weight_offset=0.0, in_dtype="float16",
                 out_dtype="float16", device=None, stream=None):
        import torch
        self.handle = None
        if layout not in ("half", "interleaved"):
            raise ValueError(f"layout must be 'half' or 'interleaved', not {layout!r}")
        self.q_heads, self.kv_heads, self.head_dim = int(q_heads), int(kv_heads), int(head_dim)
        self.rotary_dim = self.head_dim if rotary_dim is None else int(rotary_dim)
        self.in_dtype, code_in = _dtype(in_dtype)
        self.out_dtype, code_out = _dtype(out_dtype)
        how = dict(scaling or {"type": "none"})
        kind = how.pop("type", None)
        if kind != "none" and kind not in self._SCALING:
            raise ValueError(f"scaling type must be one of {sorted(self._SCALING)}, not {kind!r}")
        unknown = set(how) - {"factor", "original", "low", "high", "magnitude"}
        if unknown:
            raise ValueError(f"unknown scaling entries {sorted(unknown)}")
        self.device = _cuda_device(device)
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is not None and (w.dtype != torch.float16 or w.device != self.device or
                                  tuple(w.shape) != (self.head_dim,) or not w.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous float16 tensor ({self.head_dim},) on {self.device}")
        self.desc = eva_rope_desc(self.q_heads, self.kv_heads, self.head_dim, self.rotary_dim,
                                  EVA_ROPE_HALF if layout == "half" else EVA_ROPE_INTERLEAVED, int(bool(norm)), code_in,
                                  code_out, self._SCALING.get(kind, EVA_ROPE_UNSCALED), float(eps), float(weight_offset),
                                  float(theta), float(how.get("factor", 1.0)), float(how.get("original", 0.0)),
                                  float(how.get("low", 1.0)), float(how.get("high", 4.0 if kind == "bands" else 32.0)),
                                  float(how.get("magnitude", 0.0)))
        self._prepare()
        with torch.cuda.device(self.device):
            self.handle = eva_rope_create(self.desc, _ptr(q_weight), _ptr(k_weight), self._stream(stream))
        self._run = load().eva_rope_run

    def __call__(self, q, k, positions, q_out=None, k_out=None, stream=None):
        """(q_out, k_out) of q [T][q_heads][head_dim], k [T][kv_heads][head_dim] (rows may lie apart, as columns of
        a fused projection) and positions int32 [T].  q_out=q, k_out=k write in place when the types are equal."""
        Hq, Hk, D, dev = self.q_heads, self.kv_heads, self.head_dim, self.device
        T, ldq = _rows("q", q, Hq, D, self.in_dtype, dev)
        Tk, ldk = _rows("k", k, Hk, D, self.in_dtype, dev)
        if T != Tk:
            raise ValueError(f"q has {T} rows, k has {Tk}")
        if positions is not None:
            _indices("positions", positions, (T,), dev)
        elif self.rotary_dim:
            raise ValueError("positions are needed")
        if q_out is None:
            q_out, ldqo = self._empty((T, Hq, D), self.out_dtype, stream, q), Hq * D
        else:
            To, ldqo = _rows("q_out", q_out, Hq, D, self.out_dtype, dev)
            if To != T:
                raise ValueError(f"q_out has {To} rows, q has {T}")
        if k_out is None:
            k_out, ldko = self._empty((T, Hk, D), self.out_dtype, stream, k), Hk * D
        else:
            To, ldko = _rows("k_out", k_out, Hk, D, self.out_dtype, dev)
            if To != T:
                raise ValueError(f"k_out has {To} rows, k has {T}")
        rc = self._run(self.handle, q.data_ptr(), ldq, k.data_ptr(), ldk,
                       None if positions is None else positions.data_ptr(), T, q_out.data_ptr(), ldqo,
                       k_out.data_ptr(), ldko, self._stream(stream))
        if rc:
            _check("eva_rope_run", rc)
        return q_out, k_out

    def close(self):
        if self.handle is not None:
            eva_rope_destroy(self.handle)
            self.handle = None


class KVCache(_OnDevice):
    """A paged 8-bit cache of keys and values and the attention over it.

    k, v: codes [num_pages][kv_heads][page_size][head_dim] (int8, or float8_e4m3fn), k_scale, v_scale: float32
    [num_pages][kv_heads]; made here (zeros) when not given.  max_seqs and max_pages bound a call's sequences
    and the page table's columns.  One handle must not attend on two streams at once; clone(), another handle over
    the same buffers, may."""

    def __init__(self, q_heads, kv_heads, head_dim, *, num_pages, max_seqs, max_pages, page_size=64, dtype="int8",
                 window=0, softcap=0.0, scale=None, out_dtype="float16", k=None, v=None, k_scale=None, v_scale=None,
                 device=None, stream=None):
        import torch
        self.handle = None
        if dtype not in ("int8", "e4m3"):
            raise ValueError(f"dtype must be 'int8' or 'e4m3', not {dtype!r}")
        if scale is not None and not scale > 0:
            raise ValueError("scale must be positive")
        self._args = dict(num_pages=num_pages, max_seqs=max_seqs, max_pages=max_pages, page_size=page_size, dtype=dtype,
                          window=window, softcap=softcap, scale=scale, out_dtype=out_dtype)
        self.q_heads, self.kv_heads, self.head_dim = int(q_heads), int(kv_heads), int(head_dim)
        self.max_seqs, self.max_pages = int(max_seqs), int(max_pages)
        self.out_dtype, code_out = _dtype(out_dtype)
        given = [t for t in (k, v, k_scale, v_scale) if t is not None]
        self.device = _cuda_device(given[0].device if device is None and given else device)
        code_type = torch.int8 if dtype == "int8" else torch.float8_e4m3fn
        tile = (int(num_pages), self.kv_heads)
        made = []
        for name, t, shape, kind in (("k", k, tile + (int(page_size), self.head_dim), code_type),
                                     ("v", v, tile + (int(page_size), self.head_dim), code_type),
                                     ("k_scale", k_scale, tile, torch.float32), ("v_scale", v_scale, tile, torch.float32)):
            if t is None:                      # on the stream that __init__ waits for: the first call may be on any other
                with torch.cuda.stream(stream):
                    t = torch.zeros(shape, dtype=kind, device=self.device)
            elif t.dtype != kind or t.device != self.device or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {kind} tensor {shape} on {self.device}")
            made.append(t)
        self.k, self.v, self.k_scale, self.v_scale = made
        self.desc = eva_kv_desc(self.q_heads, self.kv_heads, self.head_dim, int(page_size), int(num_pages), self.max_seqs,
                                self.max_pages, EVA_CACHE_INT8 if dtype == "int8" else EVA_CACHE_E4M3, code_out,
                                int(window), float(softcap), float(scale or 0.0))
        self._prepare()
        with torch.cuda.device(self.device):
            self.handle = eva_kv_create(self.desc, *map(_ptr, made), self._stream(stream))
        lib = load()
        self._append, self._attend, self._read = lib.eva_kv_append, lib.eva_kv_attend, lib.eva_kv_read

    def clone(self, **changes):
        """Another handle (its own workspace) over the same buffers; changes: window, softcap, scale, out_dtype,
        max_seqs, max_pages."""
        return KVCache(self.q_heads, self.kv_heads, self.head_dim, **{**self._args, **changes}, k=self.k, v=self.v,
                       k_scale=self.k_scale, v_scale=self.v_scale)

    def _sequences(self, starts, lens, page_table, what="lens"):
        dev = self.device
        B = lens.shape[0]
        if not 1 <= B <= self.max_seqs:
            raise ValueError(f"{B} sequences: 1 to {self.max_seqs} were planned for")
        _indices(what, lens, (B,), dev)
        _indices("starts", starts, (B + 1,), dev)
        _indices("page_table", page_table, (B, self.max_pages), dev)
        return B

    def append(self, k, v, starts, lens, page_table, stream=None):
        """Write the keys and values of new tokens: k, v [T][kv_heads][head_dim], fp16 or fp32 (rows may lie apart);
        starts int32 [B + 1] (rows of each sequence), lens int32 [B] (lengths with them), page_table int32
        [B][max_pages]."""
        B = self._sequences(starts, lens, page_table)
        dtype, code = _dtype(k.dtype)
        T, ldk = _rows("k", k, self.kv_heads, self.head_dim, dtype, self.device)
        Tv, ldv = _rows("v", v, self.kv_heads, self.head_dim, dtype, self.device)
        if T != Tv:
            raise ValueError(f"k has {T} rows, v has {Tv}")
        rc = self._append(self.handle, k.data_ptr(), ldk, v.data_ptr(), ldv, code, starts.data_ptr(), lens.data_ptr(),
                          page_table.data_ptr(), B, T, self._stream(stream))
        if rc:
            _check("eva_kv_append", rc)

    def attend(self, q, starts, lens, page_table, out=None, lse=None, stream=None):
        """Causal attention of q fp16 [T][q_heads][head_dim] over the cache -> [T][q_heads][head_dim].  Rows
        behind starts[B] are not written: give `out` where they matter.  lse: optional float32 [T][q_heads]."""
        B = self._sequences(starts, lens, page_table)
        Hq, D, dev = self.q_heads, self.head_dim, self.device
        T, ldq = _rows("q", q, Hq, D, self._half, dev)
        if out is None:
            out = self._empty((T, Hq, D), self.out_dtype, stream, q)
        elif _rows("out", out, Hq, D, self.out_dtype, dev) != (T, Hq * D):
            raise ValueError(f"out must be a contiguous [{T}][{Hq}][{D}] tensor")
        if lse is not None and (lse.dtype != self._single or lse.device != dev or lse.shape != (T, Hq) or
                                not lse.is_contiguous()):
            raise ValueError(f"lse must be a contiguous float32 tensor ({T}, {Hq}) on {dev}")
        rc = self._attend(self.handle, q.data_ptr(), ldq, starts.data_ptr(), lens.data_ptr(), page_table.data_ptr(), B, T,
                          out.data_ptr(), None if lse is None else lse.data_ptr(), self._stream(stream))
        if rc:
            _check("eva_kv_attend", rc)
        return out

    def read(self, starts, begins, page_table, rows, k_out=None, v_out=None, dtype="float16", stream=None):
        """The stored values back: (k, v) [rows][kv_heads][head_dim], where rows starts[b] .. hold the tokens at
        positions begins[b] .. of sequence b."""
        B = self._sequences(starts, begins, page_table, "begins")
        dtype, code = _dtype(dtype)
        shape = (int(rows), self.kv_heads, self.head_dim)
        outs = []
        for name, t in (("k_out", k_out), ("v_out", v_out)):
            if t is None:
                t = self._empty(shape, dtype, stream)
            elif t.dtype != dtype or t.device != self.device or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dtype} tensor {shape} on {self.device}")
            outs.append(t)
        rc = self._read(self.handle, starts.data_ptr(), begins.data_ptr(), page_table.data_ptr(), B, shape[0], code,
                        outs[0].data_ptr(), outs[1].data_ptr(), self._stream(stream))
        if rc:
            _check("eva_kv_read", rc)
        return tuple(outs)

    def status(self) -> int:
        """Waits for the device; EVA_OK, EVA_ERR_BAD_INDEX or EVA_ERR_DEVICE_TIMEOUT since the last call of this."""
        return eva_kv_sync_status(self.handle)

    def info(self) -> eva_kv_info:
        return eva_kv_cache_info(self.handle)

    def close(self):
        if self.handle is not None:
            eva_kv_destroy(self.handle)
            self.handle = None
