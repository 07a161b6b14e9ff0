"""ctypes binding of ``libnspack.so`` (declared in ``include/nspack.h`` and, for
the training operators, ``include/nstrain.h``).

Argument marshalling only: every step of the packing path and every operator
runs in the library's CUDA kernels.  There is no fallback: if the library is missing or
fails to load, importing this module raises.
"""
from __future__ import annotations

import ctypes as C
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libnspack.so")

NS_OK = 0
NS_ERR_INVALID_ARG = -1
NS_ERR_CUDA = -2
NS_ERR_OOM = -3
NS_ERR_EXHAUSTED = -4
NS_ERR_HORIZON = -5
NS_ERR_BAD_INPUT = -6
NS_ERR_DEVICE = -7
NS_PACK_DRAIN = 1
NS_PACK_HELDOUT = 2
NS_PACK_SHUFFLE_ROWS = 4
NS_PACK_WRAP = 8
NS_PACK_HOST_CORPUS = 16
NS_PACK_ORDERED_FREE = 32
NS_DISPATCH_MAX_EXPERTS = 1024
NS_F32 = 0
NS_BF16 = 1
NS_F16 = 2
NS_SCAN_TILE = 32
NS_MAX_T = 1 << 24
NS_MAX_TOKENS = 1 << 47

ns_alloc_fn = C.CFUNCTYPE(C.c_void_p, C.c_size_t, C.c_void_p)
ns_free_fn = C.CFUNCTYPE(None, C.c_void_p, C.c_void_p)


class ns_pack_config(C.Structure):
    _fields_ = [
        ("tokens", C.c_void_p),
        ("n_tokens", C.c_uint64),
        ("doc_offsets", C.c_void_p),
        ("loss_start", C.c_void_p),
        ("n_docs", C.c_uint32),
        ("n_sources", C.c_uint32),
        ("n_streams", C.c_uint32),
        ("T", C.c_uint32),
        ("stream_doc_begin", C.c_void_p),
        ("stream_source", C.c_void_p),
        ("source_weight", C.c_void_p),
        ("stream_weight", C.c_void_p),
        ("source_heldout_bp", C.c_void_p),
        ("seed", C.c_uint64),
        ("hash_key", C.c_uint64),
        ("B", C.c_uint32),
        ("max_steps", C.c_uint32),
        ("flags", C.c_uint32),
        ("pad_id", C.c_int32),
        ("window_segment", C.c_uint32),
        ("n_pieces", C.c_uint32),
        ("piece_begin", C.c_void_p),
        ("piece_B", C.c_void_p),
        ("piece_source_weight", C.c_void_p),
        ("piece_stream_weight", C.c_void_p),
        ("len_bucket", C.c_uint32),
        ("cuda_stream", C.c_void_p),
        ("alloc", ns_alloc_fn),
        ("free", ns_free_fn),
        ("alloc_user", C.c_void_p),
    ]


class ns_pack_out(C.Structure):
    _fields_ = [
        ("tokens", C.c_void_p),
        ("pos", C.c_void_p),
        ("doc", C.c_void_p),
        ("mask", C.c_void_p),
        ("row_fp", C.c_void_p),
        ("row_learned", C.c_void_p),
        ("row_len", C.c_void_p),
    ]


class ns_pack_info_t(C.Structure):
    _fields_ = [
        ("valid_steps", C.c_uint32),
        ("max_steps", C.c_uint32),
        ("n_streams", C.c_uint32),
        ("T", C.c_uint32),
        ("B", C.c_uint32),
        ("levels", C.c_uint32),
        ("order_digest", C.c_uint64),
        ("n_pieces", C.c_uint64),
        ("table_bytes", C.c_uint64),
        ("init_launches", C.c_uint32),
        ("init_passes", C.c_uint32),
        ("host_bytes", C.c_uint64),
        ("hashed_tokens", C.c_uint64),
        ("hashed_docs", C.c_uint64),
        ("hash_ns", C.c_uint64),
    ]


def _fits(name: str, v: int) -> None:
    """Refuse a size that is not one of 32 bits: ctypes would pass what is left of it."""
    if v >> 32:
        raise NsPackError(NS_ERR_INVALID_ARG, f"{name}: {v}, expected 0 to 2**32 - 1")


class _Sized(C.Structure):
    """A structure with sizes of 32 bits, checked where all its fields are given in order."""

    def __init_subclass__(cls):
        super().__init_subclass__()
        cls._sizes = [(i, f[0]) for i, f in enumerate(cls._fields_) if f[1] is C.c_uint32]

    def __init__(self, *args):
        if args:
            for i, name in self._sizes:
                _fits(name, args[i])
        super().__init__(*args)


class ns_scan_inputs(_Sized):
    _fields_ = [
        ("z", C.c_void_p),
        ("f", C.c_void_p),
        ("z_row", C.c_int64),
        ("z_time", C.c_int64),
        ("f_row", C.c_int64),
        ("f_time", C.c_int64),
        ("bias", C.c_void_p),
        ("pos", C.c_void_p),
        ("doc", C.c_void_p),
        ("B", C.c_uint32),
        ("T", C.c_uint32),
        ("D", C.c_uint32),
        ("dtype", C.c_int32),
    ]


class ns_distill_inputs(_Sized):
    _fields_ = [
        ("logits", C.c_void_p),
        ("logits_row", C.c_int64),
        ("top_logits", C.c_void_p),
        ("top_ids", C.c_void_p),
        ("teacher_lse", C.c_void_p),
        ("mask", C.c_void_p),
        ("weight", C.c_void_p),
        ("N", C.c_uint32),
        ("V", C.c_uint32),
        ("K", C.c_uint32),
        ("dtype", C.c_int32),
        ("top_dtype", C.c_int32),
        ("ids_64", C.c_int32),
        ("temperature", C.c_float),
    ]


class ns_route_inputs(_Sized):
    _fields_ = [
        ("logits", C.c_void_p),
        ("logits_row", C.c_int64),
        ("doc", C.c_void_p),
        ("N", C.c_uint32),
        ("E", C.c_uint32),
        ("k", C.c_uint32),
        ("dtype", C.c_int32),
        ("normalize", C.c_int32),
    ]


class ns_embed_inputs(_Sized):
    _fields_ = [
        ("tokens", C.c_void_p),
        ("doc", C.c_void_p),
        ("N", C.c_uint32),
        ("V", C.c_uint32),
        ("D", C.c_uint32),
        ("table_dtype", C.c_int32),
        ("dtype", C.c_int32),
        ("ids_64", C.c_int32),
        ("scale", C.c_float),
    ]


class ns_norm_inputs(_Sized):
    _fields_ = [
        ("x", C.c_void_p),
        ("x_row", C.c_int64),
        ("weight", C.c_void_p),
        ("bias", C.c_void_p),
        ("doc", C.c_void_p),
        ("N", C.c_uint32),
        ("D", C.c_uint32),
        ("dtype", C.c_int32),
        ("weight_dtype", C.c_int32),
        ("eps", C.c_float),
    ]


class ns_expert_sizes(_Sized):
    _fields_ = [
        ("N", C.c_uint32),
        ("k", C.c_uint32),
        ("E", C.c_uint32),
        ("D", C.c_uint32),
        ("dtype", C.c_int32),
    ]


def _packer(layout: str, of):
    """The bytes of a structure from its fields in order: as good an argument as the structure,
    and made in a tenth of the time.  Sizes that 32 bits do not hold are refused."""
    pack = struct.Struct(layout).pack
    assert struct.calcsize(layout) == C.sizeof(of)

    def packed(*fields) -> bytes:
        try:
            return pack(*fields)
        except (struct.error, OverflowError) as e:
            raise NsPackError(NS_ERR_INVALID_ARG, f"{of.__name__}{fields}: {e}") from None

    return packed


pack_embed = _packer("@PPIIIiiif4x", ns_embed_inputs)
pack_norm = _packer("@PqPPPIIiif4x", ns_norm_inputs)
pack_experts = _packer("@IIIIi", ns_expert_sizes)


def _argument(inputs):
    """A structure, or the bytes of one, as an argument."""
    return inputs if type(inputs) is bytes else C.byref(inputs)


# Every symbol the headers declare, for the load check.
SYMBOLS = ("ns_pack_init", "ns_pack_step", "ns_pack_fingerprint", "ns_pack_batch_fp",
           "ns_pack_step_learned", "ns_pack_info", "ns_pack_stream_windows",
           "ns_pack_quota_table", "ns_pack_check", "ns_pack_free", "ns_pack_strerror",
           "ns_pack_quota_noalloc", "ns_pack_probe_hash_terms",
           "ns_scan_forward", "ns_scan_workspace", "ns_scan_backward", "ns_distill",
           "ns_route_workspace", "ns_route_forward", "ns_route_backward",
           "ns_embed_forward", "ns_embed_workspace", "ns_embed_backward",
           "ns_norm_forward", "ns_norm_workspace", "ns_norm_backward",
           "ns_norm_probe_forward", "ns_norm_probe_backward",
           "ns_dispatch_workspace", "ns_dispatch", "ns_combine", "ns_combine_backward")


def _load() -> C.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python -c \"import __graft_entry__ as g; g.build()\"` "
            "(there is no CPU fallback)")
    L = C.CDLL(LIB_PATH)
    vp, u32, u64, i32 = C.c_void_p, C.c_uint32, C.c_uint64, C.c_int
    L.ns_pack_init.restype = i32
    L.ns_pack_init.argtypes = [C.POINTER(ns_pack_config), C.POINTER(vp)]
    L.ns_pack_step.restype = i32
    L.ns_pack_step.argtypes = [vp, u32, u32, u32, u32, C.POINTER(ns_pack_out), vp]
    L.ns_pack_fingerprint.restype = i32
    L.ns_pack_fingerprint.argtypes = [vp, vp, u32, C.POINTER(C.c_uint64), vp]
    L.ns_pack_batch_fp.restype = i32
    L.ns_pack_batch_fp.argtypes = [vp, vp, u32, u32, vp, vp]
    L.ns_pack_info.restype = i32
    L.ns_pack_info.argtypes = [vp, C.POINTER(ns_pack_info_t)]
    L.ns_pack_step_learned.restype = i32
    L.ns_pack_step_learned.argtypes = [vp, vp, u32, u32, vp, vp]
    L.ns_pack_stream_windows.restype = i32
    L.ns_pack_stream_windows.argtypes = [vp, vp, vp]
    L.ns_pack_quota_table.restype = i32
    L.ns_pack_quota_table.argtypes = [vp, vp, vp]
    L.ns_pack_check.restype = i32
    L.ns_pack_check.argtypes = [vp]
    L.ns_pack_free.restype = None
    L.ns_pack_free.argtypes = [vp]
    L.ns_pack_strerror.restype = C.c_char_p
    L.ns_pack_strerror.argtypes = [i32]
    L.ns_pack_probe_hash_terms.restype = i32
    L.ns_pack_probe_hash_terms.argtypes = [u32, u32, vp, vp]
    L.ns_pack_quota_noalloc.restype = i32
    L.ns_pack_quota_noalloc.argtypes = [vp, u32, vp, vp, u32, u32, u32, vp, vp, vp]
    i64 = C.c_int64
    scan, distill, route = (C.POINTER(t) for t in
                            (ns_scan_inputs, ns_distill_inputs, ns_route_inputs))
    L.ns_scan_forward.restype = i32
    L.ns_scan_forward.argtypes = [scan, vp, vp, vp, vp, vp]
    L.ns_scan_workspace.restype = u64
    L.ns_scan_workspace.argtypes = [u32, u32, u32]
    L.ns_scan_backward.restype = i32
    L.ns_scan_backward.argtypes = [scan, vp, vp, i64, i64, vp, vp, vp, vp, vp, vp, vp]
    L.ns_distill.restype = i32
    L.ns_distill.argtypes = [distill, vp, vp, i64, vp]
    L.ns_route_workspace.restype = u64
    L.ns_route_workspace.argtypes = [u32, u32]
    L.ns_route_forward.restype = i32
    L.ns_route_forward.argtypes = [route, vp, vp, vp, vp, vp, vp, vp]
    L.ns_route_backward.restype = i32
    L.ns_route_backward.argtypes = [route, vp, vp, vp, vp, vp, vp, vp, vp]
    embed = norm = experts = vp  # structures or their bytes
    L.ns_embed_forward.restype = i32
    L.ns_embed_forward.argtypes = [embed, vp, i64, vp, vp]
    L.ns_embed_workspace.restype = u64
    L.ns_embed_workspace.argtypes = [u32, u32, u32]
    L.ns_embed_backward.restype = i32
    L.ns_embed_backward.argtypes = [embed, vp, i64, vp, vp, vp]
    L.ns_norm_forward.restype = i32
    L.ns_norm_forward.argtypes = [norm, vp, vp, vp, vp]
    L.ns_norm_workspace.restype = u64
    L.ns_norm_workspace.argtypes = [u32, u32]
    L.ns_norm_backward.restype = i32
    L.ns_norm_backward.argtypes = [norm, vp, vp, vp, i64, vp, vp, vp, vp, vp]
    L.ns_norm_probe_forward.restype = i32
    L.ns_norm_probe_forward.argtypes = [norm, u32, vp, vp, vp, vp]
    L.ns_norm_probe_backward.restype = i32
    L.ns_norm_probe_backward.argtypes = [norm, u32, vp, vp, vp, i64, vp, vp, vp, vp, vp]
    L.ns_dispatch_workspace.restype = u64
    L.ns_dispatch_workspace.argtypes = [u32, u32, u32]
    L.ns_dispatch.restype = i32
    L.ns_dispatch.argtypes = [experts, vp, vp, i64, vp, vp, vp, vp, vp, vp]
    L.ns_combine.restype = i32
    L.ns_combine.argtypes = [experts, vp, vp, vp, vp, i64, vp, vp]
    L.ns_combine_backward.restype = i32
    L.ns_combine_backward.argtypes = [experts, vp, vp, vp, vp, i64, vp, i64, vp, vp, vp]
    return L


lib = _load()


class NsPackError(RuntimeError):
    def __init__(self, code: int, what: str):
        msg = lib.ns_pack_strerror(code).decode()
        super().__init__(f"{what}: {msg} ({code})")
        self.code = code


def check(code: int, what: str) -> None:
    if code != NS_OK:
        raise NsPackError(code, what)


# ---- the C ABI under the same names ------------------------------------------
def ns_pack_init(cfg: ns_pack_config) -> C.c_void_p:
    h = C.c_void_p()
    check(lib.ns_pack_init(C.byref(cfg), C.byref(h)), "ns_pack_init")
    return h


def ns_pack_step(ctx, step0: int, n_steps: int, row_begin: int, row_end: int,
                 out: ns_pack_out, stream: int | None = None) -> None:
    check(lib.ns_pack_step(ctx, step0, n_steps, row_begin, row_end, C.byref(out), stream),
          f"ns_pack_step(step0={step0}, n_steps={n_steps}, rows=[{row_begin},{row_end}))")


def ns_pack_fingerprint(ctx, row_fp_ptr: int, n_rows: int, stream: int | None = None) -> int:
    v = C.c_uint64()
    check(lib.ns_pack_fingerprint(ctx, row_fp_ptr, n_rows, C.byref(v), stream),
          "ns_pack_fingerprint")
    return v.value


def ns_pack_batch_fp(ctx, row_fp_ptr: int, n_steps: int, n_rows: int, out_ptr: int,
                     stream: int | None = None) -> None:
    check(lib.ns_pack_batch_fp(ctx, row_fp_ptr, n_steps, n_rows, out_ptr, stream),
          "ns_pack_batch_fp")


def ns_pack_step_learned(ctx, row_learned_ptr: int, n_steps: int, n_rows: int, out_ptr: int,
                         stream: int | None = None) -> None:
    check(lib.ns_pack_step_learned(ctx, row_learned_ptr, n_steps, n_rows, out_ptr, stream),
          "ns_pack_step_learned")


def ns_pack_info(ctx) -> dict:
    info = ns_pack_info_t()
    check(lib.ns_pack_info(ctx, C.byref(info)), "ns_pack_info")
    return {name: getattr(info, name) for name, _ in ns_pack_info_t._fields_}


def ns_pack_stream_windows(ctx, n_streams: int):
    import numpy as np
    w = np.zeros(n_streams, np.uint64)
    c = np.zeros(n_streams, np.uint8)
    check(lib.ns_pack_stream_windows(ctx, w.ctypes.data, c.ctypes.data), "ns_pack_stream_windows")
    return w, c.astype(bool)


def ns_pack_quota_table(ctx, max_steps: int, n_streams: int):
    import numpy as np
    q = np.zeros((max_steps, n_streams), np.int32)
    cum = np.zeros((max_steps + 1, n_streams), np.int32)
    check(lib.ns_pack_quota_table(ctx, q.ctypes.data, cum.ctypes.data), "ns_pack_quota_table")
    return q, cum


def ns_pack_check(ctx) -> None:
    check(lib.ns_pack_check(ctx), "ns_pack_check")


def ns_pack_free(ctx) -> None:
    lib.ns_pack_free(ctx)


def ns_pack_quota_noalloc(source_weight, stream_source, stream_weight, B: int, max_steps: int,
                          quota_ptr: int, cum_ptr: int, stream: int | None = None) -> None:
    """Quota tables of a recipe into caller-owned device buffers, with no
    device allocation (for callers that cannot call cudaMalloc)."""
    import numpy as np
    sw = np.ascontiguousarray(source_weight, dtype=np.uint32)
    ss = np.ascontiguousarray(stream_source, dtype=np.uint32)
    tw = np.ascontiguousarray(stream_weight, dtype=np.uint32)
    check(lib.ns_pack_quota_noalloc(sw.ctypes.data, sw.size, ss.ctypes.data, tw.ctypes.data,
                                    ss.size, B, max_steps, quota_ptr, cum_ptr, stream),
          "ns_pack_quota_noalloc")


def ns_pack_strerror(code: int) -> str:
    return lib.ns_pack_strerror(code).decode()


def ns_pack_probe_hash_terms(blocks: int, terms_per_thread: int, sum_dev: int,
                             stream: int = 0) -> None:
    """Launch the register-only loop of the held-out hash's term (see
    include/nspack_probe.h); adds its sum to the device u64 at sum_dev."""
    check(lib.ns_pack_probe_hash_terms(blocks, terms_per_thread, sum_dev, stream or None),
          "ns_pack_probe_hash_terms")


# ---- training operators (include/nstrain.h) -----------------------------------
def ns_scan_forward(inputs: ns_scan_inputs, h0, y, h_last, states, stream) -> None:
    check(lib.ns_scan_forward(C.byref(inputs), h0, y, h_last, states, stream), "ns_scan_forward")


def ns_scan_workspace(B: int, T: int, D: int) -> int:
    _fits("B", B), _fits("T", T), _fits("D", D)
    return lib.ns_scan_workspace(B, T, D)


def ns_scan_backward(inputs: ns_scan_inputs, states, dy, dy_row: int, dy_time: int, dh_last, dz,
                     df, dbias, dh0, workspace, stream) -> None:
    check(lib.ns_scan_backward(C.byref(inputs), states, dy, dy_row, dy_time, dh_last, dz, df, dbias,
                               dh0, workspace, stream), "ns_scan_backward")


def ns_distill(inputs: ns_distill_inputs, loss, dlogits, dlogits_row: int, stream) -> None:
    check(lib.ns_distill(C.byref(inputs), loss, dlogits, dlogits_row, stream), "ns_distill")


def ns_route_workspace(N: int, E: int) -> int:
    _fits("N", N), _fits("E", E)
    return lib.ns_route_workspace(N, E)


def ns_route_forward(inputs: ns_route_inputs, ids, weights, counts, tokens, loss, workspace,
                     stream) -> None:
    check(lib.ns_route_forward(C.byref(inputs), ids, weights, counts, tokens, loss, workspace,
                               stream), "ns_route_forward")


def ns_route_backward(inputs: ns_route_inputs, ids, weights, counts, tokens, d_weights, d_loss,
                      dlogits, stream) -> None:
    check(lib.ns_route_backward(C.byref(inputs), ids, weights, counts, tokens, d_weights, d_loss,
                                dlogits, stream), "ns_route_backward")


def ns_embed_forward(inputs, table, table_row: int, y, stream) -> None:
    check(lib.ns_embed_forward(_argument(inputs), table, table_row, y, stream), "ns_embed_forward")


def ns_embed_workspace(N: int, V: int, D: int) -> int:
    _fits("N", N), _fits("V", V), _fits("D", D)
    return lib.ns_embed_workspace(N, V, D)


def ns_embed_backward(inputs, dy, dy_row: int, dtable, workspace, stream) -> None:
    check(lib.ns_embed_backward(_argument(inputs), dy, dy_row, dtable, workspace, stream),
          "ns_embed_backward")


def ns_norm_forward(inputs, y, mean, rstd, stream) -> None:
    check(lib.ns_norm_forward(_argument(inputs), y, mean, rstd, stream), "ns_norm_forward")


def ns_norm_workspace(N: int, D: int) -> int:
    _fits("N", N), _fits("D", D)
    return lib.ns_norm_workspace(N, D)


def ns_norm_backward(inputs, mean, rstd, dy, dy_row: int, dx, dweight, dbias,
                     workspace, stream) -> None:
    check(lib.ns_norm_backward(_argument(inputs), mean, rstd, dy, dy_row, dx, dweight, dbias,
                               workspace, stream), "ns_norm_backward")


def ns_norm_probe_forward(inputs, fed: int, y, mean, rstd, stream) -> None:
    """ns_norm_forward where only ``fed`` rows come (see include/nstrain_probe.h)."""
    check(lib.ns_norm_probe_forward(_argument(inputs), fed, y, mean, rstd, stream),
          "ns_norm_probe_forward")


def ns_norm_probe_backward(inputs, fed: int, mean, rstd, dy, dy_row: int, dx, dweight,
                           dbias, workspace, stream) -> None:
    check(lib.ns_norm_probe_backward(_argument(inputs), fed, mean, rstd, dy, dy_row, dx,
                                     dweight, dbias, workspace, stream), "ns_norm_probe_backward")


def ns_dispatch_workspace(N: int, k: int, E: int) -> int:
    _fits("N", N), _fits("k", k), _fits("E", E)
    return lib.ns_dispatch_workspace(N, k, E)


def ns_dispatch(sizes, ids, x, x_row: int, place, slots, offsets, rows, workspace,
                stream) -> None:
    check(lib.ns_dispatch(_argument(sizes), ids, x, x_row, place, slots, offsets, rows, workspace,
                          stream), "ns_dispatch")


def ns_combine(sizes, place, offsets, weights, rows, rows_row: int, out,
               stream) -> None:
    check(lib.ns_combine(_argument(sizes), place, offsets, weights, rows, rows_row, out, stream),
          "ns_combine")


def ns_combine_backward(sizes, place, offsets, weights, rows, rows_row: int, d_out,
                        d_out_row: int, d_rows, d_weights, stream) -> None:
    check(lib.ns_combine_backward(_argument(sizes), place, offsets, weights, rows, rows_row, d_out,
                                  d_out_row, d_rows, d_weights, stream), "ns_combine_backward")
