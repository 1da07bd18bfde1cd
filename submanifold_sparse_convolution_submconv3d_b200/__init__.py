"""Python binding of the B200 SubMConv3d library (``include/spconv.h``).

Argument marshalling only: every step of the hot path (map build, gather, GEMM,
store) runs in the CUDA library ``libspconv_b200.so``.  PyTorch supplies device
memory and the current stream.  Importing this package fails loudly if the
library has not been built (``python -m submanifold_sparse_convolution_submconv3d_b200.build``).

The functions carry the C names:

* ``spconv_build_map(coords, extent, kernel_size=3, flip_kernel=False, sorted_keys=False)``
  -> ``SubmMap`` (``spconv_build_map_ex`` when an option is set)
* ``spconv_subm_forward(map, x, w, bias=None, out=None)`` -> ``out``
* ``spconv_free(map)``
* ``spconv_downsample_build(coords, extent, factor=2)`` -> ``Downsample``;
  ``spconv_downsample_amax(ds, x)``, ``spconv_upsample(ds, x_coarse)``
* ``spconv_subdivide(coords, extent, x=None)`` -> ``(coords_out, x_out)``
* ``spconv_rms_norm(x, weight, residual=None)`` -> ``out`` or ``(out, sum)``; ``spconv_rms_norm_q8`` ->
  ``(q, scale)`` or ``(q, scale, sum)``; ``spconv_rms_norm_backward(dy, h, weight, rstd)`` -> ``(dx, dweight)``
* ``spconv_rope_create(head_dim)`` -> ``Rope``; ``spconv_rope_apply(rope, coords, x, inverse=False)`` -> ``out``
* ``spconv_w4_quantize(w)`` -> ``(packed, scales, offsets)``; ``spconv_w4_dequantize``;
  ``spconv_linear_w4(x, packed, scales, offsets, bias=None, x_scale=None)`` -> ``out``
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspconv_b200.so")

OK, INVALID_ARG, UNSUPPORTED, COORD_RANGE, DUPLICATE, TABLE_FULL, OOM, CUDA_ERROR, TIMEOUT = range(9)
MAP_DEFAULT, MAP_FLIP_KERNEL, MAP_SORTED_KEYS, MAP_HASH_TABLE, MAP_SHORT_TILES = 0, 1, 2, 4, 8
ALGO_AUTO, ALGO_SIMT, ALGO_TCGEN05 = 0, 1, 2
ROPE_INTERLEAVED, ROPE_HALVES = 0, 1
ROPE_LAYOUTS = {"interleaved": ROPE_INTERLEAVED, "halves": ROPE_HALVES}
W4_MAX_ROWS = 32
KERNEL_SIMT, KERNEL_TCGEN05, KERNEL_TCGEN05_GEMM = 0, 1, 2
KERNEL_NAMES = ("simt", "tcgen05", "tcgen05_gemm")
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}

EXPORTED = ("spconv_build_map", "spconv_subm_forward", "spconv_free", "spconv_map_info", "spconv_map_check",
            "spconv_map_tile_rows",
            "spconv_last_error", "spconv_subm_forward_algo", "spconv_debug_set_table_slots",
            "spconv_debug_set_tile_rows", "spconv_build_neighbor_map_noalloc", "spconv_map_launch_counts",
            "spconv_map_stats", "spconv_debug_set_ring_depths", "spconv_build_map_ex", "spconv_downsample_build",
            "spconv_downsample_info", "spconv_downsample_amax", "spconv_upsample", "spconv_downsample_free",
            "spconv_subdivide", "spconv_subm_forward_ex", "spconv_rms_norm", "spconv_rms_norm_q8",
            "spconv_rms_norm_workspace", "spconv_rms_norm_backward", "spconv_rope_create", "spconv_rope_free",
            "spconv_rope_apply", "spconv_w4_quantize", "spconv_w4_dequantize", "spconv_linear_w4")


class _MapStats(ctypes.Structure):
    _fields_ = [("tiles", ctypes.c_int64), ("rows_per_tile", ctypes.c_int32), ("job_stride", ctypes.c_int32),
                ("spans", ctypes.c_int64), ("span_cols", ctypes.c_int64), ("perm_dev", ctypes.c_void_p),
                ("nbr_t_dev", ctypes.c_void_p), ("jobs_dev", ctypes.c_void_p), ("order_dev", ctypes.c_void_p)]


class _Epilogue(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int), ("residual", ctypes.c_void_p), ("stats", ctypes.c_void_p)]


ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3}


class SpconvError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"spconv status {status}: {message}")
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"CUDA library not built: {LIB_PATH} is missing "
                          "(run python -m submanifold_sparse_convolution_submconv3d_b200.build)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.spconv_build_map.argtypes = [vp, i64, vp, i32, vp, ctypes.POINTER(vp)]
    lib.spconv_subm_forward.argtypes = [vp, ctypes.c_int, vp, i32, vp, vp, vp, i32, vp]
    lib.spconv_subm_forward_algo.argtypes = [vp, ctypes.c_int, vp, i32, vp, vp, vp, i32, ctypes.c_int, vp]
    lib.spconv_free.argtypes = [vp]
    lib.spconv_map_info.argtypes = [vp, ctypes.POINTER(i64), ctypes.POINTER(i32), ctypes.POINTER(i64),
                                    ctypes.POINTER(vp)]
    lib.spconv_map_check.argtypes = [vp, vp]
    lib.spconv_map_tile_rows.argtypes = [vp, ctypes.POINTER(i32)]
    lib.spconv_debug_set_table_slots.argtypes = [i64]
    lib.spconv_debug_set_tile_rows.argtypes = [i32]
    lib.spconv_build_neighbor_map_noalloc.argtypes = [vp, i64, vp, vp, ctypes.POINTER(i64), vp]
    lib.spconv_map_launch_counts.argtypes = [vp, ctypes.POINTER(i64), i32]
    lib.spconv_map_stats.argtypes = [vp, ctypes.POINTER(_MapStats)]
    lib.spconv_debug_set_ring_depths.argtypes = [i32, i32]
    lib.spconv_build_map_ex.argtypes = [vp, i64, vp, i32, ctypes.c_uint32, vp, ctypes.POINTER(vp)]
    lib.spconv_downsample_build.argtypes = [vp, i64, vp, i32, vp, ctypes.POINTER(vp)]
    lib.spconv_downsample_info.argtypes = [vp, ctypes.POINTER(i64), ctypes.POINTER(i64), vp, ctypes.POINTER(vp),
                                           ctypes.POINTER(vp)]
    lib.spconv_downsample_amax.argtypes = [vp, ctypes.c_int, vp, i32, vp, vp]
    lib.spconv_upsample.argtypes = [vp, ctypes.c_int, vp, i32, vp, vp]
    lib.spconv_downsample_free.argtypes = [vp]
    lib.spconv_subdivide.argtypes = [vp, i64, vp, ctypes.c_int, vp, i32, vp, vp, vp]
    lib.spconv_subm_forward_ex.argtypes = [vp, ctypes.c_int, vp, i32, vp, vp, vp, i32, ctypes.POINTER(_Epilogue),
                                           ctypes.c_int, vp]
    f32, fn = ctypes.c_float, ctypes.c_int
    lib.spconv_rms_norm.argtypes = [fn, vp, vp, vp, i64, i32, f32, vp, vp, vp, vp]
    lib.spconv_rms_norm_q8.argtypes = [fn, vp, vp, vp, i64, i32, f32, vp, vp, vp, vp]
    lib.spconv_rms_norm_workspace.argtypes = [i64, i32, ctypes.POINTER(i64)]
    lib.spconv_rms_norm_backward.argtypes = [fn, vp, vp, vp, vp, vp, i64, i32, vp, vp, vp, vp]
    lib.spconv_rope_create.argtypes = [i32, fn, ctypes.c_double, vp, vp, ctypes.POINTER(vp)]
    lib.spconv_rope_free.argtypes = [vp]
    lib.spconv_rope_apply.argtypes = [vp, fn, vp, i64, vp, i32, i64, i64, vp, i64, i64, i32, vp]
    lib.spconv_w4_quantize.argtypes = [fn, vp, i32, i32, i32, vp, vp, vp, vp]
    lib.spconv_w4_dequantize.argtypes = [fn, vp, vp, vp, i32, i32, i32, vp, vp]
    lib.spconv_linear_w4.argtypes = [fn, vp, vp, i64, i32, vp, vp, vp, i32, vp, vp, i32, vp]
    lib.spconv_last_error.restype = ctypes.c_char_p
    for name in ("spconv_build_map", "spconv_subm_forward", "spconv_subm_forward_algo", "spconv_free",
                 "spconv_map_info", "spconv_map_check", "spconv_map_tile_rows", "spconv_debug_set_table_slots",
                 "spconv_debug_set_tile_rows", "spconv_build_neighbor_map_noalloc", "spconv_map_launch_counts",
                 "spconv_map_stats", "spconv_debug_set_ring_depths", "spconv_build_map_ex",
                 "spconv_downsample_build", "spconv_downsample_info", "spconv_downsample_amax", "spconv_upsample",
                 "spconv_downsample_free", "spconv_subdivide", "spconv_subm_forward_ex", "spconv_rms_norm",
                 "spconv_rms_norm_q8", "spconv_rms_norm_workspace", "spconv_rms_norm_backward", "spconv_rope_create",
                 "spconv_rope_free", "spconv_rope_apply", "spconv_w4_quantize", "spconv_w4_dequantize",
                 "spconv_linear_w4"):
        getattr(lib, name).restype = ctypes.c_int
    return lib


try:
    lib = _load()
    _LOAD_ERROR = None
except (OSError, AttributeError, ImportError) as _exc:  # missing or stale library
    lib = None
    _LOAD_ERROR = _exc


def _require() -> None:
    """Raise if the CUDA library could not be loaded: there is no fallback path."""
    if lib is None:
        raise ImportError(f"the CUDA library {LIB_PATH} is unavailable ({_LOAD_ERROR}); build it with "
                          "python -m submanifold_sparse_convolution_submconv3d_b200.build")


def _check(status: int) -> None:
    if status != OK:
        raise SpconvError(status, lib.spconv_last_error().decode())


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


class SubmMap:
    """Owns a neighbour-map handle; freed by ``free()`` or garbage collection."""

    def __init__(self, handle: int, device: torch.device):
        self.handle = handle
        self.device = device
        n, ks, pairs, ptr = ctypes.c_int64(), ctypes.c_int32(), ctypes.c_int64(), ctypes.c_void_p()
        _check(lib.spconv_map_info(handle, ctypes.byref(n), ctypes.byref(ks), ctypes.byref(pairs), ctypes.byref(ptr)))
        self.n, self.kernel_size, self.pairs = n.value, ks.value, pairs.value
        self._nbr_ptr = ptr.value
        rows = ctypes.c_int32()
        _check(lib.spconv_map_tile_rows(handle, ctypes.byref(rows)))
        self.tile_rows = rows.value  # rows per forward tile (<= 384)

    def _copy_device(self, ptr: int, shape: tuple, typestr: str, dtype) -> torch.Tensor:
        """Copy of a library-owned device buffer, viewed through the CUDA array interface."""
        out = torch.empty(shape, dtype=dtype, device=self.device)
        if out.numel():
            class _View:
                __cuda_array_interface__ = {"shape": shape, "typestr": typestr, "data": (ptr, False), "version": 3}
            out.copy_(torch.as_tensor(_View(), device=self.device))
        return out

    def neighbor_map(self) -> torch.Tensor:
        """Copy of the dense int32 [n, 27] map (identity column for kernel size 1)."""
        if self.kernel_size == 1:
            return torch.arange(self.n, dtype=torch.int32, device=self.device).view(-1, 1)
        return self._copy_device(self._nbr_ptr, (self.n, 27), "<i4", torch.int32)

    def stats(self, copy_arrays: bool = False) -> dict:
        """The tensor-core forward's metadata (spconv_map_stats): tiling, span counts
        and, with copy_arrays, copies of perm [n], nbr_t [27, tiles * rows_per_tile],
        jobs [tiles, job_stride] (uint32 words as int64) and order [tiles]."""
        st = _MapStats()
        _check(lib.spconv_map_stats(self.handle, ctypes.byref(st)))
        d = {"tiles": st.tiles, "rows_per_tile": st.rows_per_tile, "job_stride": st.job_stride, "spans": st.spans,
             "span_cols": st.span_cols}
        if copy_arrays and st.perm_dev:
            npad = st.tiles * st.rows_per_tile
            d["perm"] = self._copy_device(st.perm_dev, (self.n,), "<i4", torch.int32)
            d["nbr_t"] = self._copy_device(st.nbr_t_dev, (27, npad), "<i4", torch.int32)
            d["jobs"] = self._copy_device(st.jobs_dev, (st.tiles, st.job_stride), "<i4",
                                          torch.int32).to(torch.int64) & 0xFFFFFFFF
            d["order"] = self._copy_device(st.order_dev, (st.tiles,), "<i4", torch.int32)
        return d

    def launch_counts(self) -> dict:
        """Forward launches on this map per kernel family, e.g. {"simt": 0, "tcgen05": 3}."""
        counts = (ctypes.c_int64 * len(KERNEL_NAMES))()
        _check(lib.spconv_map_launch_counts(self.handle, counts, len(KERNEL_NAMES)))
        return dict(zip(KERNEL_NAMES, counts))

    def check(self, stream=None) -> None:
        """Synchronise and raise if a forward kernel's bounded wait gave up.  The
        default stream is the current stream of the map's device."""
        with torch.cuda.device(self.device):
            _check(lib.spconv_map_check(self.handle, _stream(stream)))

    def free(self) -> None:
        if self.handle:
            lib.spconv_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def _coords_arg(coords: torch.Tensor) -> torch.Tensor:
    if coords.dtype != torch.int32 or not coords.is_cuda or coords.dim() != 2 or coords.shape[1] != 4:
        raise ValueError("coords must be a CUDA int32 tensor of shape [N, 4]")
    return coords.contiguous()


def spconv_build_map(coords: torch.Tensor, extent, kernel_size: int = 3, stream=None, flip_kernel: bool = False,
                     sorted_keys: bool | None = None, short_tiles: bool = False) -> SubmMap:
    """Build the neighbour map of int32 [N, 4] (b, x, y, z) CUDA coordinates.
    ``flip_kernel`` gathers p - d_k; ``sorted_keys`` True builds the dictionary from
    sorted keys instead of the hash table (same map; None and False: the hash table);
    ``short_tiles`` cuts the forward's tiles at 128 rows (faster for layers with 128
    or more input channels)."""
    _require()
    coords = _coords_arg(coords)
    ext = (ctypes.c_int32 * 3)(*[int(v) for v in extent])
    handle = ctypes.c_void_p()
    flags = (MAP_FLIP_KERNEL if flip_kernel else 0) | (MAP_SHORT_TILES if short_tiles else 0) | \
        {None: 0, True: MAP_SORTED_KEYS, False: MAP_HASH_TABLE}[sorted_keys]
    with torch.cuda.device(coords.device):
        ptr = coords.data_ptr() if coords.numel() else None
        if flags:
            _check(lib.spconv_build_map_ex(ptr, coords.shape[0], ext, kernel_size, flags, _stream(stream),
                                           ctypes.byref(handle)))
        else:
            _check(lib.spconv_build_map(ptr, coords.shape[0], ext, kernel_size, _stream(stream),
                                        ctypes.byref(handle)))
    return SubmMap(handle.value, coords.device)


def spconv_subm_forward(m: SubmMap, x: torch.Tensor, w: torch.Tensor, bias: torch.Tensor | None = None,
                        out: torch.Tensor | None = None, algo: int = ALGO_AUTO, stream=None, act: str | None = None,
                        residual: torch.Tensor | None = None, stats: torch.Tensor | None = None) -> torch.Tensor:
    """One SubMConv3d layer: x [N, Cin], w [K^3, Cin, Cout], bias [Cout] -> out [N, Cout].
    Fused epilogue (spconv_subm_forward_ex): out = act(conv + bias) (+ residual [N, Cout],
    which may be ``out`` itself); ``stats``, a float32 CUDA tensor [2, Cout], receives the
    per-channel sum and sum of squares of out."""
    _require()
    if x.dtype not in _DTYPES:
        raise ValueError("x must be float32 or bfloat16")
    for t in (w,) + (() if bias is None else (bias,)):
        if t.dtype != x.dtype or t.device != x.device:
            raise ValueError("w and bias must match x in dtype and device")
    if x.dim() != 2 or w.dim() != 3:
        raise ValueError(f"x must be [N, Cin] and w [K^3, Cin, Cout]; got x {tuple(x.shape)}, w {tuple(w.shape)}")
    cin, cout = int(w.shape[1]), int(w.shape[2])
    if x.shape != (m.n, cin) or w.shape[0] != m.kernel_size ** 3:
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, w {tuple(w.shape)}, map n={m.n} k={m.kernel_size}")
    if bias is not None and bias.shape != (cout,):
        raise ValueError(f"bias must be [Cout] = [{cout}]; got {tuple(bias.shape)}")
    if out is not None and (out.shape != (m.n, cout) or out.dtype != x.dtype or not out.is_contiguous()):
        raise ValueError("out must be a contiguous [N, Cout] tensor of x's dtype")
    # The library reads and writes these through raw device pointers: a host
    # tensor, or one on another GPU than the map, must never reach it.
    if not x.is_cuda or x.device != m.device or (out is not None and out.device != x.device):
        raise ValueError(f"x, w, bias and out must be CUDA tensors on the map's device {m.device}")
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(k for k in ACTIVATIONS if k)} or None")
    if residual is not None and (residual.shape != (m.n, cout) or residual.dtype != x.dtype
                                 or residual.device != x.device or not residual.is_contiguous()):
        raise ValueError("residual must be a contiguous [N, Cout] tensor of x's dtype on x's device")
    if stats is not None and (stats.shape != (2, cout) or stats.dtype != torch.float32
                              or stats.device != x.device or not stats.is_contiguous()):
        raise ValueError("stats must be a contiguous float32 [2, Cout] tensor on x's device")
    x, w = x.contiguous(), w.contiguous()
    bias = None if bias is None else bias.contiguous()
    if out is None:
        out = torch.empty((m.n, cout), dtype=x.dtype, device=x.device)
    if m.n == 0:
        if stats is not None:
            stats.zero_()
        return out
    with torch.cuda.device(x.device):
        if ACTIVATIONS[act] or residual is not None or stats is not None:
            epi = _Epilogue(ACTIVATIONS[act], None if residual is None else residual.data_ptr(),
                            None if stats is None else stats.data_ptr())
            _check(lib.spconv_subm_forward_ex(m.handle, _DTYPES[x.dtype], x.data_ptr(), cin, w.data_ptr(),
                                              None if bias is None else bias.data_ptr(), out.data_ptr(), cout,
                                              ctypes.byref(epi), algo, _stream(stream)))
        else:
            _check(lib.spconv_subm_forward_algo(m.handle, _DTYPES[x.dtype], x.data_ptr(), cin, w.data_ptr(),
                                                None if bias is None else bias.data_ptr(), out.data_ptr(), cout,
                                                algo, _stream(stream)))
    return out


def spconv_free(m: SubmMap) -> None:
    m.free()


def spconv_build_neighbor_map_noalloc(coords: torch.Tensor, extent, out: torch.Tensor | None = None,
                                      stream=None) -> tuple[torch.Tensor, int]:
    """Dense int32 [N, 27] neighbour map built without any device allocation by
    the library (scratch in a static device array; N <= 524288).  The caller may
    pass ``out``; otherwise the binding allocates it with torch before the call.
    Returns (map, pairs)."""
    _require()
    if coords.dtype != torch.int32 or not coords.is_cuda or coords.dim() != 2 or coords.shape[1] != 4:
        raise ValueError("coords must be a CUDA int32 tensor of shape [N, 4]")
    coords = coords.contiguous()
    n = coords.shape[0]
    if out is None:
        out = torch.empty((n, 27), dtype=torch.int32, device=coords.device)
    elif out.shape != (n, 27) or out.dtype != torch.int32 or not out.is_contiguous() or out.device != coords.device:
        raise ValueError("out must be a contiguous int32 [N, 27] tensor on the device of coords")
    ext = (ctypes.c_int32 * 3)(*[int(v) for v in extent])
    pairs = ctypes.c_int64()
    with torch.cuda.device(coords.device):
        _check(lib.spconv_build_neighbor_map_noalloc(coords.data_ptr() if n else None, n, ext,
                                                     out.data_ptr() if n else None, ctypes.byref(pairs),
                                                     _stream(stream)))
    return out, pairs.value


class Downsample:
    """Owns a downsample handle (spconv_downsample_build): the coarse voxel set and
    the pairing of input voxels with coarse voxels."""

    def __init__(self, handle: int, device: torch.device):
        self.handle = handle
        self.device = device
        nf, nc, ext = ctypes.c_int64(), ctypes.c_int64(), (ctypes.c_int32 * 3)()
        cptr, pptr = ctypes.c_void_p(), ctypes.c_void_p()
        _check(lib.spconv_downsample_info(handle, ctypes.byref(nf), ctypes.byref(nc), ext, ctypes.byref(cptr),
                                          ctypes.byref(pptr)))
        self.n, self.n_coarse, self.coarse_extent = nf.value, nc.value, tuple(ext)
        self._coarse_ptr, self._parent_ptr = cptr.value, pptr.value

    def _copy(self, ptr, shape) -> torch.Tensor:
        out = torch.empty(shape, dtype=torch.int32, device=self.device)
        if out.numel():
            class _View:
                __cuda_array_interface__ = {"shape": shape, "typestr": "<i4", "data": (ptr, False), "version": 3}
            out.copy_(torch.as_tensor(_View(), device=self.device))
        return out

    def coarse_coords(self) -> torch.Tensor:
        """Copy of the coarse coordinates, int32 [n_coarse, 4], sorted."""
        return self._copy(self._coarse_ptr, (self.n_coarse, 4))

    def parent(self) -> torch.Tensor:
        """Copy of the coarse row of every input row, int32 [n]."""
        return self._copy(self._parent_ptr, (self.n,))

    def free(self) -> None:
        if self.handle:
            lib.spconv_downsample_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def spconv_downsample_build(coords: torch.Tensor, extent, factor: int = 2, stream=None) -> Downsample:
    """SparseDownsample(factor) coordinates of int32 [N, 4] CUDA coordinates."""
    _require()
    coords = _coords_arg(coords)
    ext = (ctypes.c_int32 * 3)(*[int(v) for v in extent])
    handle = ctypes.c_void_p()
    with torch.cuda.device(coords.device):
        _check(lib.spconv_downsample_build(coords.data_ptr() if coords.numel() else None, coords.shape[0], ext,
                                           int(factor), _stream(stream), ctypes.byref(handle)))
    return Downsample(handle.value, coords.device)


def _rows_arg(x: torch.Tensor, rows: int, device, what: str) -> torch.Tensor:
    if x.dtype not in _DTYPES or not x.is_cuda or x.device != device or x.dim() != 2 or x.shape[0] != rows:
        raise ValueError(f"{what} must be a float32 or bfloat16 CUDA tensor [{rows}, C] on {device}")
    return x.contiguous()


def spconv_downsample_amax(ds: Downsample, x: torch.Tensor, out: torch.Tensor | None = None,
                           stream=None) -> torch.Tensor:
    """Max pooling of x [n, C] onto the coarse voxels -> [n_coarse, C]."""
    _require()
    x = _rows_arg(x, ds.n, ds.device, "x")
    if out is None:
        out = torch.empty((ds.n_coarse, x.shape[1]), dtype=x.dtype, device=x.device)
    elif out.shape != (ds.n_coarse, x.shape[1]) or out.dtype != x.dtype or not out.is_contiguous() \
            or out.device != x.device:
        raise ValueError("out must be a contiguous [n_coarse, C] tensor like x")
    if ds.n:
        with torch.cuda.device(x.device):
            _check(lib.spconv_downsample_amax(ds.handle, _DTYPES[x.dtype], x.data_ptr(), x.shape[1], out.data_ptr(),
                                              _stream(stream)))
    return out


def spconv_upsample(ds: Downsample, x_coarse: torch.Tensor, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Coarse features [n_coarse, C] back onto the downsample's input voxels -> [n, C]."""
    _require()
    x_coarse = _rows_arg(x_coarse, ds.n_coarse, ds.device, "x_coarse")
    if out is None:
        out = torch.empty((ds.n, x_coarse.shape[1]), dtype=x_coarse.dtype, device=x_coarse.device)
    elif out.shape != (ds.n, x_coarse.shape[1]) or out.dtype != x_coarse.dtype or not out.is_contiguous() \
            or out.device != x_coarse.device:
        raise ValueError("out must be a contiguous [n, C] tensor like x_coarse")
    if ds.n:
        with torch.cuda.device(x_coarse.device):
            _check(lib.spconv_upsample(ds.handle, _DTYPES[x_coarse.dtype], x_coarse.data_ptr(), x_coarse.shape[1],
                                       out.data_ptr(), _stream(stream)))
    return out


def spconv_subdivide(coords: torch.Tensor, extent, x: torch.Tensor | None = None,
                     stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """SparseSubdivide: int32 [N, 4] coordinates (and optional features [N, C]) ->
    the 8 N children (coordinates [8N, 4], features [8N, C]) on the grid 2 * extent."""
    _require()
    coords = _coords_arg(coords)
    n = coords.shape[0]
    ext = (ctypes.c_int32 * 3)(*[int(v) for v in extent])
    coords_out = torch.empty((8 * n, 4), dtype=torch.int32, device=coords.device)
    x_out = None
    if x is not None:
        x = _rows_arg(x, n, coords.device, "x")
        x_out = torch.empty((8 * n, x.shape[1]), dtype=x.dtype, device=x.device)
    with torch.cuda.device(coords.device):
        _check(lib.spconv_subdivide(coords.data_ptr() if n else None, n, ext,
                                    _DTYPES[x.dtype] if x is not None else 0,
                                    x.data_ptr() if x is not None and n else None,
                                    x.shape[1] if x is not None else 0, coords_out.data_ptr() if n else None,
                                    x_out.data_ptr() if x_out is not None and n else None, _stream(stream)))
    return coords_out, x_out


# ------------------------------------------------------------ operators on feature rows
# One token's row is a few microseconds of GPU work, so these calls keep the host side
# short: they enter a device or stream context only where it is not current already, ask
# torch for the current stream's handle without making a Stream object (0.1 us against
# 3.2) and make results like an input where they can (1.3 us against 2.4).

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


@contextlib.contextmanager
def _on(device: torch.device, stream):
    """Make ``stream`` (None: the device's current stream) the current one, so that the
    results and temporaries of a call are allocated and written in its order."""
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(_stream(stream), device=device)
            if stream.device != device:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
            with torch.cuda.stream(stream):
                yield


def _in(t: torch.Tensor) -> torch.Tensor:
    """An input as the library reads it: contiguous, on a 16-byte boundary."""
    if not t.is_contiguous():
        return t.contiguous()
    return t.clone() if t.data_ptr() & 15 else t


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _like(t, shape, dtype, device, what: str) -> None:
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        raise ValueError(f"{what} must be a {str(dtype)[6:]} tensor {list(shape)} on {device}; got "
                         f"{str(t.dtype)[6:]} {list(t.shape)} on {t.device}")


def _out(t, like: torch.Tensor, shape, dtype, what: str) -> torch.Tensor:
    """The result tensor the caller gave, checked, or a new one on ``like``'s device."""
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    _like(t, shape, dtype, like.device, what)
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t


def _out_like(t, like: torch.Tensor, what: str) -> torch.Tensor:
    """``_out`` of the shape and type of ``like``, which is contiguous."""
    return torch.empty_like(like) if t is None else _out(t, like, like.shape, like.dtype, what)


def _norm_rows(x, weight, what: str, more=(), names=()) -> int:
    """Checks rows, the weight and ``more`` tensors shaped like the rows; returns the device."""
    shape, dtype, index = x.shape, x.dtype, x.get_device()
    if dtype not in _DTYPES or index < 0 or len(shape) != 2:
        raise ValueError(f"{what} must be a float32 or bfloat16 CUDA tensor [N, C]")
    if weight is not None and (weight.dtype is not dtype or weight.get_device() != index or weight.dim() != 1
                               or weight.numel() != shape[1]):
        _like(weight, shape[1:], dtype, x.device, "weight")
    for t, name in zip(more, names):
        if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
            _like(t, shape, dtype, x.device, name)
    return index


def spconv_rms_norm(x: torch.Tensor, weight: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                    eps: float = 1e-6, out: torch.Tensor | None = None, sum_out: torch.Tensor | None = None,
                    rstd: torch.Tensor | None = None, stream=None):
    """Root-mean-square norm of rows x [N, C], with the residual's addition: returns
    ``out``, or ``(out, sum)`` with sum = x + residual where a residual is given.
    ``sum_out`` may be ``residual`` or ``x`` itself; ``rstd``, a float32 CUDA tensor [N],
    receives what ``spconv_rms_norm_backward`` reads.  Inputs that are not contiguous, such
    as the heads of a packed projection, are copied first."""
    _require()
    index = _norm_rows(x, weight, "x", () if residual is None else (residual,), ("residual",))
    if stream is not None or index != _device_now():
        with _on(x.device, stream):
            return spconv_rms_norm(x, weight, residual, eps, out, sum_out, rstd)
    n, c = x.shape
    x = _in(x)
    if weight is not None:
        weight = _in(weight)
    if residual is not None:
        residual, sum_out = _in(residual), _out_like(sum_out, x, "sum_out")
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual")
    if rstd is not None:
        _out(rstd, x, (n,), torch.float32, "rstd")
    out = _out_like(out, x, "out")
    _check(lib.spconv_rms_norm(_DTYPES[x.dtype], x.data_ptr(), _ptr(residual), _ptr(weight), n, c, eps, _ptr(sum_out),
                               out.data_ptr(), _ptr(rstd), _raw_stream(index)))
    return out if residual is None else (out, sum_out)


def spconv_rms_norm_q8(x: torch.Tensor, weight: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                       eps: float = 1e-6, out: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                       sum_out: torch.Tensor | None = None, stream=None):
    """``spconv_rms_norm`` with the result in 8 bits: returns ``(q, scale)`` or ``(q,
    scale, sum)``, q float8_e4m3fn [N, C] and scale float32 [N], the norm being about
    q * scale.  ``spconv_linear_w4`` takes both, for up to W4_MAX_ROWS rows; the layers for
    more rows take float32 and bfloat16, as ``spconv_rms_norm`` writes them."""
    _require()
    index = _norm_rows(x, weight, "x", () if residual is None else (residual,), ("residual",))
    if stream is not None or index != _device_now():
        with _on(x.device, stream):
            return spconv_rms_norm_q8(x, weight, residual, eps, out, scale, sum_out)
    n, c = x.shape
    x = _in(x)
    if weight is not None:
        weight = _in(weight)
    if residual is not None:
        residual, sum_out = _in(residual), _out_like(sum_out, x, "sum_out")
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual")
    out = torch.empty_like(x, dtype=torch.float8_e4m3fn) if out is None else \
        _out(out, x, (n, c), torch.float8_e4m3fn, "out")
    scale = _out(scale, x, (n,), torch.float32, "scale")
    _check(lib.spconv_rms_norm_q8(_DTYPES[x.dtype], x.data_ptr(), _ptr(residual), _ptr(weight), n, c, eps,
                                  _ptr(sum_out), out.data_ptr(), scale.data_ptr(), _raw_stream(index)))
    return (out, scale) if residual is None else (out, scale, sum_out)


@functools.lru_cache(maxsize=256)
def _norm_workspace(n: int, c: int) -> int:
    size = ctypes.c_int64()
    _check(lib.spconv_rms_norm_workspace(n, c, ctypes.byref(size)))
    return size.value


def spconv_rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor | None, rstd: torch.Tensor,
                             dsum: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                             weight_grad: bool = True, stream=None):
    """Gradient of ``spconv_rms_norm``: returns ``(dx, dweight)``.  h is the sum (or x
    where there was no residual); dx is the gradient of x and of the residual, with
    ``dsum``, the gradient that reaches the sum by other ways, added (dx may be dsum
    itself).  dweight is float32 [C], or None without a weight or with weight_grad False."""
    _require()
    index = _norm_rows(h, weight, "h", (dy,) if dsum is None else (dy, dsum), ("dy", "dsum"))
    if stream is not None or index != _device_now():
        with _on(h.device, stream):
            return spconv_rms_norm_backward(dy, h, weight, rstd, dsum, dx, weight_grad)
    n, c = h.shape
    if rstd.dim() != 1 or rstd.numel() != n or rstd.dtype is not torch.float32 or rstd.get_device() != index:
        _like(rstd, (n,), torch.float32, h.device, "rstd")
    dy, h, rstd = _in(dy), _in(h), _in(rstd)
    if dsum is not None:
        dsum = _in(dsum)
    dx = _out_like(dx, h, "dx")
    dweight = workspace = None
    if weight is not None:
        weight = _in(weight)
        if weight_grad:
            workspace = rstd.new_empty(_norm_workspace(n, c) // 4)
            dweight = rstd.new_empty(c)
    _check(lib.spconv_rms_norm_backward(_DTYPES[h.dtype], dy.data_ptr(), h.data_ptr(), _ptr(weight), rstd.data_ptr(),
                                        _ptr(dsum), n, c, dx.data_ptr(), _ptr(dweight), _ptr(workspace),
                                        _raw_stream(index)))
    return dx, dweight


class Rope:
    """Owns a rope handle (spconv_rope_create): the turns of a head's pairs.  It holds
    no device memory and serves every device and stream."""

    def __init__(self, handle: int, head_dim: int):
        self.handle = handle
        self.head_dim = head_dim

    def free(self) -> None:
        if self.handle:
            lib.spconv_rope_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def spconv_rope_create(head_dim: int, layout: str = "interleaved", base: float = 10000.0, freqs=None,
                       axes=None) -> Rope:
    """Rotary positions of heads of ``head_dim`` elements.  ``layout``: "interleaved"
    pairs (2j, 2j + 1), "halves" pairs (j, j + head_dim / 2).  ``freqs`` and ``axes``,
    sequences of head_dim / 2 numbers, give each pair's radians per unit (under 2^64) and its
    coordinate (0, 1, 2 = x, y, z; -1 = the pair does not turn); without them every axis
    has head_dim // 6 pairs with the ladder base^(-j / (head_dim // 6))."""
    _require()
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}")
    if (freqs is None) != (axes is None):
        raise ValueError("freqs and axes are given together or not at all")
    pairs = int(head_dim) // 2
    if freqs is not None:
        freqs, axes = [float(f) for f in freqs], [int(a) for a in axes]
        if len(freqs) != pairs or len(axes) != pairs:
            raise ValueError(f"freqs and axes must have head_dim / 2 = {pairs} entries")
        freqs, axes = (ctypes.c_double * pairs)(*freqs), (ctypes.c_int32 * pairs)(*axes)
    handle = ctypes.c_void_p()
    _check(lib.spconv_rope_create(int(head_dim), ROPE_LAYOUTS[layout], float(base), freqs, axes, ctypes.byref(handle)))
    return Rope(handle.value, int(head_dim))


def spconv_rope_free(rope: Rope) -> None:
    rope.free()


def spconv_rope_apply(rope: Rope, coords: torch.Tensor, x: torch.Tensor, out: torch.Tensor | None = None,
                      inverse: bool = False, stream=None) -> torch.Tensor:
    """Turn the heads x [N, heads, head_dim] by their voxels' coordinates (int32 [N, 4],
    columns b, x, y, z).  x and out may be parts of a packed projection (any strides
    whose heads are contiguous); out may be x itself.  ``inverse`` turns back, which is
    also the gradient."""
    _require()
    if not rope.handle:
        raise ValueError("the rope has been freed")
    shape, dtype, index = x.shape, x.dtype, x.get_device()
    if dtype not in _DTYPES or index < 0 or len(shape) != 3 or shape[2] != rope.head_dim or shape[1] < 1:
        raise ValueError(f"x must be a float32 or bfloat16 CUDA tensor [N, heads, {rope.head_dim}]")
    n, heads, d = shape
    if coords.dtype is not torch.int32 or coords.shape != (n, 4) or coords.get_device() != index:
        raise ValueError(f"coords must be an int32 tensor [{n}, 4] on {x.device}")
    if stream is not None or index != _device_now():
        with _on(x.device, stream):
            return spconv_rope_apply(rope, coords, x, out, inverse)
    row, head, one = x.stride()
    if out is None:
        out = torch.empty_like(x) if x.is_contiguous() else x.new_empty(shape)
    else:
        _like(out, shape, dtype, x.device, "out")
        if out.stride(2) != 1:
            raise ValueError("the heads of out must be contiguous")
    if one != 1 or (n > 1 and row < d) or (heads > 1 and head < d):
        x = x.contiguous()
        row, head, one = x.stride()
    coords = _in(coords)
    out_row, out_head, one = out.stride()
    _check(lib.spconv_rope_apply(rope.handle, _DTYPES[dtype], coords.data_ptr(), n, x.data_ptr(), heads, row, head,
                                 out.data_ptr(), out_row, out_head, bool(inverse), _raw_stream(index)))
    return out


def _w4_args(packed, scales, offsets) -> tuple[int, int, int, int]:
    """(cin, cout, group, device) of 4-bit weights."""
    shape, codes, dtype, index = scales.shape, packed.shape, scales.dtype, scales.get_device()
    if dtype not in _DTYPES or index < 0 or len(shape) != 2:
        raise ValueError("scales must be a float32 or bfloat16 CUDA tensor [Cout, Cin / group]")
    if offsets.shape != shape or offsets.dtype is not dtype or offsets.get_device() != index:
        _like(offsets, shape, dtype, scales.device, "offsets")
    if packed.dtype is not torch.int32 or packed.get_device() != index or len(codes) != 2 or codes[0] != shape[0] \
            or shape[1] < 1 or codes[1] * 8 % shape[1]:
        raise ValueError(f"packed must be an int32 tensor [Cout, Cin / 8] on {scales.device}, with scales "
                         f"[Cout, Cin / group]; got {list(codes)} and {list(shape)}")
    cin = codes[1] * 8
    return cin, codes[0], cin // shape[1], index


def spconv_w4_quantize(w: torch.Tensor, group: int = 64, stream=None) -> tuple:
    """4-bit weights of w [Cin, Cout] (or [1, Cin, Cout], as a layer of kernel size 1
    has them): (packed int32 [Cout, Cin / 8], scales, offsets [Cout, Cin / group])."""
    _require()
    if w.dim() == 3 and w.shape[0] == 1:
        w = w[0]
    if w.dtype not in _DTYPES or not w.is_cuda or w.dim() != 2:
        raise ValueError("w must be a float32 or bfloat16 CUDA tensor [Cin, Cout]")
    cin, cout = w.shape
    if group not in (32, 64, 128) or cin < group or cin % group or cout < 1:
        raise ValueError(f"group must be 32, 64 or 128 and divide Cin = {cin}; Cout must be at least 1")
    if stream is not None or w.get_device() != _device_now():
        with _on(w.device, stream):
            return spconv_w4_quantize(w, group)
    w = _in(w)
    packed = w.new_empty((cout, cin // 8), dtype=torch.int32)
    scales, offsets = w.new_empty((cout, cin // group)), w.new_empty((cout, cin // group))
    _check(lib.spconv_w4_quantize(_DTYPES[w.dtype], w.data_ptr(), cin, cout, group, packed.data_ptr(),
                                  scales.data_ptr(), offsets.data_ptr(), _raw_stream(w.get_device())))
    return packed, scales, offsets


def spconv_w4_dequantize(packed: torch.Tensor, scales: torch.Tensor, offsets: torch.Tensor,
                         out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The weights back, [1, Cin, Cout] of the scales' dtype: the weights of a layer of
    kernel size 1, for more rows than ``spconv_linear_w4`` takes."""
    _require()
    cin, cout, group, index = _w4_args(packed, scales, offsets)
    if stream is not None or index != _device_now():
        with _on(scales.device, stream):
            return spconv_w4_dequantize(packed, scales, offsets, out)
    out = _out(out, scales, (1, cin, cout), scales.dtype, "out")
    packed, scales, offsets = _in(packed), _in(scales), _in(offsets)
    _check(lib.spconv_w4_dequantize(_DTYPES[scales.dtype], packed.data_ptr(), scales.data_ptr(), offsets.data_ptr(),
                                    cin, cout, group, out.data_ptr(), _raw_stream(scales.get_device())))
    return out


def spconv_linear_w4(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, offsets: torch.Tensor,
                     bias: torch.Tensor | None = None, x_scale: torch.Tensor | None = None,
                     out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Linear layer on 4-bit weights for up to W4_MAX_ROWS rows: x [N, Cin] of the
    scales' dtype, or float8_e4m3fn with ``x_scale`` float32 [N] (as
    ``spconv_rms_norm_q8`` returns them) -> out [N, Cout] of the scales' dtype."""
    _require()
    cin, cout, group, index = _w4_args(packed, scales, offsets)
    dtype, n = scales.dtype, x.shape[0] if x.dim() else 0
    if x.shape != (n, cin) or x.dtype is not (dtype if x_scale is None else torch.float8_e4m3fn) \
            or x.get_device() != index:
        _like(x, (n, cin), dtype if x_scale is None else torch.float8_e4m3fn, scales.device, "x")
    if stream is not None or index != _device_now():
        with _on(scales.device, stream):
            return spconv_linear_w4(x, packed, scales, offsets, bias, x_scale, out)
    if x_scale is not None:
        _like(x_scale, (n,), torch.float32, scales.device, "x_scale")
        x_scale = _in(x_scale)
    if bias is not None:
        _like(bias, (cout,), dtype, scales.device, "bias")
        bias = _in(bias)
    out = scales.new_empty((n, cout)) if out is None else _out(out, scales, (n, cout), dtype, "out")
    x, packed, scales, offsets = _in(x), _in(packed), _in(scales), _in(offsets)
    _check(lib.spconv_linear_w4(_DTYPES[dtype], x.data_ptr(), _ptr(x_scale), n, cin, packed.data_ptr(),
                                scales.data_ptr(), offsets.data_ptr(), group, _ptr(bias), out.data_ptr(), cout,
                                _raw_stream(index)))
    return out


def spconv_debug_set_table_slots(slots: int) -> None:
    _require()
    _check(lib.spconv_debug_set_table_slots(int(slots)))


def spconv_debug_set_tile_rows(rows: int) -> None:
    _require()
    _check(lib.spconv_debug_set_tile_rows(int(rows)))


def spconv_debug_set_ring_depths(a_slots: int, b_units: int) -> None:
    _require()
    _check(lib.spconv_debug_set_ring_depths(int(a_slots), int(b_units)))


__all__ = ["OK", "INVALID_ARG", "UNSUPPORTED", "COORD_RANGE", "DUPLICATE", "TABLE_FULL", "OOM", "CUDA_ERROR",
           "TIMEOUT", "SubmMap", "SpconvError", "spconv_build_map", "spconv_subm_forward", "spconv_free",
           "spconv_debug_set_table_slots", "spconv_debug_set_tile_rows", "spconv_debug_set_ring_depths",
           "spconv_build_neighbor_map_noalloc", "lib", "Downsample", "spconv_downsample_build",
           "spconv_downsample_amax", "spconv_upsample", "spconv_subdivide", "MAP_DEFAULT", "MAP_FLIP_KERNEL",
           "MAP_SORTED_KEYS", "MAP_HASH_TABLE", "MAP_SHORT_TILES", "ACTIVATIONS",
           "LIB_PATH", "EXPORTED",
           "ALGO_AUTO", "ALGO_SIMT", "ALGO_TCGEN05", "KERNEL_SIMT", "KERNEL_TCGEN05", "KERNEL_TCGEN05_GEMM",
           "KERNEL_NAMES", "ROPE_INTERLEAVED", "ROPE_HALVES", "ROPE_LAYOUTS", "W4_MAX_ROWS", "Rope", "spconv_rms_norm",
           "spconv_rms_norm_q8", "spconv_rms_norm_backward", "spconv_rope_create", "spconv_rope_free",
           "spconv_rope_apply", "spconv_w4_quantize", "spconv_w4_dequantize", "spconv_linear_w4"]
