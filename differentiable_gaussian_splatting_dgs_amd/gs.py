"""Thin Python binding of the C ABI in include/gs.h (libgs.so).

Argument marshalling only: every step runs in the HIP kernels of libgs.so.
PyTorch supplies device memory (tensors) and the current HIP stream.  If the
library is missing or no GPU is present the calls raise; there is no CPU
fallback.
"""
from __future__ import annotations

import ctypes as C
import math
import os
import struct
from dataclasses import dataclass, field

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libgs.so")

TILE = 16
SPLAT_STRIDE = 12
GRAD2D_STRIDE = 12
SPLAT16_STRIDE = 6  # 4-byte words per 16-bit splat record (24 bytes)


class GsError(RuntimeError):
    pass


class GsCamera(C.Structure):
    _fields_ = [("fx", C.c_double), ("fy", C.c_double), ("cx", C.c_double), ("cy", C.c_double),
                ("width", C.c_int32), ("height", C.c_int32), ("R", C.c_double * 9), ("t", C.c_double * 3)]


class GsSettings(C.Structure):
    _fields_ = [("near_z", C.c_double), ("alpha_min", C.c_double), ("alpha_max", C.c_double),
                ("T_min", C.c_double), ("dilation", C.c_double), ("bg", C.c_double * 3)]


class GsAdamGroup(C.Structure):
    _fields_ = [("param", C.c_void_p), ("grad", C.c_void_p), ("exp_avg", C.c_void_p), ("exp_avg_sq", C.c_void_p),
                ("rows", C.c_int64), ("row_len", C.c_int32), ("col_begin", C.c_int32), ("col_end", C.c_int32),
                ("normalize_rows", C.c_int32), ("lr", C.c_float)]


class GsAdamState(C.Structure):
    _fields_ = [("exp_avg", C.c_void_p * 5), ("exp_avg_sq", C.c_void_p * 5), ("lr", C.c_float * 6),
                ("beta1", C.c_float), ("beta2", C.c_float), ("eps", C.c_float), ("step", C.c_int32)]


class GsDensifyParams(C.Structure):
    _fields_ = [("grad_threshold", C.c_float), ("prune_logit", C.c_float), ("split_log_gap", C.c_float),
                ("split_shrink", C.c_float), ("split_offset", C.c_float), ("clone_offset", C.c_float)]


class GsGaussianSet(C.Structure):
    _fields_ = [("means", C.c_void_p), ("log_scales", C.c_void_p), ("quats", C.c_void_p),
                ("opacity_logits", C.c_void_p), ("sh", C.c_void_p), ("exp_avg", C.c_void_p * 5),
                ("exp_avg_sq", C.c_void_p * 5), ("densify_accum", C.c_void_p), ("densify_count", C.c_void_p)]


class GsLinear(C.Structure):
    _fields_ = [("rows", C.c_int64), ("n_in", C.c_int32), ("n_out", C.c_int32), ("dtype", C.c_int32),
                ("act", C.c_int32), ("ld_x", C.c_int64), ("ld_y", C.c_int64), ("ld_res", C.c_int64),
                ("ld_dx", C.c_int64)]


class GsGradTensor(C.Structure):
    _fields_ = [("grad", C.c_void_p), ("out", C.c_void_p), ("count", C.c_int64), ("dtype", C.c_int32)]


class GsAdamTensor(C.Structure):
    _fields_ = [("param", C.c_void_p), ("grad", C.c_void_p), ("exp_avg", C.c_void_p), ("exp_avg_sq", C.c_void_p),
                ("copy", C.c_void_p), ("rows", C.c_int64), ("row_len", C.c_int32), ("col_begin", C.c_int32),
                ("col_end", C.c_int32), ("normalize_rows", C.c_int32), ("grad_dtype", C.c_int32),
                ("copy_dtype", C.c_int32), ("lr", C.c_float)]


SYMBOLS = ["gs_error_string", "gs_version", "gs_tile_grid", "gs_preprocess", "gs_preprocess_colorjac",
           "gs_bin_workspace_size",
           "gs_bin_sort", "gs_bin_sort_noalloc", "gs_bin_scratch_bytes", "gs_debug_sort_wait_limit", "gs_bin_keys", "gs_render_fwd", "gs_render_fwd_loss",
           "gs_render_bwd", "gs_preprocess_bwd", "gs_preprocess_bwd_colorjac", "gs_preprocess_bwd_adam",
           "gs_image_loss", "gs_densify_accum",
           "gs_adam_step", "gs_count_pairs", "gs_densify_workspace_size", "gs_densify", "gs_opacity_reset",
           "gs_preprocess_views", "gs_bin_workspace_size_views", "gs_bin_sort_views", "gs_render_fwd_views",
           "gs_render_fwd_loss_views", "gs_render_bwd_views", "gs_preprocess_bwd_views",
           "gs_preprocess_bwd_adam_views", "gs_count_pairs_views", "gs_count_nonfinite",
           "gs_preprocess_h16", "gs_render_fwd_h16", "gs_render_bwd_h16", "gs_count_pairs_h16",
           "gs_linear_fwd", "gs_linear_bwd_workspace_size", "gs_linear_bwd", "gs_grad_workspace_size", "gs_grad_norm",
           "gs_grad_clip", "gs_adam_step_clipped"]
MAX_VIEWS = 8
PARAM_ORDER = ("means", "log_scales", "quats", "opacity_logits", "sh")

_lib = None
_vp = C.c_void_p
_i32 = C.c_int32
_i64 = C.c_int64


def load_library(path=LIB_PATH):
    """Load libgs.so (no GPU needed to load it) and declare the signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise GsError(f"{path} is not built: run `python -m differentiable_gaussian_splatting_dgs_amd.build`")
    lib = C.CDLL(path)
    P = C.POINTER
    lib.gs_error_string.restype = C.c_char_p
    lib.gs_error_string.argtypes = [C.c_int]
    lib.gs_version.argtypes = []
    lib.gs_tile_grid.argtypes = [P(GsCamera), P(_i32), P(_i32)]
    lib.gs_preprocess.argtypes = [P(GsCamera), P(GsSettings), _i32, _i32] + [_vp] * 10 + [_vp]
    lib.gs_preprocess_colorjac.argtypes = [P(GsCamera), P(GsSettings), _i32, _i32] + [_vp] * 11 + [_vp]
    lib.gs_bin_workspace_size.argtypes = [_i32, P(GsCamera), _i64, P(C.c_size_t)]
    lib.gs_bin_sort.argtypes = [P(GsCamera), _i32, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, C.c_size_t, _vp]
    lib.gs_bin_keys.argtypes = [P(GsCamera), _vp, _vp, _vp, _vp, _vp]
    lib.gs_debug_sort_wait_limit.argtypes = [_i64]
    lib.gs_bin_sort_noalloc.argtypes = [P(GsCamera), _i32, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp]
    lib.gs_bin_scratch_bytes.argtypes = []
    lib.gs_render_fwd.argtypes = [P(GsCamera), P(GsSettings), _i32] + [_vp] * 9 + [_vp]
    lib.gs_render_fwd_loss.argtypes = [P(GsCamera), P(GsSettings), _i32] + [_vp] * 8 + [_i32] + [_vp] * 4 + [_vp]
    lib.gs_render_bwd.argtypes = [P(GsCamera), P(GsSettings), _i32] + [_vp] * 9 + [_i32, _vp]
    lib.gs_preprocess_bwd.argtypes = [P(GsCamera), P(GsSettings), _i32, _i32] + [_vp] * 13 + [_vp]
    lib.gs_preprocess_bwd_colorjac.argtypes = [P(GsCamera), P(GsSettings), _i32, _i32] + [_vp] * 13 + [_vp]
    lib.gs_preprocess_bwd_adam.argtypes = ([P(GsCamera), P(GsSettings), _i32, _i32] + [_vp] * 8 +
                                           [P(GsAdamState)] + [_vp] * 7 + [_vp])
    lib.gs_image_loss.argtypes = [_i32, _i64, _vp, _vp, _vp, _vp, _vp]
    lib.gs_densify_accum.argtypes = [_i32, _vp, _vp, _vp, _vp, _vp]
    lib.gs_adam_step.argtypes = [_i32, P(GsAdamGroup), C.c_float, C.c_float, C.c_float, _i32, _vp]
    lib.gs_count_pairs.argtypes = [P(GsCamera), P(GsSettings), _i32, _vp, _vp, _vp, _vp, _vp, _vp]
    lib.gs_densify_workspace_size.argtypes = [_i32, P(C.c_size_t)]
    lib.gs_densify.argtypes = [P(GsDensifyParams), _i32, _i32, P(GsGaussianSet), _i64, P(GsGaussianSet),
                               _vp, _vp, _vp, _vp, C.c_size_t, _vp]
    lib.gs_opacity_reset.argtypes = [_i32, C.c_float, _vp, _vp, _vp, _vp]
    V = [P(GsCamera), _i32]
    lib.gs_preprocess_views.argtypes = V + [P(GsSettings), _i32, _i32] + [_vp] * 10 + [_vp]
    lib.gs_bin_workspace_size_views.argtypes = [_i32, P(GsCamera), _i32, _i64, P(C.c_size_t)]
    lib.gs_bin_sort_views.argtypes = V + [_i32, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, C.c_size_t, _vp]
    lib.gs_render_fwd_views.argtypes = V + [P(GsSettings), _i32] + [_vp] * 9 + [_vp]
    lib.gs_render_fwd_loss_views.argtypes = V + [P(GsSettings), _i32] + [_vp] * 8 + [_i32] + [_vp] * 4 + [_vp]
    lib.gs_render_bwd_views.argtypes = V + [P(GsSettings), _i32] + [_vp] * 9 + [_i32, _vp]
    lib.gs_preprocess_bwd_views.argtypes = V + [P(GsSettings), _i32, _i32] + [_vp] * 13 + [_vp]
    lib.gs_preprocess_bwd_adam_views.argtypes = (V + [P(GsSettings), _i32, _i32] + [_vp] * 8 + [P(GsAdamState)] +
                                                 [_vp] * 7 + [_vp])
    lib.gs_count_pairs_views.argtypes = V + [P(GsSettings), _i32, _vp, _vp, _vp, _vp, _vp, _vp]
    lib.gs_count_nonfinite.argtypes = [_vp, _i64, _vp, _vp]
    lib.gs_preprocess_h16.argtypes = [P(GsCamera), P(GsSettings), _i32, _i32] + [_vp] * 11 + [_vp]
    lib.gs_render_fwd_h16.argtypes = [P(GsCamera), P(GsSettings), _i32] + [_vp] * 9 + [_vp]
    lib.gs_render_bwd_h16.argtypes = [P(GsCamera), P(GsSettings), _i32] + [_vp] * 9 + [_i32, _vp]
    lib.gs_count_pairs_h16.argtypes = [P(GsCamera), P(GsSettings), _i32, _vp, _vp, _vp, _vp, _vp, _vp]
    # the descriptors of the network calls go as pointers to packed bytes or to the structures
    lib.gs_linear_fwd.argtypes = [_vp] * 7
    lib.gs_linear_bwd_workspace_size.argtypes = [_vp, P(C.c_size_t)]
    lib.gs_linear_bwd.argtypes = [_vp] * 9 + [C.c_size_t, _vp]
    lib.gs_grad_workspace_size.argtypes = [_i32, P(C.c_size_t)]
    lib.gs_grad_norm.argtypes = [_i32, _vp, C.c_float, _vp, _vp, C.c_size_t, _vp]
    lib.gs_grad_clip.argtypes = [_i32, _vp, C.c_float, _vp, _vp, C.c_size_t, _vp]
    lib.gs_adam_step_clipped.argtypes = [_i32, _vp, C.c_float, C.c_float, C.c_float, _i32, _vp, _vp]
    for name in SYMBOLS:
        if name not in ("gs_error_string",):
            getattr(lib, name).restype = C.c_int
    lib.gs_debug_sort_wait_limit.restype = _i64
    lib.gs_bin_scratch_bytes.restype = _i64
    _lib = lib
    return lib


def _check(rc, name):
    if rc != 0:
        raise GsError(f"{name} failed: {load_library().gs_error_string(rc).decode()} ({rc})")


def _stream():
    return C.c_void_p(torch.cuda.current_stream().cuda_stream)


def _p(t, dtype=None, name="tensor"):
    """Device pointer of a contiguous CUDA tensor (None -> NULL)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise GsError(f"{name} must be a CUDA (HIP) tensor")
    if not t.is_contiguous():
        raise GsError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise GsError(f"{name} must be {dtype}, got {t.dtype}")
    return C.c_void_p(t.data_ptr())


@dataclass
class Settings:
    near_z: float = 0.2
    alpha_min: float = 1.0 / 255.0
    alpha_max: float = 0.99
    T_min: float = 1e-4
    dilation: float = 0.3
    bg: tuple = (0.0, 0.0, 0.0)

    def struct(self):
        s = GsSettings()
        s.near_z, s.alpha_min, s.alpha_max, s.T_min, s.dilation = (self.near_z, self.alpha_min, self.alpha_max,
                                                                   self.T_min, self.dilation)
        for i in range(3):
            s.bg[i] = self.bg[i]
        return s


def camera_struct(cam):
    """From any object with width, height, fx, fy, cx, cy, R [3,3], t [3]."""
    c = GsCamera()
    c.fx, c.fy, c.cx, c.cy = float(cam.fx), float(cam.fy), float(cam.cx), float(cam.cy)
    c.width, c.height = int(cam.width), int(cam.height)
    R = [float(v) for row in cam.R for v in row]
    for i in range(9):
        c.R[i] = R[i]
    for i in range(3):
        c.t[i] = float(cam.t[i])
    return c


# ---------------------------------------------------------------------------
# One wrapper per C entry point, same names.
# ---------------------------------------------------------------------------

def gs_tile_grid(cam):
    tx, ty = _i32(), _i32()
    _check(load_library().gs_tile_grid(C.byref(camera_struct(cam)), C.byref(tx), C.byref(ty)), "gs_tile_grid")
    return tx.value, ty.value


def gs_preprocess(cam, settings, sh_degree, means, log_scales, quats, opacity_logits, sh,
                  splats, depth, rect, tiles_touched, clamp_mask):
    f32, n = torch.float32, means.shape[0]
    rc = load_library().gs_preprocess(
        C.byref(camera_struct(cam)), C.byref(settings.struct()), n, sh_degree,
        _p(means, f32, "means"), _p(log_scales, f32, "log_scales"), _p(quats, f32, "quats"),
        _p(opacity_logits, f32, "opacity_logits"), _p(sh, f32, "sh"), _p(splats, f32, "splats"),
        _p(depth, f32, "depth"), _p(rect, torch.int16, "rect"), _p(tiles_touched, torch.int32, "tiles_touched"),
        _p(clamp_mask, torch.uint8, "clamp_mask"), _stream())
    _check(rc, "gs_preprocess")


def gs_preprocess_colorjac(cam, settings, sh_degree, means, log_scales, quats, opacity_logits, sh,
                           splats, depth, rect, tiles_touched, clamp_mask, colorjac):
    f32, n = torch.float32, means.shape[0]
    rc = load_library().gs_preprocess_colorjac(
        C.byref(camera_struct(cam)), C.byref(settings.struct()), n, sh_degree,
        _p(means, f32, "means"), _p(log_scales, f32, "log_scales"), _p(quats, f32, "quats"),
        _p(opacity_logits, f32, "opacity_logits"), _p(sh, f32, "sh"), _p(splats, f32, "splats"),
        _p(depth, f32, "depth"), _p(rect, torch.int16, "rect"), _p(tiles_touched, torch.int32, "tiles_touched"),
        _p(clamp_mask, torch.uint8, "clamp_mask"), _p(colorjac, f32, "colorjac"), _stream())
    _check(rc, "gs_preprocess_colorjac")


def gs_preprocess_h16(cam, settings, sh_degree, means, log_scales, quats, opacity_logits, sh,
                      splats16, depth, rect, tiles_touched, clamp_mask, colorjac=None):
    """gs_preprocess writing 16-bit splat records (splats16 [n, 6] float32 storage); colorjac optional."""
    f32, n = torch.float32, means.shape[0]
    rc = load_library().gs_preprocess_h16(
        C.byref(camera_struct(cam)), C.byref(settings.struct()), n, sh_degree,
        _p(means, f32, "means"), _p(log_scales, f32, "log_scales"), _p(quats, f32, "quats"),
        _p(opacity_logits, f32, "opacity_logits"), _p(sh, f32, "sh"), _p(splats16, f32, "splats16"),
        _p(depth, f32, "depth"), _p(rect, torch.int16, "rect"), _p(tiles_touched, torch.int32, "tiles_touched"),
        _p(clamp_mask, torch.uint8, "clamp_mask"), _p(colorjac, f32, "colorjac"), _stream())
    _check(rc, "gs_preprocess_h16")


def gs_bin_workspace_size(n, cam, key_capacity):
    b = C.c_size_t()
    _check(load_library().gs_bin_workspace_size(n, C.byref(camera_struct(cam)), key_capacity, C.byref(b)),
           "gs_bin_workspace_size")
    return b.value


def gs_bin_sort(cam, n, depth, rect, tiles_touched, key_capacity, point_list, tile_ranges, num_keys, overflow,
                workspace):
    rc = load_library().gs_bin_sort(
        C.byref(camera_struct(cam)), n, _p(depth, torch.float32, "depth"), _p(rect, torch.int16, "rect"),
        _p(tiles_touched, torch.int32, "tiles_touched"), key_capacity, _p(point_list, torch.int32, "point_list"),
        _p(tile_ranges, torch.int32, "tile_ranges"), _p(num_keys, torch.int32, "num_keys"),
        _p(overflow, torch.int32, "overflow"), _p(workspace, torch.uint8, "workspace"), workspace.numel(), _stream())
    _check(rc, "gs_bin_sort")


def gs_bin_keys(cam, tile_ranges, point_list, depth, keys):
    rc = load_library().gs_bin_keys(C.byref(camera_struct(cam)), _p(tile_ranges, torch.int32), _p(point_list, torch.int32),
                                    _p(depth, torch.float32), _p(keys, torch.int64), _stream())
    _check(rc, "gs_bin_keys")


def gs_bin_sort_noalloc(cam, n, depth, rect, tiles_touched, key_capacity, point_list, tile_ranges, num_keys,
                        overflow):
    """gs_bin_sort on the library's own per-GPU scratch (no workspace, nothing allocated)."""
    rc = load_library().gs_bin_sort_noalloc(
        C.byref(camera_struct(cam)), n, _p(depth, torch.float32, "depth"), _p(rect, torch.int16, "rect"),
        _p(tiles_touched, torch.int32, "tiles_touched"), key_capacity, _p(point_list, torch.int32, "point_list"),
        _p(tile_ranges, torch.int32, "tile_ranges"), _p(num_keys, torch.int32, "num_keys"),
        _p(overflow, torch.int32, "overflow"), _stream())
    _check(rc, "gs_bin_sort_noalloc")


def gs_bin_scratch_bytes():
    return int(load_library().gs_bin_scratch_bytes())


def gs_debug_sort_wait_limit(limit=-1):
    """Sets the radix sort's look-back wait limit for later binning calls (limit < 0:
    leave it); returns the previous limit.  0 makes every sort report failure."""
    return int(load_library().gs_debug_sort_wait_limit(int(limit)))


BIN_OVERFLOW = 1     # bit 0 of the binning status word: more list entries than capacity
BIN_SORT_FAILED = 2  # bit 1: the radix sort gave up waiting; the lists are void


def check_bin_status(word, what="gs_bin_sort"):
    """Reads the status word gs_bin_sort leaves in overflow_dev: raises GsError when the
    sort failed (bit 1), returns True when the lists overflowed their capacity (bit 0)
    and the call should be repeated with a larger one, False when the lists are valid."""
    word = int(word)
    if word & BIN_SORT_FAILED:
        raise GsError(f"{what}: a radix-sort pass gave up waiting for its predecessors; the tile lists are void")
    if word & ~(BIN_OVERFLOW | BIN_SORT_FAILED):
        raise GsError(f"{what}: unknown status word {word:#x}")
    return bool(word & BIN_OVERFLOW)


def gs_render_fwd(cam, settings, n, tile_ranges, point_list, splats, image, final_T, n_contrib, contrib,
                  tile_order=None, grad2d_clear=None):
    rc = load_library().gs_render_fwd(
        C.byref(camera_struct(cam)), C.byref(settings.struct()), n, _p(tile_ranges, torch.int32, "tile_ranges"),
        _p(point_list, torch.int32, "point_list"), _p(splats, torch.float32, "splats"),
        _p(image, torch.float32, "image"), _p(final_T, torch.float32, "final_T"),
        _p(n_contrib, torch.int32, "n_contrib"), _p(contrib, torch.uint8, "contrib"),
        _p(tile_order, torch.int32, "tile_order"), _p(grad2d_clear, torch.float32, "grad2d_clear"), _stream())
    _check(rc, "gs_render_fwd")


def gs_render_fwd_h16(cam, settings, n, tile_ranges, point_list, splats16, image, final_T, n_contrib, contrib,
                      tile_order=None, grad2d_clear=None):
    rc = load_library().gs_render_fwd_h16(
        C.byref(camera_struct(cam)), C.byref(settings.struct()), n, _p(tile_ranges, torch.int32, "tile_ranges"),
        _p(point_list, torch.int32, "point_list"), _p(splats16, torch.float32, "splats16"),
        _p(image, torch.float32, "image"), _p(final_T, torch.float32, "final_T"),
        _p(n_contrib, torch.int32, "n_contrib"), _p(contrib, torch.uint8, "contrib"),
        _p(tile_order, torch.int32, "tile_order"), _p(grad2d_clear, torch.float32, "grad2d_clear"), _stream())
    _check(rc, "gs_render_fwd_h16")


def gs_render_fwd_loss(cam, settings, n, tile_ranges, point_list, splats, image, final_T, n_contrib, contrib,
                       tile_order, mode, target, dL_dimage, loss_dev, grad2d_clear=None):
    """gs_render_fwd with the L1/L2 image loss fused in (loss_dev [1 + tiles] float64; loss_dev[0] = loss)."""
    mode_id = {"l1": 1, "l2": 2}[mode]
    tx, ty = gs_tile_grid(cam)
    if loss_dev.numel() < 1 + tx * ty:
        raise GsError(f"loss buffer needs {1 + tx * ty} float64 entries (1 + tiles)")
    rc = load_library().gs_render_fwd_loss(
        C.byref(camera_struct(cam)), C.byref(settings.struct()), n, _p(tile_ranges, torch.int32, "tile_ranges"),
        _p(point_list, torch.int32, "point_list"), _p(splats, torch.float32, "splats"),
        _p(image, torch.float32, "image"), _p(final_T, torch.float32, "final_T"),
        _p(n_contrib, torch.int32, "n_contrib"), _p(contrib, torch.uint8, "contrib"),
        _p(tile_order, torch.int32, "tile_order"), mode_id, _p(target, torch.float32, "target"),
        _p(dL_dimage, torch.float32, "dL_dimage"), _p(loss_dev, torch.float64, "loss_dev"),
        _p(grad2d_clear, torch.float32, "grad2d_clear"), _stream())
    _check(rc, "gs_render_fwd_loss")


def gs_render_bwd(cam, settings, n, tile_ranges, point_list, splats, final_T, n_contrib, contrib, dL_dimage, grad2d,
                  accumulate=False, tile_order=None):
    rc = load_library().gs_render_bwd(
        C.byref(camera_struct(cam)), C.byref(settings.struct()), n, _p(tile_ranges, torch.int32, "tile_ranges"),
        _p(point_list, torch.int32, "point_list"), _p(splats, torch.float32, "splats"),
        _p(final_T, torch.float32, "final_T"), _p(n_contrib, torch.int32, "n_contrib"),
        _p(contrib, torch.uint8, "contrib"), _p(tile_order, torch.int32, "tile_order"),
        _p(dL_dimage, torch.float32, "dL_dimage"),
        _p(grad2d, torch.float32, "grad2d"), 1 if accumulate else 0, _stream())
    _check(rc, "gs_render_bwd")


def gs_render_bwd_h16(cam, settings, n, tile_ranges, point_list, splats16, final_T, n_contrib, contrib, dL_dimage,
                      grad2d, accumulate=False, tile_order=None):
    rc = load_library().gs_render_bwd_h16(
        C.byref(camera_struct(cam)), C.byref(settings.struct()), n, _p(tile_ranges, torch.int32, "tile_ranges"),
        _p(point_list, torch.int32, "point_list"), _p(splats16, torch.float32, "splats16"),
        _p(final_T, torch.float32, "final_T"), _p(n_contrib, torch.int32, "n_contrib"),
        _p(contrib, torch.uint8, "contrib"), _p(tile_order, torch.int32, "tile_order"),
        _p(dL_dimage, torch.float32, "dL_dimage"),
        _p(grad2d, torch.float32, "grad2d"), 1 if accumulate else 0, _stream())
    _check(rc, "gs_render_bwd_h16")


def gs_preprocess_bwd(cam, settings, sh_degree, means, log_scales, quats, opacity_logits, sh, tiles_touched,
                      clamp_mask, grad2d, dmeans, dlog_scales, dquats, dopacity_logits, dsh):
    f32, n = torch.float32, means.shape[0]
    rc = load_library().gs_preprocess_bwd(
        C.byref(camera_struct(cam)), C.byref(settings.struct()), n, sh_degree,
        _p(means, f32, "means"), _p(log_scales, f32, "log_scales"), _p(quats, f32, "quats"),
        _p(opacity_logits, f32, "opacity_logits"), _p(sh, f32, "sh"),
        _p(tiles_touched, torch.int32, "tiles_touched"), _p(clamp_mask, torch.uint8, "clamp_mask"),
        _p(grad2d, f32, "grad2d"), _p(dmeans, f32, "dmeans"), _p(dlog_scales, f32, "dlog_scales"),
        _p(dquats, f32, "dquats"), _p(dopacity_logits, f32, "dopacity_logits"), _p(dsh, f32, "dsh"), _stream())
    _check(rc, "gs_preprocess_bwd")


def gs_preprocess_bwd_colorjac(cam, settings, sh_degree, means, log_scales, quats, opacity_logits, colorjac,
                               tiles_touched, clamp_mask, grad2d, dmeans, dlog_scales, dquats, dopacity_logits, dsh):
    f32, n = torch.float32, means.shape[0]
    rc = load_library().gs_preprocess_bwd_colorjac(
        C.byref(camera_struct(cam)), C.byref(settings.struct()), n, sh_degree,
        _p(means, f32, "means"), _p(log_scales, f32, "log_scales"), _p(quats, f32, "quats"),
        _p(opacity_logits, f32, "opacity_logits"), _p(colorjac, f32, "colorjac"),
        _p(tiles_touched, torch.int32, "tiles_touched"), _p(clamp_mask, torch.uint8, "clamp_mask"),
        _p(grad2d, f32, "grad2d"), _p(dmeans, f32, "dmeans"), _p(dlog_scales, f32, "dlog_scales"),
        _p(dquats, f32, "dquats"), _p(dopacity_logits, f32, "dopacity_logits"), _p(dsh, f32, "dsh"), _stream())
    _check(rc, "gs_preprocess_bwd_colorjac")


LOSS_PARTIALS = 1024


def gs_preprocess_bwd_adam(cam, settings, sh_degree, params, tiles_touched, clamp_mask, grad2d, exp_avg,
                           exp_avg_sq, lr, step, beta1=0.9, beta2=0.999, eps=1e-8, densify_accum=None,
                           densify_count=None, grads=None):
    """Fused 2D->3D backward + densification statistic + Adam step, updating `params` in place.

    params, exp_avg, exp_avg_sq, grads: dicts keyed by PARAM_ORDER; lr: dict with keys means,
    log_scales, quats, opacity_logits, sh_dc, sh_rest; grads=None skips the gradient writes."""
    f32, n = torch.float32, params["means"].shape[0]
    st = GsAdamState()
    for i, k in enumerate(PARAM_ORDER):
        st.exp_avg[i] = _p(exp_avg[k], f32, "exp_avg." + k).value
        st.exp_avg_sq[i] = _p(exp_avg_sq[k], f32, "exp_avg_sq." + k).value
    for i, k in enumerate(("means", "log_scales", "quats", "opacity_logits", "sh_dc", "sh_rest")):
        st.lr[i] = float(lr[k])
    st.beta1, st.beta2, st.eps, st.step = beta1, beta2, eps, int(step)
    g = grads or {}
    rc = load_library().gs_preprocess_bwd_adam(
        C.byref(camera_struct(cam)), C.byref(settings.struct()), n, sh_degree,
        *[_p(params[k], f32, k) for k in PARAM_ORDER], _p(tiles_touched, torch.int32, "tiles_touched"),
        _p(clamp_mask, torch.uint8, "clamp_mask"), _p(grad2d, f32, "grad2d"), C.byref(st),
        _p(densify_accum, f32, "densify_accum"), _p(densify_count, torch.int32, "densify_count"),
        *[_p(g.get(k), f32, "grad." + k) for k in PARAM_ORDER], _stream())
    _check(rc, "gs_preprocess_bwd_adam")


def _adam_struct(exp_avg, exp_avg_sq, lr, step, beta1, beta2, eps):
    f32 = torch.float32
    st = GsAdamState()
    for i, k in enumerate(PARAM_ORDER):
        if k in exp_avg:
            st.exp_avg[i] = _p(exp_avg[k], f32, "exp_avg." + k).value
            st.exp_avg_sq[i] = _p(exp_avg_sq[k], f32, "exp_avg_sq." + k).value
    for i, k in enumerate(("means", "log_scales", "quats", "opacity_logits", "sh_dc", "sh_rest")):
        st.lr[i] = float(lr[k])
    st.beta1, st.beta2, st.eps, st.step = beta1, beta2, eps, int(step)
    return st


def gs_image_loss(mode, pred, target, dL_dpred, loss):
    """loss: float64 CUDA tensor with at least 1 + LOSS_PARTIALS entries; loss[0] receives L."""
    m = {"l1": 1, "l2": 2}[mode] if isinstance(mode, str) else int(mode)
    if loss.numel() < 1 + LOSS_PARTIALS:
        raise GsError(f"loss buffer needs {1 + LOSS_PARTIALS} float64 entries")
    rc = load_library().gs_image_loss(m, pred.numel(), _p(pred, torch.float32, "pred"),
                                      _p(target, torch.float32, "target"), _p(dL_dpred, torch.float32, "dL_dpred"),
                                      _p(loss, torch.float64, "loss"), _stream())
    _check(rc, "gs_image_loss")


def gs_densify_accum(n, tiles_touched, grad2d, accum, count):
    rc = load_library().gs_densify_accum(n, _p(tiles_touched, torch.int32), _p(grad2d, torch.float32),
                                         _p(accum, torch.float32), _p(count, torch.int32), _stream())
    _check(rc, "gs_densify_accum")


def gs_adam_step(groups, beta1, beta2, eps, step):
    """groups: list of dicts with param, grad, exp_avg, exp_avg_sq (tensors), rows, row_len,
    col_begin, col_end, normalize_rows, lr."""
    arr = (GsAdamGroup * max(len(groups), 1))()
    for i, g in enumerate(groups):
        a = arr[i]
        a.param, a.grad = _p(g["param"], torch.float32).value, _p(g["grad"], torch.float32).value
        a.exp_avg, a.exp_avg_sq = _p(g["exp_avg"], torch.float32).value, _p(g["exp_avg_sq"], torch.float32).value
        a.rows, a.row_len = int(g["rows"]), int(g["row_len"])
        a.col_begin, a.col_end = int(g.get("col_begin", 0)), int(g.get("col_end", g["row_len"]))
        a.normalize_rows, a.lr = int(g.get("normalize_rows", 0)), float(g["lr"])
    rc = load_library().gs_adam_step(len(groups), arr, beta1, beta2, eps, step, _stream())
    _check(rc, "gs_adam_step")


def gs_count_pairs(cam, settings, n, tile_ranges, point_list, splats, counts, evaluated_px=None):
    rc = load_library().gs_count_pairs(C.byref(camera_struct(cam)), C.byref(settings.struct()), n,
                                       _p(tile_ranges, torch.int32), _p(point_list, torch.int32),
                                       _p(splats, torch.float32), _p(counts, torch.int64),
                                       _p(evaluated_px, torch.int32, "evaluated_px"), _stream())
    _check(rc, "gs_count_pairs")


def gs_count_pairs_h16(cam, settings, n, tile_ranges, point_list, splats16, counts, evaluated_px=None):
    rc = load_library().gs_count_pairs_h16(C.byref(camera_struct(cam)), C.byref(settings.struct()), n,
                                           _p(tile_ranges, torch.int32), _p(point_list, torch.int32),
                                           _p(splats16, torch.float32), _p(counts, torch.int64),
                                           _p(evaluated_px, torch.int32, "evaluated_px"), _stream())
    _check(rc, "gs_count_pairs_h16")


def gs_count_nonfinite(x, out=None):
    """Device int64 tensor [1] holding the number of NaN / infinite values of the float32 tensor x."""
    if out is None:
        out = torch.empty(1, dtype=torch.int64, device=x.device)
    _check(load_library().gs_count_nonfinite(_p(x, torch.float32, "x"), x.numel(), _p(out, torch.int64, "out"),
                                             _stream()), "gs_count_nonfinite")
    return out


def check_finite(tensors):
    """Debug check: raise GsError naming every float32 tensor of `tensors` (a dict) that holds NaN or
    infinite values.  Synchronises."""
    bad = []
    for name, t in tensors.items():
        c = int(gs_count_nonfinite(t).item())
        if c:
            bad.append(f"{name} ({c} of {t.numel()})")
    if bad:
        raise GsError("non-finite values in " + ", ".join(bad))


@dataclass
class DensifyParams:
    """The numbers the training notes ([P4] D.1-D.3) leave out, as readings.

    grad_threshold: mean |dL/d(u,v)| (pixels, summed image loss) at or above which a
        Gaussian is densified.  It has no default: it scales with the loss
        normalisation and the image size.  threshold_for(height) gives the value
        matching Kerbl et al.'s 2e-4 (a per-pixel mean L1 of weight 0.8, NDC units):
        2e-4 * 6 * height / 0.8.
    min_opacity: Gaussians below it are removed (Kerbl et al.: 0.005).
    split_ratio: eigenvalue ratio of Sigma at or above which a densified Gaussian is
        split rather than cloned (4: the longest axis twice the shortest).
    split_factor: the children's scales are the parent's divided by it (Kerbl et al.: 1.6).
    split_offset, clone_offset: displacements along the longest axis, in units of
        its scale (children one standard deviation out; the copy a tenth).
    """
    grad_threshold: float
    min_opacity: float = 0.005
    split_ratio: float = 4.0
    split_factor: float = 1.6
    split_offset: float = 1.0
    clone_offset: float = 0.1

    @staticmethod
    def threshold_for(height):
        return 2e-4 * 6.0 * height / 0.8

    def struct(self):
        return GsDensifyParams(self.grad_threshold, math.log(self.min_opacity / (1.0 - self.min_opacity)),
                               0.5 * math.log(self.split_ratio), math.log(self.split_factor), self.split_offset,
                               self.clone_offset)


OPACITY_RESET_FACTOR = 0.3  # [P4] E.1 step 6


def _set_struct(d, with_stats, name):
    """GsGaussianSet from a dict: the five groups, optional 'exp_avg' / 'exp_avg_sq' dicts and
    'densify_accum' / 'densify_count'."""
    f32 = torch.float32
    st = GsGaussianSet()
    for k in PARAM_ORDER:
        setattr(st, k, _p(d.get(k), f32, f"{name}.{k}"))
    for i, k in enumerate(PARAM_ORDER):
        if d.get("exp_avg") is not None:
            st.exp_avg[i] = _p(d["exp_avg"][k], f32, f"{name}.exp_avg.{k}").value
            st.exp_avg_sq[i] = _p(d["exp_avg_sq"][k], f32, f"{name}.exp_avg_sq.{k}").value
    if with_stats:
        st.densify_accum = _p(d.get("densify_accum"), f32, f"{name}.densify_accum")
        st.densify_count = _p(d.get("densify_count"), torch.int32, f"{name}.densify_count")
    return st


def gs_densify_workspace_size(n):
    b = C.c_size_t()
    _check(load_library().gs_densify_workspace_size(n, C.byref(b)), "gs_densify_workspace_size")
    return b.value


def gs_densify(dp, sh_degree, inp, capacity, out, n_out, overflow, workspace, action=None):
    """inp / out: dicts as _set_struct takes; out holds `capacity` rows."""
    n = inp["means"].shape[0]
    rc = load_library().gs_densify(
        C.byref(dp.struct() if isinstance(dp, DensifyParams) else dp), n, sh_degree,
        C.byref(_set_struct(inp, True, "in")), capacity, C.byref(_set_struct(out, True, "out")),
        _p(n_out, torch.int32, "n_out"), _p(overflow, torch.int32, "overflow"), _p(action, torch.uint8, "action"),
        _p(workspace, torch.uint8, "workspace"), workspace.numel(), _stream())
    _check(rc, "gs_densify")


def densify_and_prune(dp, sh_degree, params, densify_accum, densify_count, exp_avg=None, exp_avg_sq=None):
    """Allocates outputs for the worst case (2 n rows), runs gs_densify and returns
    (params, exp_avg, exp_avg_sq, densify_accum, densify_count, action), each trimmed to
    the output count (exp_avg / exp_avg_sq None when not given).  Synchronises once to
    read the count."""
    n = params["means"].shape[0]
    dev = params["means"].device
    cap = 2 * n

    def like(t):
        return torch.empty((cap,) + tuple(t.shape[1:]), dtype=t.dtype, device=dev)

    out = {k: like(params[k]) for k in PARAM_ORDER}
    if exp_avg is not None:
        out["exp_avg"] = {k: like(exp_avg[k]) for k in PARAM_ORDER}
        out["exp_avg_sq"] = {k: like(exp_avg_sq[k]) for k in PARAM_ORDER}
    out["densify_accum"] = like(densify_accum)
    out["densify_count"] = like(densify_count)
    inp = dict(params, densify_accum=densify_accum, densify_count=densify_count, exp_avg=exp_avg,
               exp_avg_sq=exp_avg_sq)
    n_out = torch.zeros(1, dtype=torch.int32, device=dev)
    overflow = torch.zeros(1, dtype=torch.int32, device=dev)
    action = torch.empty(n, dtype=torch.uint8, device=dev)
    ws = torch.empty(max(gs_densify_workspace_size(n), 1) + 256, dtype=torch.uint8, device=dev)
    off = (-ws.data_ptr()) % 256
    gs_densify(dp, sh_degree, inp, cap, out, n_out, overflow, ws[off:off + gs_densify_workspace_size(n)], action)
    m = int(n_out.item())
    if int(overflow.item()):
        raise GsError("gs_densify overflowed a 2 n capacity")
    trim = {k: out[k][:m] for k in PARAM_ORDER}
    ea = {k: out["exp_avg"][k][:m] for k in PARAM_ORDER} if exp_avg is not None else None
    eq = {k: out["exp_avg_sq"][k][:m] for k in PARAM_ORDER} if exp_avg is not None else None
    return trim, ea, eq, out["densify_accum"][:m], out["densify_count"][:m], action


def gs_opacity_reset(opacity_logits, factor=OPACITY_RESET_FACTOR, exp_avg=None, exp_avg_sq=None):
    f32 = torch.float32
    rc = load_library().gs_opacity_reset(opacity_logits.numel(), factor, _p(opacity_logits, f32, "opacity_logits"),
                                         _p(exp_avg, f32, "exp_avg"), _p(exp_avg_sq, f32, "exp_avg_sq"), _stream())
    _check(rc, "gs_opacity_reset")


def camera_array(cams):
    """A C array of GsCamera for the batched (views) calls."""
    cams = list(cams)
    if not 1 <= len(cams) <= MAX_VIEWS:
        raise GsError(f"1 to {MAX_VIEWS} views, got {len(cams)}")
    arr = (GsCamera * len(cams))()
    for i, c in enumerate(cams):
        arr[i] = camera_struct(c)
    return arr, len(cams)


def gs_preprocess_views(cams, settings, sh_degree, params, splats, depth, rect, tiles_touched, clamp_mask):
    """Per-view outputs are [views, n, ...]."""
    f32, n = torch.float32, params["means"].shape[0]
    arr, v = camera_array(cams)
    rc = load_library().gs_preprocess_views(
        arr, v, C.byref(settings.struct()), n, sh_degree, *[_p(params[k], f32, k) for k in PARAM_ORDER],
        _p(splats, f32, "splats"), _p(depth, f32, "depth"), _p(rect, torch.int16, "rect"),
        _p(tiles_touched, torch.int32, "tiles_touched"), _p(clamp_mask, torch.uint8, "clamp_mask"), _stream())
    _check(rc, "gs_preprocess_views")


def gs_bin_workspace_size_views(n, cams, key_capacity):
    arr, v = camera_array(cams)
    b = C.c_size_t()
    _check(load_library().gs_bin_workspace_size_views(n, arr, v, key_capacity, C.byref(b)),
           "gs_bin_workspace_size_views")
    return b.value


def gs_bin_sort_views(cams, n, depth, rect, tiles_touched, key_capacity, point_list, tile_ranges, num_keys,
                      overflow, workspace):
    arr, v = camera_array(cams)
    rc = load_library().gs_bin_sort_views(
        arr, v, n, _p(depth, torch.float32, "depth"), _p(rect, torch.int16, "rect"),
        _p(tiles_touched, torch.int32, "tiles_touched"), key_capacity, _p(point_list, torch.int32, "point_list"),
        _p(tile_ranges, torch.int32, "tile_ranges"), _p(num_keys, torch.int32, "num_keys"),
        _p(overflow, torch.int32, "overflow"), _p(workspace, torch.uint8, "workspace"), workspace.numel(), _stream())
    _check(rc, "gs_bin_sort_views")


def gs_render_fwd_views(cams, settings, n, tile_ranges, point_list, splats, image, final_T, n_contrib, contrib,
                        tile_order=None, mode=None, target=None, dL_dimage=None, loss_dev=None, grad2d_clear=None):
    """Forward blend of a batch of views; with mode ('l1' / 'l2') the image loss is fused in
    (loss_dev [1 + views tiles] float64; loss_dev[0] = the batch's loss)."""
    arr, v = camera_array(cams)
    common = (arr, v, C.byref(settings.struct()), n, _p(tile_ranges, torch.int32, "tile_ranges"),
              _p(point_list, torch.int32, "point_list"), _p(splats, torch.float32, "splats"),
              _p(image, torch.float32, "image"), _p(final_T, torch.float32, "final_T"),
              _p(n_contrib, torch.int32, "n_contrib"), _p(contrib, torch.uint8, "contrib"),
              _p(tile_order, torch.int32, "tile_order"))
    if mode is None:
        _check(load_library().gs_render_fwd_views(*common, _p(grad2d_clear, torch.float32, "grad2d_clear"),
                                                  _stream()), "gs_render_fwd_views")
        return
    tx, ty = gs_tile_grid(cams[0])
    if loss_dev.numel() < 1 + v * tx * ty:
        raise GsError(f"loss buffer needs {1 + v * tx * ty} float64 entries (1 + views tiles)")
    rc = load_library().gs_render_fwd_loss_views(
        *common, {"l1": 1, "l2": 2}[mode], _p(target, torch.float32, "target"),
        _p(dL_dimage, torch.float32, "dL_dimage"), _p(loss_dev, torch.float64, "loss_dev"),
        _p(grad2d_clear, torch.float32, "grad2d_clear"), _stream())
    _check(rc, "gs_render_fwd_loss_views")


def gs_render_fwd_loss_views(cams, settings, n, tile_ranges, point_list, splats, image, final_T, n_contrib,
                             contrib, tile_order, mode, target, dL_dimage, loss_dev, grad2d_clear=None):
    gs_render_fwd_views(cams, settings, n, tile_ranges, point_list, splats, image, final_T, n_contrib, contrib,
                        tile_order, mode, target, dL_dimage, loss_dev, grad2d_clear)


def gs_render_bwd_views(cams, settings, n, tile_ranges, point_list, splats, final_T, n_contrib, contrib, dL_dimage,
                        grad2d, accumulate=False, tile_order=None):
    arr, v = camera_array(cams)
    rc = load_library().gs_render_bwd_views(
        arr, v, C.byref(settings.struct()), n, _p(tile_ranges, torch.int32, "tile_ranges"),
        _p(point_list, torch.int32, "point_list"), _p(splats, torch.float32, "splats"),
        _p(final_T, torch.float32, "final_T"), _p(n_contrib, torch.int32, "n_contrib"),
        _p(contrib, torch.uint8, "contrib"), _p(tile_order, torch.int32, "tile_order"),
        _p(dL_dimage, torch.float32, "dL_dimage"), _p(grad2d, torch.float32, "grad2d"), 1 if accumulate else 0,
        _stream())
    _check(rc, "gs_render_bwd_views")


def gs_preprocess_bwd_views(cams, settings, sh_degree, params, tiles_touched, clamp_mask, grad2d, out):
    """3D gradients summed over the views into out (dict of the five groups)."""
    f32, n = torch.float32, params["means"].shape[0]
    arr, v = camera_array(cams)
    rc = load_library().gs_preprocess_bwd_views(
        arr, v, C.byref(settings.struct()), n, sh_degree, *[_p(params[k], f32, k) for k in PARAM_ORDER],
        _p(tiles_touched, torch.int32, "tiles_touched"), _p(clamp_mask, torch.uint8, "clamp_mask"),
        _p(grad2d, f32, "grad2d"), *[_p(out[k], f32, "d" + k) for k in PARAM_ORDER], _stream())
    _check(rc, "gs_preprocess_bwd_views")


def gs_preprocess_bwd_adam_views(cams, settings, sh_degree, params, tiles_touched, clamp_mask, grad2d, exp_avg,
                                 exp_avg_sq, lr, step, beta1=0.9, beta2=0.999, eps=1e-8, densify_accum=None,
                                 densify_count=None, grads=None):
    """One Adam step with the gradients summed over the views (params updated in place)."""
    f32, n = torch.float32, params["means"].shape[0]
    arr, v = camera_array(cams)
    st = _adam_struct(exp_avg, exp_avg_sq, lr, step, beta1, beta2, eps)
    g = grads or {}
    rc = load_library().gs_preprocess_bwd_adam_views(
        arr, v, C.byref(settings.struct()), n, sh_degree, *[_p(params[k], f32, k) for k in PARAM_ORDER],
        _p(tiles_touched, torch.int32, "tiles_touched"), _p(clamp_mask, torch.uint8, "clamp_mask"),
        _p(grad2d, f32, "grad2d"), C.byref(st), _p(densify_accum, f32, "densify_accum"),
        _p(densify_count, torch.int32, "densify_count"), *[_p(g.get(k), f32, "grad." + k) for k in PARAM_ORDER],
        _stream())
    _check(rc, "gs_preprocess_bwd_adam_views")


def gs_count_pairs_views(cams, settings, n, tile_ranges, point_list, splats, counts, evaluated_px=None):
    arr, v = camera_array(cams)
    rc = load_library().gs_count_pairs_views(arr, v, C.byref(settings.struct()), n, _p(tile_ranges, torch.int32),
                                             _p(point_list, torch.int32), _p(splats, torch.float32),
                                             _p(counts, torch.int64), _p(evaluated_px, torch.int32, "evaluated_px"),
                                             _stream())
    _check(rc, "gs_count_pairs_views")


# ---------------------------------------------------------------------------
# Networks beside the Gaussians: the fused linear layer, gradient clipping and
# the clipped Adam step (the classes over them are in network.py).
# ---------------------------------------------------------------------------

# A layer of a few rows takes a few microseconds on the GPU, so these wrappers keep
# the host's part as short: one look at each property of a tensor, descriptors
# packed in one go (gs_linear, gs_grad_tensor and gs_adam_tensor as bytes).  They run on their tensors' device, on the
# stream that is current there.
# ---------------------------------------------------------------------------

DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}
CLIP_STATE_FLOATS = 4

_pack_linear = struct.Struct("=qiiiiqqqq").pack
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _refuse(t, shape, dtype, name):
    """Raises what is wrong with a tensor that should be a CUDA tensor of this shape and type."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise GsError(f"{name} must be a CUDA (HIP) tensor")
    if dtype is not None and t.dtype != dtype:
        raise GsError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dtype not in DTYPES:
        raise GsError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise GsError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise GsError(f"{name} must be contiguous and on the other tensors' device")


def _rows(t, shape, dtype, device, name):
    """Row stride of a 2-D tensor on that CUDA device whose rows are contiguous."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.get_device() != device:
        _refuse(t, shape, dtype, name)
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] > 1:
        raise GsError(f"{name} must have contiguous rows")
    return s0 if shape[0] > 1 else shape[1]


def _whole(t, shape, dtype, device, name):
    """Device pointer of a contiguous tensor on that CUDA device (None -> NULL)."""
    if t is None:
        return None
    if (not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.get_device() != device or
            not t.is_contiguous()):
        _refuse(t, shape, dtype, name)
    return t.data_ptr()


def _linear_shape(x, w, act):
    """(rows, n_in, n_out, type code, activation code, device, ld_x) of x [rows, n_in] and w [n_out, n_in]."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise GsError("x and w must be 2-D tensors")
    code = DTYPES.get(x.dtype)
    if code is None or not x.is_cuda:
        _refuse(x, None, None, "x")
    a = ACTS.get(act)
    if a is None:
        raise GsError(f"act must be one of {sorted(ACTS)}, got {act!r}")
    shape = x.shape
    rows, n_in = shape
    n_out, w_in = w.shape
    if w_in != n_in:
        raise GsError(f"w must have shape [n_out, {n_in}], got {tuple(w.shape)}")
    device = x.get_device()
    return rows, n_in, n_out, code, a, device, _rows(x, shape, x.dtype, device, "x")


def linear_fwd_into(x, w, bias, residual, y, act):
    """gs_linear_fwd; y None: a new [rows, n_out] tensor.  Returns y."""
    rows, n_in, n_out, code, a, device, ld_x = _linear_shape(x, w, act)
    if device != _current_device():
        with torch.cuda.device(device):
            return linear_fwd_into(x, w, bias, residual, y, act)
    dtype, shape = x.dtype, (rows, n_out)
    if y is None:
        y, ld_y = x.new_empty(shape), n_out
    else:
        ld_y = _rows(y, shape, dtype, device, "y")
    pr, ld_res = None, 0
    if residual is not None:
        ld_res = _rows(residual, shape, dtype, device, "residual")
        pr = residual.data_ptr()
    rc = (_lib or load_library()).gs_linear_fwd(
        _pack_linear(rows, n_in, n_out, code, a, ld_x, ld_y, ld_res, 0), x.data_ptr(),
        _whole(w, w.shape, dtype, device, "w"), _whole(bias, (n_out,), dtype, device, "bias"), pr, y.data_ptr(),
        _raw_stream(device))
    if rc:
        _check(rc, "gs_linear_fwd")
    return y


def gs_linear_fwd(x, w, bias, residual, y, act="none"):
    """y [rows, n_out] = act(x w^T + bias) + residual; bias and residual may be None.  Rows of x, residual and y
    may be strided; a residual with row stride 0 is one row for all."""
    linear_fwd_into(x, w, bias, residual, y, act)


def gs_linear_bwd_workspace_size(x, w, act="none"):
    rows, n_in, n_out, code, a, _, _ = _linear_shape(x, w, act)
    b = C.c_size_t()
    _check(load_library().gs_linear_bwd_workspace_size(_pack_linear(rows, n_in, n_out, code, a, 0, 0, 0, 0),
                                                       C.byref(b)), "gs_linear_bwd_workspace_size")
    return b.value


def linear_bwd_into(x, w, bias, dy, dx, dw, db, workspace, act):
    """gs_linear_bwd; workspace None: one of the size the call needs."""
    rows, n_in, n_out, code, a, device, ld_x = _linear_shape(x, w, act)
    if device != _current_device():
        with torch.cuda.device(device):
            return linear_bwd_into(x, w, bias, dy, dx, dw, db, workspace, act)
    dtype = x.dtype
    ld_y = _rows(dy, (rows, n_out), dtype, device, "dy")
    pdx, ld_dx = None, 0
    if dx is not None:
        ld_dx = _rows(dx, (rows, n_in), dtype, device, "dx")
        pdx = dx.data_ptr()
    lib = _lib or load_library()
    d = _pack_linear(rows, n_in, n_out, code, a, ld_x, ld_y, 0, ld_dx)
    if workspace is None:
        b = C.c_size_t()
        _check(lib.gs_linear_bwd_workspace_size(d, C.byref(b)), "gs_linear_bwd_workspace_size")
        # torch's device allocations start at multiples of 512 bytes
        workspace = torch.empty(b.value, dtype=torch.uint8, device=x.device)
    rc = lib.gs_linear_bwd(
        d, x.data_ptr(), _whole(w, w.shape, dtype, device, "w"), _whole(bias, (n_out,), dtype, device, "bias"),
        dy.data_ptr(), pdx, _whole(dw, w.shape, dtype, device, "dw"), _whole(db, (n_out,), dtype, device, "db"),
        _whole(workspace, workspace.shape, torch.uint8, device, "workspace"), workspace.numel(),
        _raw_stream(device))
    if rc:
        _check(rc, "gs_linear_bwd")


def gs_linear_bwd(x, w, bias, dy, dx, dw, db, workspace, act="none"):
    """The layer's gradients from dy [rows, n_out] into dx, dw and db (each may be None: not computed);
    workspace: uint8, gs_linear_bwd_workspace_size bytes, 256-byte aligned."""
    linear_bwd_into(x, w, bias, dy, dx, dw, db, workspace, act)


def gs_grad_workspace_size(n_tensors):
    b = C.c_size_t()
    _check(load_library().gs_grad_workspace_size(n_tensors, C.byref(b)), "gs_grad_workspace_size")
    return b.value


def _grad_table(grads, out):
    """The gs_grad_tensor array of a list of gradients, as bytes."""
    flat, codes = [], DTYPES
    try:
        device = grads[0].get_device() if grads else 0
        if out is None or out is grads:
            for g in grads:
                if not g.is_contiguous() or g.get_device() != device:
                    _refuse(g, None, None, "a gradient")
                p = g.data_ptr()
                flat += (p, p if out is grads else 0, g.numel(), codes[g.dtype])
        else:
            for g, o in zip(grads, out):
                n, dtype = g.numel(), g.dtype
                if not g.is_contiguous() or g.get_device() != device:
                    _refuse(g, None, None, "a gradient")
                if not o.is_contiguous() or o.get_device() != device or o.numel() != n or o.dtype != dtype:
                    _refuse(o, g.shape, dtype, "an output")
                flat += (g.data_ptr(), o.data_ptr(), n, codes[dtype])
    except (AttributeError, KeyError):
        raise GsError("gradients must be float32, float16 or bfloat16 tensors") from None
    if device < 0:
        raise GsError("gradients must be CUDA (HIP) tensors")
    return struct.pack("=%dq" % len(flat), *flat)


def _clip_state(clip):
    if clip.numel() != CLIP_STATE_FLOATS:
        raise GsError(f"the clipping state holds {CLIP_STATE_FLOATS} floats")
    return _p(clip, torch.float32, "clip")


def _clip_device(grads, clip, workspace):
    """The one device of a clipping call's tensors (each list's tensors are compared with each other in its table)."""
    _p(clip, None, "clip")
    device = clip.get_device()
    if workspace.get_device() != device or (grads and grads[0].get_device() != device):
        raise GsError("gradients, clipping state and workspace must be on one device")
    return device


def gs_grad_norm(grads, max_norm, clip, workspace):
    """Global norm and clipping coefficient of the list grads into clip [4] float32 (words 0 and 1)."""
    table, device = _grad_table(grads, None), _clip_device(grads, clip, workspace)
    if device != _current_device():
        with torch.cuda.device(device):
            return grad_norm_table(len(grads), table, max_norm, clip, workspace)
    grad_norm_table(len(grads), table, max_norm, clip, workspace)


def grad_norm_table(n, table, max_norm, clip, workspace):
    """gs_grad_norm of n packed gs_grad_tensor descriptors of the current device."""
    rc = (_lib or load_library()).gs_grad_norm(n, table, max_norm, _clip_state(clip),
                                               _p(workspace, torch.uint8, "workspace"), workspace.numel(),
                                               _raw_stream(_current_device()))
    _check(rc, "gs_grad_norm")


def gs_grad_clip(grads, out, max_norm, clip, workspace):
    """gs_grad_norm, then out[i] = coefficient * grads[i] (out may be grads itself)."""
    if len(out) != len(grads):
        raise GsError("out needs one tensor for each gradient")
    device = _clip_device(grads, clip, workspace)
    if device != _current_device():
        with torch.cuda.device(device):
            return gs_grad_clip(grads, out, max_norm, clip, workspace)
    rc = (_lib or load_library()).gs_grad_clip(len(grads), _grad_table(grads, out), max_norm, _clip_state(clip),
                                               _p(workspace, torch.uint8, "workspace"), workspace.numel(),
                                               _raw_stream(_current_device()))
    _check(rc, "gs_grad_clip")


def gs_adam_step_clipped(tensors, beta1, beta2, eps, step, clip=None):
    """One Adam step on coefficient * gradient for a ctypes array of GsAdamTensor of the current device; clip: the
    state of gs_grad_norm, or None."""
    rc = (_lib or load_library()).gs_adam_step_clipped(len(tensors), tensors, beta1, beta2, eps, step,
                                                       None if clip is None else _clip_state(clip),
                                                       _raw_stream(_current_device()))
    _check(rc, "gs_adam_step_clipped")


# ---------------------------------------------------------------------------
# Buffer owner for one camera and one Gaussian count (plumbing: allocation).
# ---------------------------------------------------------------------------

class Rasterizer:
    """Owns the forward/backward buffers of one view and runs the C ABI calls.

    forward(params) runs gs_preprocess, gs_bin_sort and gs_render_fwd;
    backward(params, dL_dimage) runs gs_render_bwd and gs_preprocess_bwd.
    With colorjac (the default, at SH degree >= 1) the preprocess is
    gs_preprocess_colorjac and the 2D -> 3D backward gs_preprocess_bwd_colorjac:
    the forward keeps each Gaussian's colour gradient with respect to the view
    direction (9 floats), so the backward does not read the SH coefficients again.
    The number of (tile, Gaussian) pairs K is data dependent: the list buffer has
    `key_capacity` entries and binning raises a device flag when K exceeds it.
    `forward(check=True)` synchronises once, grows the capacity and re-bins when
    that happened, and raises GsError when binning reports a failed sort; with
    check=False nothing synchronises (check_bin_status(r.overflow.item()) does
    the same check later).
    debug=True checks the parameters before the forward, and the image and the
    gradients after each pass, for NaN and infinite values (gs_count_nonfinite),
    raising GsError with the names of the tensors that hold them.
    record16=True keeps 16-bit splat records (gs_preprocess_h16 and the _h16
    blends): the blends gather 24 bytes per list entry instead of 48, and compute
    with the conic factor, opacity and colour rounded to binary16.
    """

    def __init__(self, cam, n, sh_degree, settings=None, key_capacity=None, device="cuda", debug=False,
                 colorjac=True, record16=False):
        load_library()
        self.cam, self.n, self.deg = cam, int(n), int(sh_degree)
        self.debug = bool(debug)
        self.settings = settings or Settings()
        self.device = torch.device(device)
        dev, n = self.device, self.n
        self.tiles_x, self.tiles_y = gs_tile_grid(cam)
        self.ntiles = self.tiles_x * self.tiles_y
        self.record16 = bool(record16)
        self.splats = torch.empty((n, SPLAT16_STRIDE if self.record16 else SPLAT_STRIDE), dtype=torch.float32,
                                  device=dev)
        self.depth = torch.empty(n, dtype=torch.float32, device=dev)
        self.rect = torch.empty((n, 4), dtype=torch.int16, device=dev)
        self.tiles_touched = torch.empty(n, dtype=torch.int32, device=dev)
        self.clamp = torch.empty(n, dtype=torch.uint8, device=dev)
        self.tile_ranges = torch.empty((self.ntiles, 2), dtype=torch.int32, device=dev)
        # row 0: forward schedule, row 1: backward schedule (written by the forward)
        self.tile_order = torch.empty((2, self.ntiles), dtype=torch.int32, device=dev)
        self.num_keys = torch.zeros(1, dtype=torch.int32, device=dev)
        self.overflow = torch.zeros(1, dtype=torch.int32, device=dev)
        H, W = cam.height, cam.width
        self.image = torch.empty((3, H, W), dtype=torch.float32, device=dev)
        self.final_T = torch.empty((H, W), dtype=torch.float32, device=dev)
        self.n_contrib = torch.empty((H, W), dtype=torch.int32, device=dev)
        self.grad2d = torch.empty((n, GRAD2D_STRIDE), dtype=torch.float32, device=dev)
        self.colorjac = (torch.empty((n, 9), dtype=torch.float32, device=dev)
                         if colorjac and self.deg > 0 else None)
        self.generation = 0  # forward passes run so far; the autograd wrapper checks it
        self._alloc_lists(key_capacity if key_capacity is not None else max(4 * n, 1 << 16))

    def _alloc_lists(self, cap):
        self.key_capacity = int(cap)
        self.point_list = torch.empty(max(self.key_capacity, 1), dtype=torch.int32, device=self.device)
        self.contrib = torch.empty(max(self.key_capacity, 1), dtype=torch.uint8, device=self.device)
        ws = gs_bin_workspace_size(self.n, self.cam, self.key_capacity)
        self.workspace = torch.empty(ws + 256, dtype=torch.uint8, device=self.device)
        off = (-self.workspace.data_ptr()) % 256
        self.workspace = self.workspace[off:off + ws]

    def preprocess(self, p):
        if self.record16:
            gs_preprocess_h16(self.cam, self.settings, self.deg, p["means"], p["log_scales"], p["quats"],
                              p["opacity_logits"], p["sh"], self.splats, self.depth, self.rect,
                              self.tiles_touched, self.clamp, self.colorjac)
        elif self.colorjac is not None:
            gs_preprocess_colorjac(self.cam, self.settings, self.deg, p["means"], p["log_scales"], p["quats"],
                                   p["opacity_logits"], p["sh"], self.splats, self.depth, self.rect,
                                   self.tiles_touched, self.clamp, self.colorjac)
        else:
            gs_preprocess(self.cam, self.settings, self.deg, p["means"], p["log_scales"], p["quats"],
                          p["opacity_logits"], p["sh"], self.splats, self.depth, self.rect, self.tiles_touched,
                          self.clamp)

    def bin(self):
        gs_bin_sort(self.cam, self.n, self.depth, self.rect, self.tiles_touched, self.key_capacity, self.point_list,
                    self.tile_ranges, self.num_keys, self.overflow, self.workspace)

    def render(self, clear_grad2d=False):
        """Forward blend; with clear_grad2d the 2D-gradient buffer is zeroed by the same kernel, for
        backward_2d(..., accumulate=True)."""
        fwd = gs_render_fwd_h16 if self.record16 else gs_render_fwd
        fwd(self.cam, self.settings, self.n, self.tile_ranges, self.point_list, self.splats, self.image,
            self.final_T, self.n_contrib, self.contrib, self.tile_order, self.grad2d if clear_grad2d else None)

    def render_loss(self, target, mode, dL_dimage, loss_dev, clear_grad2d=True):
        """Forward blend with the fused image loss; with clear_grad2d the 2D-gradient buffer is zeroed too,
        for backward_2d(..., accumulate=True).  loss_dev: [1 + ntiles] float64."""
        if self.record16:
            raise GsError("the fused-loss forward reads float32 splat records (record16=False)")
        gs_render_fwd_loss(self.cam, self.settings, self.n, self.tile_ranges, self.point_list, self.splats,
                           self.image, self.final_T, self.n_contrib, self.contrib, self.tile_order, mode, target,
                           dL_dimage, loss_dev, self.grad2d if clear_grad2d else None)

    def forward(self, p, check=True):
        if self.debug:
            check_finite({k: p[k] for k in PARAM_ORDER})
        self.generation += 1
        self.preprocess(p)
        self.bin()
        if check and check_bin_status(self.overflow.item()):
            K = int(self.num_keys.item())
            self._alloc_lists(int(K * 1.25) + 1024)
            self.bin()
            if check_bin_status(self.overflow.item()):
                raise GsError("gs_bin_sort overflowed a capacity of 1.25 K")
        self.render()
        if self.debug:
            check_finite({"image": self.image, "final_T": self.final_T})
        return self.image

    def backward_2d(self, dL_dimage, accumulate=False):
        bwd = gs_render_bwd_h16 if self.record16 else gs_render_bwd
        bwd(self.cam, self.settings, self.n, self.tile_ranges, self.point_list, self.splats, self.final_T,
            self.n_contrib, self.contrib, dL_dimage, self.grad2d, accumulate, self.tile_order[1])
        return self.grad2d

    def backward_3d(self, p, out):
        """The 2D -> 3D backward of the last forward's parameters p into out (from self.grad2d)."""
        if self.colorjac is not None:
            gs_preprocess_bwd_colorjac(self.cam, self.settings, self.deg, p["means"], p["log_scales"], p["quats"],
                                       p["opacity_logits"], self.colorjac, self.tiles_touched, self.clamp,
                                       self.grad2d, out["means"], out["log_scales"], out["quats"],
                                       out["opacity_logits"], out["sh"])
        else:
            gs_preprocess_bwd(self.cam, self.settings, self.deg, p["means"], p["log_scales"], p["quats"],
                              p["opacity_logits"], p["sh"], self.tiles_touched, self.clamp, self.grad2d,
                              out["means"], out["log_scales"], out["quats"], out["opacity_logits"], out["sh"])
        return out

    def backward(self, p, dL_dimage, out=None):
        self.backward_2d(dL_dimage)
        if out is None:
            out = {k: torch.empty_like(p[k]) for k in ("means", "log_scales", "quats", "opacity_logits", "sh")}
        self.backward_3d(p, out)
        if self.debug:
            check_finite({"dL_dimage": dL_dimage, "grad2d": self.grad2d, **{"d" + k: v for k, v in out.items()}})
        return out

    def count_pairs(self, per_pixel=False):
        """Device int64 [3]: evaluated, walked and blended pairs; with per_pixel also the [H, W]
        int32 evaluated count of each pixel."""
        c = torch.zeros(3, dtype=torch.int64, device=self.device)
        ev = torch.empty_like(self.n_contrib) if per_pixel else None
        count = gs_count_pairs_h16 if self.record16 else gs_count_pairs
        count(self.cam, self.settings, self.n, self.tile_ranges, self.point_list, self.splats, c, ev)
        return (c, ev) if per_pixel else c


class OnceFunction(torch.autograd.Function):
    """Hands a gradient on, and raises when it is differentiated itself."""

    @staticmethod
    def forward(ctx, name, grad, *inputs):
        ctx.name = name
        return grad.detach()

    @staticmethod
    def backward(ctx, _):
        raise GsError(f"{ctx.name} can be differentiated once: its gradients have no derivatives")


def differentiated_once(name, grads, inputs):
    """grads of a backward that the kernels made, for the autograd graph.  Under create_graph they hang on inputs, the
    tensors that they depend on, by a node that raises: without it they would be constants in a second derivative."""
    if not torch.is_grad_enabled():
        return grads
    return tuple(g if g is None else OnceFunction.apply(name, g, *inputs) for g in grads)


class RasterizeFunction(torch.autograd.Function):
    """image = rasterize(means, log_scales, quats, opacity_logits, sh) for one Rasterizer.

    The backward reuses the forward's intermediates (lists, ranges, final_T,
    n_contrib, flags), which the Rasterizer keeps in its own buffers: one
    backward per forward, before the Rasterizer renders again.  A backward after
    a newer forward on the same Rasterizer raises GsError, and so does a second
    derivative."""

    @staticmethod
    def forward(ctx, rast, means, log_scales, quats, opacity_logits, sh):
        p = dict(means=means.contiguous(), log_scales=log_scales.contiguous(), quats=quats.contiguous(),
                 opacity_logits=opacity_logits.contiguous(), sh=sh.contiguous())
        img = rast.forward(p).clone()
        ctx.rast = rast
        ctx.generation = rast.generation
        ctx.save_for_backward(p["means"], p["log_scales"], p["quats"], p["opacity_logits"], p["sh"])
        return img

    @staticmethod
    def backward(ctx, dL_dimage):
        if ctx.rast.generation != ctx.generation:
            raise GsError("rasterize: the Rasterizer ran another forward pass since this one; its buffers no "
                          "longer hold this pass's intermediates (use one Rasterizer per pending backward)")
        m, s, q, o, c = ctx.saved_tensors
        p = dict(means=m, log_scales=s, quats=q, opacity_logits=o, sh=c)
        g = ctx.rast.backward(p, dL_dimage.contiguous())
        return None, *differentiated_once("rasterize", [g[k] for k in PARAM_ORDER], (dL_dimage, m, s, q, o, c))


def rasterize(rast, means, log_scales, quats, opacity_logits, sh):
    # contiguous out here: a copy that the function makes has no place in the graph
    return RasterizeFunction.apply(rast, *(t.contiguous() for t in (means, log_scales, quats, opacity_logits, sh)))


class RasterizerViews:
    """Buffers of a batch of views of one Gaussian set ([P4] E.1: render a batch of
    views, sum the losses, one optimizer step), all through the *_views calls.
    Per-view arrays have a leading views dimension; list entries index
    splats.view(-1, 12), i.e. entry v n + i is Gaussian i in view v."""

    def __init__(self, cams, n, sh_degree, settings=None, key_capacity=None, device="cuda"):
        load_library()
        self.cams = list(cams)
        self.views = len(self.cams)
        camera_array(self.cams)  # checks the count
        cam = self.cams[0]
        if any(c.width != cam.width or c.height != cam.height for c in self.cams):
            raise GsError("the views of a batch must share one image size")
        self.n, self.deg = int(n), int(sh_degree)
        self.settings = settings or Settings()
        self.device = torch.device(device)
        dev, n, V = self.device, self.n, self.views
        self.tiles_x, self.tiles_y = gs_tile_grid(cam)
        self.ntiles = V * self.tiles_x * self.tiles_y
        self.splats = torch.empty((V, n, SPLAT_STRIDE), dtype=torch.float32, device=dev)
        self.depth = torch.empty((V, n), dtype=torch.float32, device=dev)
        self.rect = torch.empty((V, n, 4), dtype=torch.int16, device=dev)
        self.tiles_touched = torch.empty((V, n), dtype=torch.int32, device=dev)
        self.clamp = torch.empty((V, n), dtype=torch.uint8, device=dev)
        self.tile_ranges = torch.empty((self.ntiles, 2), dtype=torch.int32, device=dev)
        self.tile_order = torch.empty((2, self.ntiles), dtype=torch.int32, device=dev)
        self.num_keys = torch.zeros(1, dtype=torch.int32, device=dev)
        self.overflow = torch.zeros(1, dtype=torch.int32, device=dev)
        H, W = cam.height, cam.width
        self.image = torch.empty((V, 3, H, W), dtype=torch.float32, device=dev)
        self.final_T = torch.empty((V, H, W), dtype=torch.float32, device=dev)
        self.n_contrib = torch.empty((V, H, W), dtype=torch.int32, device=dev)
        self.grad2d = torch.empty((V, n, GRAD2D_STRIDE), dtype=torch.float32, device=dev)
        self._alloc_lists(key_capacity if key_capacity is not None else max(4 * n * V, 1 << 16))

    def _alloc_lists(self, cap):
        self.key_capacity = int(cap)
        self.point_list = torch.empty(max(self.key_capacity, 1), dtype=torch.int32, device=self.device)
        self.contrib = torch.empty(max(self.key_capacity, 1), dtype=torch.uint8, device=self.device)
        ws = gs_bin_workspace_size_views(self.n, self.cams, self.key_capacity)
        self.workspace = torch.empty(ws + 256, dtype=torch.uint8, device=self.device)
        off = (-self.workspace.data_ptr()) % 256
        self.workspace = self.workspace[off:off + ws]

    def preprocess(self, p):
        gs_preprocess_views(self.cams, self.settings, self.deg, p, self.splats, self.depth, self.rect,
                            self.tiles_touched, self.clamp)

    def bin(self):
        gs_bin_sort_views(self.cams, self.n, self.depth, self.rect, self.tiles_touched, self.key_capacity,
                          self.point_list, self.tile_ranges, self.num_keys, self.overflow, self.workspace)

    def render(self):
        gs_render_fwd_views(self.cams, self.settings, self.n, self.tile_ranges, self.point_list, self.splats,
                            self.image, self.final_T, self.n_contrib, self.contrib, self.tile_order)

    def render_loss(self, target, mode, dL_dimage, loss_dev, clear_grad2d=True):
        """loss_dev: [1 + views tiles] float64; loss_dev[0] = the loss summed over the views."""
        gs_render_fwd_views(self.cams, self.settings, self.n, self.tile_ranges, self.point_list, self.splats,
                            self.image, self.final_T, self.n_contrib, self.contrib, self.tile_order, mode, target,
                            dL_dimage, loss_dev, self.grad2d if clear_grad2d else None)

    def forward(self, p, check=True):
        self.preprocess(p)
        self.bin()
        if check and check_bin_status(self.overflow.item(), "gs_bin_sort_views"):
            K = int(self.num_keys.item())
            self._alloc_lists(int(K * 1.25) + 1024)
            self.bin()
            if check_bin_status(self.overflow.item(), "gs_bin_sort_views"):
                raise GsError("gs_bin_sort_views overflowed a capacity of 1.25 K")
        self.render()
        return self.image

    def backward_2d(self, dL_dimage, accumulate=False):
        gs_render_bwd_views(self.cams, self.settings, self.n, self.tile_ranges, self.point_list, self.splats,
                            self.final_T, self.n_contrib, self.contrib, dL_dimage, self.grad2d, accumulate,
                            self.tile_order[1])
        return self.grad2d

    def backward(self, p, dL_dimage, out=None):
        """3D gradients of sum_v <dL_dimage[v], image[v]>, summed over the views."""
        self.backward_2d(dL_dimage)
        if out is None:
            out = {k: torch.empty_like(p[k]) for k in PARAM_ORDER}
        gs_preprocess_bwd_views(self.cams, self.settings, self.deg, p, self.tiles_touched, self.clamp, self.grad2d,
                                out)
        return out

    def count_pairs(self):
        c = torch.zeros(3, dtype=torch.int64, device=self.device)
        gs_count_pairs_views(self.cams, self.settings, self.n, self.tile_ranges, self.point_list, self.splats, c)
        return c


class Trainer:
    """The training loop of one view over the library's calls ([P4] E.1): each
    iteration renders with the image loss fused into the forward, back-propagates,
    and takes the fused 2D->3D backward + densification statistic + Adam step
    (bias-corrected at the iteration count); every `densify_interval` iterations
    the Gaussians are densified and pruned (N changes: the Rasterizer is rebuilt
    for the new count, the Adam moments follow their rows, the statistic
    restarts), and every `reset_interval` iterations every opacity is scaled by
    `reset_factor` (the opacity's moments restart).

    With max_grad_norm the five gradients are clipped to that global norm first: the
    2D -> 3D backward writes them (gs_preprocess_bwd), and the Adam step takes the
    clipping coefficient on the device (gs_grad_norm, gs_adam_step_clipped);
    clip[0] holds the last norm before clipping.

    Plumbing only: buffers and the order of the calls.  params: dict of device
    tensors (updated in place between densifications, replaced at them)."""

    def __init__(self, cam, params, sh_degree, target, lr, densify=None, densify_interval=100,
                 reset_interval=3000, reset_factor=OPACITY_RESET_FACTOR, loss="l1", settings=None,
                 max_grad_norm=None):
        self.cam, self.deg, self.lr = cam, int(sh_degree), dict(lr)
        self.target, self.loss_mode = target, loss
        self.densify_params = densify
        self.densify_interval, self.reset_interval, self.reset_factor = densify_interval, reset_interval, reset_factor
        self.settings = settings or Settings()
        self.p = {k: params[k].contiguous() for k in PARAM_ORDER}
        self.m = {k: torch.zeros_like(v) for k, v in self.p.items()}
        self.v = {k: torch.zeros_like(v) for k, v in self.p.items()}
        self.max_grad_norm = None if max_grad_norm is None else float(max_grad_norm)
        if self.max_grad_norm is not None and not self.max_grad_norm >= 0:
            raise GsError("max_grad_norm must be >= 0")
        self.t = 0
        self.events = []  # (iteration, "densify" | "reset", detail)
        self._rebuild()

    @property
    def n(self):
        return self.p["means"].shape[0]

    def _rebuild(self):
        dev = self.p["means"].device
        self.rast = Rasterizer(self.cam, self.n, self.deg, settings=self.settings, device=dev, colorjac=False)
        self.accum = torch.zeros(self.n, dtype=torch.float32, device=dev)
        self.count = torch.zeros(self.n, dtype=torch.int32, device=dev)
        self.dL = torch.empty_like(self.target)
        self.loss = torch.zeros(1 + self.rast.ntiles, dtype=torch.float64, device=dev)
        if self.max_grad_norm is not None:
            self.clip = torch.zeros(CLIP_STATE_FLOATS, dtype=torch.float32, device=dev)
            self.clip_workspace = torch.empty(gs_grad_workspace_size(len(PARAM_ORDER)), dtype=torch.uint8, device=dev)
            self.grads = {k: torch.empty_like(v) for k, v in self.p.items()}
        self._sized = False

    def step(self, dL_hook=None, grads=None, after_update=None):
        """One iteration.  dL_hook(dL), if given, sees (and may change in place) the loss gradient
        the forward wrote before the backward reads it; grads (dict of tensors shaped like the
        parameters) receives the iteration's 3D gradients; after_update(self) runs after the Adam
        update and before densification and the opacity reset."""
        r = self.rast
        r.generation += 1
        r.preprocess(self.p)
        r.bin()
        if not self._sized or dL_hook is not None:  # size the lists on the first pass after a rebuild
            if check_bin_status(r.overflow.item()):
                r._alloc_lists(int(int(r.num_keys.item()) * 1.25) + 1024)
                r.bin()
                if check_bin_status(r.overflow.item()):
                    raise GsError("gs_bin_sort overflowed a capacity of 1.25 K")
            self._sized = True
        r.render_loss(self.target, self.loss_mode, self.dL, self.loss, clear_grad2d=True)
        if dL_hook is not None:
            dL_hook(self.dL)
        r.backward_2d(self.dL, accumulate=True)
        self.t += 1
        if self.max_grad_norm is None:
            gs_preprocess_bwd_adam(self.cam, self.settings, self.deg, self.p, r.tiles_touched, r.clamp, r.grad2d,
                                   self.m, self.v, self.lr, self.t, densify_accum=self.accum,
                                   densify_count=self.count, grads=grads)
        else:
            self._clipped_update(self.grads if grads is None else grads)
        if after_update is not None:
            after_update(self)
        if self.densify_params is not None and self.densify_interval and self.t % self.densify_interval == 0:
            self.densify()
        if self.reset_interval and self.t % self.reset_interval == 0:
            self.reset_opacity()

    def _clipped_update(self, g):
        """The 2D -> 3D backward into g, the densification statistic, the global norm and the clipped Adam step."""
        r, p = self.rast, self.p
        gs_preprocess_bwd(self.cam, self.settings, self.deg, p["means"], p["log_scales"], p["quats"],
                          p["opacity_logits"], p["sh"], r.tiles_touched, r.clamp, r.grad2d, *[g[k] for k in PARAM_ORDER])
        gs_densify_accum(self.n, r.tiles_touched, r.grad2d, self.accum, self.count)
        gs_grad_norm([g[k] for k in PARAM_ORDER], self.max_grad_norm, self.clip, self.clip_workspace)
        bands = 3 * (self.deg + 1) ** 2
        groups = [(k, self.lr[k], 0, None) for k in PARAM_ORDER[:4]] + [("sh", self.lr["sh_dc"], 0, 3)]
        if bands > 3:
            groups.append(("sh", self.lr["sh_rest"], 3, bands))
        table = (GsAdamTensor * len(groups))()
        for a, (k, lr, c0, c1) in zip(table, groups):
            a.param, a.grad, a.exp_avg, a.exp_avg_sq = (t[k].data_ptr() for t in (p, g, self.m, self.v))
            a.rows, a.row_len = self.n, p[k].shape[1:].numel()
            a.col_begin, a.col_end, a.lr = c0, a.row_len if c1 is None else c1, lr
            a.normalize_rows = 1 if k == "quats" else 0
        gs_adam_step_clipped(table, 0.9, 0.999, 1e-8, self.t, self.clip)

    def densify(self):
        n0 = self.n
        p, ea, eq, _, _, action = densify_and_prune(self.densify_params, self.deg, self.p, self.accum, self.count,
                                                    self.m, self.v)
        self.p, self.m, self.v = ({k: t.contiguous() for k, t in d.items()} for d in (p, ea, eq))
        self.last_action = action
        self.events.append((self.t, "densify", (n0, self.n)))
        self._rebuild()

    def reset_opacity(self):
        gs_opacity_reset(self.p["opacity_logits"], self.reset_factor, self.m["opacity_logits"],
                         self.v["opacity_logits"])
        self.events.append((self.t, "reset", self.reset_factor))
