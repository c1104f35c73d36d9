"""ctypes binding of libia.so (include/ia.h), argument marshalling only.

The functions here carry the C names (ia_decoder_create, ia_decode, ...)
and take torch tensors for device buffers; every step of decode and render
runs in the HIP kernels of libia.so.  There is no CPU fallback: if the
library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes as C
import functools
import os
import struct

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "lib", "libia.so")

IA_OK = 0
IA_ERR_INVALID_ARG = -1
IA_ERR_UNSUPPORTED = -2
IA_ERR_WORKSPACE_TOO_SMALL = -3
IA_ERR_DEVICE = -4
IA_ERR_OUT_OF_MEMORY = -5
IA_DTYPE_F32, IA_DTYPE_F16, IA_DTYPE_BF16 = 0, 1, 2
IA_ACT_NONE, IA_ACT_RELU, IA_ACT_GELU = -1, 0, 1
IA_COLOR_RGB, IA_COLOR_SH3 = 0, 1
IA_BRANCHES_SHARED, IA_BRANCHES_PER_ATTRIBUTE = 0, 1
# ia_render_aux.binning
BINNING_AUTO, BINNING_TILE_SORT, BINNING_REGIONS = 0, 1, 2

# Every entry point include/ia.h declares.
EXPORTS = ("ia_last_error", "ia_decoder_create", "ia_decoder_set_params", "ia_decoder_update_params", "ia_decode",
           "ia_decode_xyzt", "ia_decoder_destroy", "ia_decode_backward", "ia_decode_feature_bytes", "ia_decode_keep",
           "ia_decode_workspace_size", "ia_decode_backward_workspace_size", "ia_lr_at", "ia_decode_xyzt_noalloc",
           "ia_spatial_order_workspace_size", "ia_spatial_order",
           "ia_hexplane_create", "ia_hexplane_set_params", "ia_hexplane_deform", "ia_hexplane_destroy",
           "ia_render_workspace_size", "ia_render", "ia_render_backward", "ia_l1_loss",
           "ia_image_loss_workspace_size", "ia_image_loss", "ia_adam_step", "ia_adam_step_strided",
           "ia_densify_accumulate", "ia_densify_workspace_size", "ia_densify",
           "ia_clip_workspace_size", "ia_grad_norm", "ia_clip_grad_norm", "ia_adam_clip_step",
           "ia_adam_clip_step_counted",
           "ia_mx4_quantize", "ia_mx4_dequantize", "ia_mx4_matmul_workspace_size", "ia_mx4_matmul",
           "ia_mx4_linear_workspace_size", "ia_mx4_linear", "ia_mx4_linear_backward_workspace_size",
           "ia_mx4_linear_backward",
           "ia_dropout", "ia_embedding", "ia_embedding_mx4", "ia_embedding_backward_workspace_size",
           "ia_embedding_backward",
           "ia_q4_quantize", "ia_q4_dequantize", "ia_q4_linear_workspace_size", "ia_q4_linear",
           "ia_profile_enable", "ia_profile_report", "ia_profile_reset")


class IAError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"ia status {status}: {msg}")
        self.status = status


class HashDesc(C.Structure):
    _fields_ = [("L", C.c_int32), ("F", C.c_int32), ("log2T", C.c_int32), ("base_res", C.c_double),
                ("growth", C.c_double), ("temporal_res", C.c_int32), ("table_dtype", C.c_int32),
                ("t_min", C.c_float), ("t_max", C.c_float)]


class MLPDesc(C.Structure):
    _fields_ = [("in_dim", C.c_int32), ("n_hidden", C.c_int32), ("hidden", C.c_int32 * 4),
                ("activation", C.c_int32), ("dtype", C.c_int32), ("color", C.c_int32), ("branches", C.c_int32)]


class Gaussians(C.Structure):
    _fields_ = [("means", C.c_void_p), ("means_stride", C.c_int32), ("scales", C.c_void_p),
                ("quats", C.c_void_p), ("colors", C.c_void_p), ("sh", C.c_void_p), ("opacity", C.c_void_p),
                ("sh_degree", C.c_int32)]


class HexPlaneDesc(C.Structure):
    _fields_ = [("res_xyz", C.c_int32), ("res_t", C.c_int32), ("channels", C.c_int32), ("aabb", C.c_float)]


class Camera(C.Structure):
    _fields_ = [("R", C.c_float * 9), ("t", C.c_float * 3), ("fx", C.c_float), ("fy", C.c_float),
                ("cx", C.c_float), ("cy", C.c_float), ("near_z", C.c_float), ("W", C.c_int32),
                ("H", C.c_int32), ("bg", C.c_float * 3)]


class RenderAux(C.Structure):
    _fields_ = [("T_final", C.c_void_p), ("n_contrib", C.c_void_p), ("n_entries", C.c_void_p),
                ("overflow", C.c_void_p), ("sorted_keys", C.c_void_p), ("sorted_vals", C.c_void_p),
                ("tile_ranges", C.c_void_p), ("proj_a", C.c_void_p), ("proj_b", C.c_void_p),
                ("proj_c", C.c_void_p), ("depth", C.c_void_p), ("tiles_touched", C.c_void_p),
                ("tile_rect", C.c_void_p), ("want_keys", C.c_int32), ("binning", C.c_int32)]


class DecoderGrads(C.Structure):
    _fields_ = [("tables", C.c_void_p), ("weights", C.c_void_p * 12), ("biases", C.c_void_p * 12)]


class GaussianGrads(C.Structure):
    _fields_ = [("means", C.c_void_p), ("scales", C.c_void_p), ("quats", C.c_void_p), ("opacity", C.c_void_p),
                ("colors", C.c_void_p), ("sh", C.c_void_p)]


class Grad(C.Structure):
    _fields_ = [("data", C.c_void_p), ("out", C.c_void_p), ("rows", C.c_int64), ("dim", C.c_int32),
                ("stride", C.c_int32), ("out_stride", C.c_int32), ("dtype", C.c_int32)]


class AdamGroup(C.Structure):
    _fields_ = [("param", C.c_void_p), ("grad", C.c_void_p), ("m", C.c_void_p), ("v", C.c_void_p),
                ("param_f16", C.c_void_p), ("rows", C.c_int64), ("dim", C.c_int32), ("param_stride", C.c_int32),
                ("lr", C.c_float)]
    PACK = struct.Struct("@5Pqiif4x")  # the same fields, to write a whole element at once


assert AdamGroup.PACK.size == C.sizeof(AdamGroup)


class Mx4(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("rows", C.c_int64), ("cols", C.c_int64)]


class Drop(C.Structure):
    _fields_ = [("p", C.c_double), ("seed", C.c_uint64), ("offset", C.c_uint64), ("step", C.c_void_p)]


class Q4(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("words", C.c_void_p), ("rows", C.c_int64), ("cols", C.c_int64),
                ("group", C.c_int32)]


_lib = None
P = C.c_void_p


def load(path: str = LIB_PATH):
    """Load libia.so; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with implicit_attribute_decode_amd/build.py "
                               "(or __graft_entry__.build()); there is no fallback path")
        L = C.CDLL(path)
        L.ia_last_error.restype = C.c_char_p
        L.ia_last_error.argtypes = []
        L.ia_decoder_create.argtypes = [P, P, P]
        L.ia_decoder_set_params.argtypes = [P, P, P, P, C.c_int32, P]
        L.ia_decode_workspace_size.argtypes = [P, C.c_int64, P]
        L.ia_decode_backward_workspace_size.argtypes = [P, C.c_int64, P]
        L.ia_decode.argtypes = [P, P, C.c_int64, C.c_float, P, P, C.c_size_t, P, P]
        L.ia_decode_xyzt.argtypes = [P, P, C.c_int64, P, P, C.c_size_t, P, P]
        L.ia_decode_xyzt_noalloc.argtypes = [P, P, C.c_int64, P, P]
        L.ia_spatial_order_workspace_size.argtypes = [C.c_int64, C.c_int32, P]
        L.ia_spatial_order.argtypes = [P, C.c_int32, C.c_int64, P, C.c_int32, P, P, P, C.c_size_t, P]
        L.ia_decoder_destroy.argtypes = [P]
        L.ia_decode_backward.argtypes = [P, P, C.c_int32, C.c_int64, C.c_float, P, P, P, P, P, C.c_size_t, P,
                                         C.c_size_t, P]
        L.ia_decode_feature_bytes.argtypes = [P, C.c_int64, P]
        L.ia_decode_keep.argtypes = [P, P, C.c_int32, C.c_int64, C.c_float, P, P, C.c_size_t, P, C.c_size_t, P, P]
        L.ia_lr_at.argtypes = [C.c_float, C.c_int32, C.c_int32, C.c_int32, C.c_float, P]
        L.ia_decoder_destroy.restype = None
        L.ia_hexplane_create.argtypes = [P, P]
        L.ia_hexplane_set_params.argtypes = [P, P, P, P, C.c_int32, P]
        L.ia_hexplane_deform.argtypes = [P, P, C.c_int64, C.c_float, P, P]
        L.ia_hexplane_destroy.argtypes = [P]
        L.ia_hexplane_destroy.restype = None
        L.ia_render_workspace_size.argtypes = [C.c_int64, C.c_int32, C.c_int32, C.c_int32, C.c_int64, P]
        L.ia_render.argtypes = [P, P, C.c_int32, P, P, C.c_size_t, C.c_int64, P, P, P]
        L.ia_render_backward.argtypes = [P, P, C.c_int32, P, P, C.c_size_t, C.c_int64, P, P, P, P, P]
        L.ia_l1_loss.argtypes = [P, P, C.c_int64, P, P, P]
        L.ia_image_loss_workspace_size.argtypes = [C.c_int32, C.c_int32, C.c_int32, P]
        L.ia_image_loss.argtypes = [P, P, C.c_int32, C.c_int32, C.c_int32, C.c_float, P, C.c_size_t, P, P, P]
        L.ia_adam_step.argtypes = [P, P, P, P, C.c_int64, C.c_float, C.c_float, C.c_float, C.c_float, C.c_int32, P,
                                   P]
        L.ia_adam_step_strided.argtypes = [P, C.c_int32, C.c_int32, P, P, P, C.c_int64, C.c_float, C.c_float,
                                           C.c_float, C.c_float, C.c_int32, P]
        L.ia_decoder_update_params.argtypes = [P, P, P, P, P]
        L.ia_densify_accumulate.argtypes = [P, C.c_int64, P, P, P]
        L.ia_densify_workspace_size.argtypes = [C.c_int64, P]
        L.ia_densify.argtypes = [P, P, P, P, P, P, P, P, P, C.c_int64, P, P, P, P, C.c_int64, P, P, C.c_size_t, P]
        L.ia_clip_workspace_size.argtypes = [C.c_int32, P]
        L.ia_grad_norm.argtypes = [P, C.c_int32, C.c_float, P, C.c_size_t, P, P]
        L.ia_clip_grad_norm.argtypes = [P, C.c_int32, C.c_float, P, C.c_size_t, P, P]
        L.ia_adam_clip_step.argtypes = [P, C.c_int32, C.c_float, C.c_float, C.c_float, C.c_float, C.c_int32, P,
                                        C.c_size_t, P, P]
        L.ia_adam_clip_step_counted.argtypes = [P, C.c_int32, C.c_float, C.c_float, C.c_float, C.c_float, C.c_int32, P, P,
                                                C.c_size_t, P, P]
        L.ia_mx4_quantize.argtypes = [P, C.c_int32, C.c_int64, C.c_int64, C.c_int64, C.c_int32, P, P]
        L.ia_mx4_dequantize.argtypes = [P, C.c_int32, P, C.c_int64, P]
        L.ia_mx4_matmul_workspace_size.argtypes = [C.c_int64, C.c_int64, C.c_int64, P]
        L.ia_mx4_matmul.argtypes = [P, P, P, C.c_int32, C.c_int32, P, C.c_int64, P, C.c_size_t, P]
        L.ia_mx4_linear_workspace_size.argtypes = [C.c_int64, C.c_int64, C.c_int64, P]
        L.ia_mx4_linear.argtypes = [P, C.c_int32, C.c_int64, C.c_int64, P, P, C.c_int32, P, C.c_int64, P, C.c_size_t,
                                    P]
        L.ia_mx4_linear_backward_workspace_size.argtypes = [C.c_int64, C.c_int64, C.c_int64, P]
        L.ia_mx4_linear_backward.argtypes = [P, C.c_int64, P, C.c_int64, P, C.c_int64, C.c_int32, C.c_int64, C.c_int64,
                                             C.c_int64, P, P, C.c_int64, P, P, P, C.c_size_t, P]
        L.ia_dropout.argtypes = [P, C.c_int32, C.c_int64, C.c_int64, C.c_int64, P, P, C.c_int64, P]
        L.ia_embedding.argtypes = [P, C.c_int32, C.c_int64, C.c_int64, C.c_int64, P, C.c_int32, C.c_int64, C.c_int64,
                                   C.c_double, P, C.c_int32, P, C.c_int64, P]
        L.ia_embedding_mx4.argtypes = [P, P, C.c_int32, C.c_int64, C.c_int64, C.c_double, P, C.c_int32, P, C.c_int64, P]
        L.ia_embedding_backward_workspace_size.argtypes = [C.c_int64, C.c_int64, C.c_int64, P]
        L.ia_embedding_backward.argtypes = [P, C.c_int32, C.c_int64, C.c_int64, P, C.c_int32, C.c_int64, C.c_int64,
                                            C.c_int64, C.c_double, P, P, P, C.c_size_t, P]
        L.ia_q4_quantize.argtypes = [P, C.c_int32, C.c_int64, P, P]
        L.ia_q4_dequantize.argtypes = [P, C.c_int32, P, C.c_int64, P]
        L.ia_q4_linear_workspace_size.argtypes = [C.c_int32, C.c_int64, C.c_int64, C.c_int64, P]
        L.ia_q4_linear.argtypes = [P, C.c_int32, C.c_int64, C.c_int64, P, P, C.c_int32, P, C.c_int64, P, C.c_size_t, P]
        L.ia_profile_enable.argtypes = [C.c_int32]
        L.ia_profile_report.argtypes = [P, C.c_size_t, P]
        L.ia_profile_reset.argtypes = []
        L.ia_profile_reset.restype = None
        for name in EXPORTS[1:]:
            if getattr(L, name).restype is C.c_int:
                getattr(L, name).restype = C.c_int32
        _lib = L
    return _lib


def _check(status: int):
    if status != IA_OK:
        raise IAError(status, load().ia_last_error().decode())


def _ptr(t) -> int | None:
    return None if t is None else int(t.data_ptr())


def _stream(stream=None) -> int:
    import torch

    if stream is None:
        # torch.cuda.current_stream().cuda_stream without the Stream object (1.4 us a call), where torch has it
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


# ----------------------------------------------------------------- decoder


def ia_last_error() -> str:
    return load().ia_last_error().decode()


def ia_decoder_create(hash_desc: HashDesc, mlp_desc: MLPDesc) -> C.c_void_p:
    h = C.c_void_p()
    _check(load().ia_decoder_create(C.byref(hash_desc), C.byref(mlp_desc), C.byref(h)))
    return h


def ia_decoder_set_params(dec, tables, weights, biases, stream=None):
    """tables / weights / biases: torch tensors on the device (kept alive by the caller until the copy runs)."""
    W = (C.c_void_p * len(weights))(*[_ptr(w) for w in weights])
    B = (C.c_void_p * len(biases))(*[_ptr(b) for b in biases])
    _check(load().ia_decoder_set_params(dec, _ptr(tables), W, B, 1, _stream(stream)))


def ia_decoder_update_params(dec, tables, weights, biases, stream=None):
    """Stream-ordered device copies of new parameter values into a decoder whose parameters are set."""
    W = (C.c_void_p * len(weights))(*[_ptr(w) for w in weights])
    B = (C.c_void_p * len(biases))(*[_ptr(b) for b in biases])
    _check(load().ia_decoder_update_params(dec, _ptr(tables), W, B, _stream(stream)))


def gaussians(means=None, scales=None, quats=None, colors=None, sh=None, opacity=None, means_stride=0,
              sh_degree=-1) -> Gaussians:
    return Gaussians(_ptr(means), means_stride, _ptr(scales), _ptr(quats), _ptr(colors), _ptr(sh), _ptr(opacity),
                     sh_degree)


def _nbytes(t) -> int:
    return 0 if t is None else int(t.numel() * t.element_size())


def _side(side) -> int | None:
    return None if side is None else int(side.cuda_stream)


def ia_decode_workspace_size(dec, N: int) -> int:
    b = C.c_size_t()
    _check(load().ia_decode_workspace_size(dec, int(N), C.byref(b)))
    return int(b.value)


def ia_decode_backward_workspace_size(dec, N: int) -> int:
    b = C.c_size_t()
    _check(load().ia_decode_backward_workspace_size(dec, int(N), C.byref(b)))
    return int(b.value)


def ia_decode(dec, xyz, N: int, t: float, out: Gaussians, ws=None, side=None, stream=None):
    """ws: device uint8 tensor (256-byte aligned) of ia_decode_workspace_size
    bytes or more; side: an optional second torch stream."""
    _check(load().ia_decode(dec, _ptr(xyz), int(N), float(t), C.byref(out), _ptr(ws), _nbytes(ws), _side(side),
                            _stream(stream)))


def ia_decode_xyzt(dec, xyzt, N: int, out: Gaussians, ws=None, side=None, stream=None):
    _check(load().ia_decode_xyzt(dec, _ptr(xyzt), int(N), C.byref(out), _ptr(ws), _nbytes(ws), _side(side),
                                 _stream(stream)))


def ia_decode_xyzt_noalloc(dec, xyzt, N: int, out: Gaussians, stream=None):
    """ia_decode_xyzt with the library's static scratch (allocates nothing)."""
    _check(load().ia_decode_xyzt_noalloc(dec, _ptr(xyzt), int(N), C.byref(out), _stream(stream)))


def ia_decode_backward(dec, pos, pos_stride: int, N: int, t: float, grad_attr: Gaussians, grad_means, grad_pos,
                       grads: DecoderGrads, features=None, ws=None, stream=None):
    _check(load().ia_decode_backward(dec, _ptr(pos), int(pos_stride), int(N), float(t), C.byref(grad_attr),
                                     _ptr(grad_means), _ptr(grad_pos), C.byref(grads), _ptr(features),
                                     _nbytes(features), _ptr(ws), _nbytes(ws), _stream(stream)))


def ia_decode_feature_bytes(dec, N: int) -> int:
    b = C.c_size_t()
    _check(load().ia_decode_feature_bytes(dec, int(N), C.byref(b)))
    return int(b.value)


def ia_decode_keep(dec, pos, pos_stride: int, N: int, t: float, out: Gaussians, features, ws=None, side=None,
                   stream=None):
    _check(load().ia_decode_keep(dec, _ptr(pos), int(pos_stride), int(N), float(t), C.byref(out), _ptr(features),
                                 _nbytes(features), _ptr(ws), _nbytes(ws), _side(side), _stream(stream)))


def ia_lr_at(base_lr: float, step: int, warmup: int, total: int, final_lr: float = 1e-7) -> float:
    """Learning rate at iteration `step` (0-based) of the warm-up + cosine schedule."""
    lr = C.c_float()
    _check(load().ia_lr_at(float(base_lr), int(step), int(warmup), int(total), float(final_lr), C.byref(lr)))
    return float(lr.value)


def ia_decoder_destroy(dec):
    load().ia_decoder_destroy(dec)


def ia_spatial_order_workspace_size(N: int, frames: int) -> int:
    b = C.c_size_t()
    _check(load().ia_spatial_order_workspace_size(int(N), int(frames), C.byref(b)))
    return int(b.value)


def ia_spatial_order(pos, frame_offsets, perm, pos_out, ws, stream=None):
    """pos: device [N, k>=3] float32 (contiguous rows); frame_offsets: host
    int64 [frames+1]; perm: device int32 [N] out; pos_out: device like pos,
    or None; ws: device uint8 workspace (256-byte aligned)."""
    fo = np.ascontiguousarray(frame_offsets, np.int64)
    N, stride = int(pos.shape[0]), int(pos.stride(0))
    _check(load().ia_spatial_order(_ptr(pos), stride, N, fo.ctypes.data_as(C.c_void_p), len(fo) - 1, _ptr(perm),
                                   _ptr(pos_out), _ptr(ws), _nbytes(ws), _stream(stream)))


# ----------------------------------------------------------------- HexPlane


def ia_hexplane_create(desc: HexPlaneDesc) -> C.c_void_p:
    h = C.c_void_p()
    _check(load().ia_hexplane_create(C.byref(desc), C.byref(h)))
    return h


def ia_hexplane_set_params(hp, planes, weights, biases, stream=None):
    Pl = (C.c_void_p * 6)(*[_ptr(p) for p in planes])
    W = (C.c_void_p * 3)(*[_ptr(w) for w in weights])
    B = (C.c_void_p * 3)(*[_ptr(b) for b in biases])
    _check(load().ia_hexplane_set_params(hp, Pl, W, B, 1, _stream(stream)))


def ia_hexplane_deform(hp, canonical: Gaussians, N: int, t: float, out: Gaussians, stream=None):
    _check(load().ia_hexplane_deform(hp, C.byref(canonical), int(N), float(t), C.byref(out), _stream(stream)))


def ia_hexplane_destroy(hp):
    load().ia_hexplane_destroy(hp)


# ----------------------------------------------------------------- render


def ia_render_workspace_size(N_total: int, frames: int, W: int, H: int, max_entries: int) -> int:
    n = C.c_size_t()
    _check(load().ia_render_workspace_size(int(N_total), int(frames), int(W), int(H), int(max_entries), C.byref(n)))
    return int(n.value)


def camera(cam) -> Camera:
    """Camera struct from any object with R, t, fx, fy, cx, cy, near, W, H, bg."""
    c = Camera()
    c.R[:] = [float(v) for v in np.asarray(cam.R, np.float32).ravel()]
    c.t[:] = [float(v) for v in np.asarray(cam.t, np.float32).ravel()]
    c.fx, c.fy, c.cx, c.cy = float(cam.fx), float(cam.fy), float(cam.cx), float(cam.cy)
    c.near_z = float(cam.near)
    c.W, c.H = int(cam.W), int(cam.H)
    c.bg[:] = [float(v) for v in np.asarray(cam.bg, np.float32).ravel()]
    return c


def ia_render(g: Gaussians, frame_offsets, cams, ws, max_entries: int, image, aux: RenderAux | None = None,
              stream=None):
    fo = np.ascontiguousarray(frame_offsets, np.int64)
    F = len(cams)
    arr = (Camera * F)(*[camera(c) for c in cams])
    _check(load().ia_render(C.byref(g), fo.ctypes.data_as(C.c_void_p), F, arr, _ptr(ws),
                            int(ws.numel() * ws.element_size()), int(max_entries), _ptr(image),
                            None if aux is None else C.byref(aux), _stream(stream)))


def ia_render_backward(g: Gaussians, frame_offsets, cams, ws, max_entries: int, grad_image, T_final, n_contrib,
                       grads: GaussianGrads, stream=None):
    """Same g / frame_offsets / cams / ws / max_entries as the ia_render it differentiates."""
    fo = np.ascontiguousarray(frame_offsets, np.int64)
    F = len(cams)
    arr = (Camera * F)(*[camera(c) for c in cams])
    _check(load().ia_render_backward(C.byref(g), fo.ctypes.data_as(C.c_void_p), F, arr, _ptr(ws),
                                     int(ws.numel() * ws.element_size()), int(max_entries), _ptr(grad_image),
                                     _ptr(T_final), _ptr(n_contrib), C.byref(grads), _stream(stream)))


def ia_l1_loss(image, target, loss, grad_image, stream=None):
    """loss: device float64 [1]; grad_image like image."""
    _check(load().ia_l1_loss(_ptr(image), _ptr(target), int(image.numel()), _ptr(loss), _ptr(grad_image),
                             _stream(stream)))


def ia_image_loss_workspace_size(frames: int, H: int, W: int) -> int:
    n = C.c_size_t()
    _check(load().ia_image_loss_workspace_size(int(frames), int(H), int(W), C.byref(n)))
    return int(n.value)


def ia_image_loss(image, target, lam: float, ws, loss, grad_image, stream=None):
    """image, target: device float [F, 3, H, W]; loss: device float64 [3]."""
    F, ch, H, W = (int(d) for d in image.shape)
    if ch != 3:
        raise ValueError("images must be [frames, 3, H, W]")
    _check(load().ia_image_loss(_ptr(image), _ptr(target), F, H, W, float(lam), _ptr(ws),
                                int(ws.numel() * ws.element_size()), _ptr(loss), _ptr(grad_image), _stream(stream)))


def ia_adam_step(param, grad, m, v, lr: float, beta1: float, beta2: float, eps: float, step: int, param_f16=None,
                 stream=None):
    _check(load().ia_adam_step(_ptr(param), _ptr(grad), _ptr(m), _ptr(v), int(param.numel()), float(lr),
                               float(beta1), float(beta2), float(eps), int(step), _ptr(param_f16), _stream(stream)))


def ia_adam_step_strided(param, grad, m, v, lr: float, beta1: float, beta2: float, eps: float, step: int,
                         stream=None):
    """param: a [rows, dim] view whose rows are param.stride(0) floats apart
    (e.g. xyzt[:, :3]); grad, m, v: dense [rows, dim]."""
    rows, dim = (int(d) for d in param.shape)
    if param.stride(1) != 1 or tuple(grad.shape) != (rows, dim) or not grad.is_contiguous():
        raise ValueError("param must be [rows, dim] with unit column stride; grad, m, v dense [rows, dim]")
    if max(dim, param.stride(0)) > 2 ** 31 - 1:  # the arguments would keep the low bits
        raise ValueError("param's rows are more than 2^31 - 1 floats apart")
    _check(load().ia_adam_step_strided(_ptr(param), int(param.stride(0)), dim, _ptr(grad), _ptr(m), _ptr(v), rows,
                                       float(lr), float(beta1), float(beta2), float(eps), int(step),
                                       _stream(stream)))


class DensifyParams(C.Structure):
    _fields_ = [("grad_threshold", C.c_float), ("scale_threshold", C.c_float), ("min_opacity", C.c_float)]


def ia_densify_accumulate(grad_pos, grad_acc, grad_count, stream=None):
    _check(load().ia_densify_accumulate(_ptr(grad_pos), int(grad_pos.shape[0]), _ptr(grad_acc), _ptr(grad_count),
                                        _stream(stream)))


def ia_densify_workspace_size(N: int) -> int:
    n = C.c_size_t()
    _check(load().ia_densify_workspace_size(int(N), C.byref(n)))
    return int(n.value)


def ia_densify(xyzt, grad_acc, grad_count, scales, quats, opacity, noise, m, v, params: DensifyParams, out_xyzt,
               out_m, out_v, out_n, ws, stream=None):
    """All device tensors; out_* of >= 2 N rows; out_n: int64 [1]."""
    _check(load().ia_densify(_ptr(xyzt), _ptr(grad_acc), _ptr(grad_count), _ptr(scales), _ptr(quats),
                             _ptr(opacity), _ptr(noise), _ptr(m), _ptr(v), int(xyzt.shape[0]), C.byref(params),
                             _ptr(out_xyzt), _ptr(out_m), _ptr(out_v), int(out_xyzt.shape[0]), _ptr(out_n),
                             _ptr(ws), 0 if ws is None else int(ws.numel() * ws.element_size()), _stream(stream)))


# ----------------------------------------------------------------- clipping


@functools.lru_cache(maxsize=64)  # a number of tensors has one size
def ia_clip_workspace_size(count: int) -> int:
    n = C.c_size_t()
    _check(load().ia_clip_workspace_size(int(count), C.byref(n)))
    return int(n.value)


def ia_grad_norm(grads, max_norm: float, ws, stats, stream=None):
    """grads: a ctypes array of Grad; stats: device float32 [3]."""
    _check(load().ia_grad_norm(grads, len(grads), float(max_norm), _ptr(ws), _nbytes(ws), _ptr(stats),
                               _stream(stream)))


def ia_clip_grad_norm(grads, max_norm: float, ws, stats, stream=None):
    _check(load().ia_clip_grad_norm(grads, len(grads), float(max_norm), _ptr(ws), _nbytes(ws), _ptr(stats),
                                    _stream(stream)))


def ia_adam_clip_step(groups, max_norm: float, beta1: float, beta2: float, eps: float, step: int, ws, stats,
                      stream=None, skipped=None):
    """groups: a ctypes array of AdamGroup; stats: device float32 [3]; skipped: device int32 [1] of
    ia_adam_clip_step_counted, or None."""
    _check(load().ia_adam_clip_step_counted(groups, len(groups), float(max_norm), float(beta1), float(beta2),
                                            float(eps), int(step), _ptr(skipped), _ptr(ws), _nbytes(ws), _ptr(stats),
                                            _stream(stream)))


# ----------------------------------------------------------------- MXFP4


def mx4(codes, scales, rows: int, cols: int) -> Mx4:
    return Mx4(_ptr(codes), _ptr(scales), rows, cols)


def ia_mx4_quantize(x, dtype: int, rows: int, cols: int, ld: int, transpose: bool, out: Mx4, stream=None):
    _check(load().ia_mx4_quantize(_ptr(x), dtype, rows, cols, ld, 1 if transpose else 0, C.byref(out),
                                  _stream(stream)))


def ia_mx4_dequantize(q: Mx4, dtype: int, x, ld: int, stream=None):
    _check(load().ia_mx4_dequantize(C.byref(q), dtype, _ptr(x), ld, _stream(stream)))


def ia_mx4_matmul_workspace_size(M: int, N: int, K: int) -> int:
    n = C.c_size_t()
    _check(load().ia_mx4_matmul_workspace_size(M, N, K, C.byref(n)))
    return n.value


def ia_mx4_matmul(a: Mx4, b: Mx4, bias, act: int, dtype: int, c, ldc: int, ws=None, stream=None):
    _check(load().ia_mx4_matmul(C.byref(a), C.byref(b), _ptr(bias), act, dtype, _ptr(c), ldc, _ptr(ws), _nbytes(ws),
                                _stream(stream)))


def ia_mx4_linear_workspace_size(M: int, K: int, N: int) -> int:
    n = C.c_size_t()
    _check(load().ia_mx4_linear_workspace_size(M, K, N, C.byref(n)))
    return n.value


def ia_mx4_linear(x, dtype: int, M: int, ldx: int, w: Mx4, bias, act: int, y, ldy: int, ws=None, stream=None):
    _check(load().ia_mx4_linear(_ptr(x), dtype, M, ldx, C.byref(w), _ptr(bias), act, _ptr(y), ldy, _ptr(ws),
                                _nbytes(ws), _stream(stream)))


def ia_mx4_linear_backward_workspace_size(M: int, N: int, K: int) -> int:
    n = C.c_size_t()
    _check(load().ia_mx4_linear_backward_workspace_size(M, N, K, C.byref(n)))
    return n.value


def ia_mx4_linear_backward(dy, lddy: int, y, ldy: int, x, ldx: int, dtype: int, M: int, N: int, K: int,
                           wt: Mx4 | None, dx, lddx: int, dw, db, ws=None, stream=None):
    _check(load().ia_mx4_linear_backward(_ptr(dy), lddy, _ptr(y), ldy, _ptr(x), ldx, dtype, M, N, K,
                                         None if wt is None else C.byref(wt), _ptr(dx), lddx, _ptr(dw), _ptr(db),
                                         _ptr(ws), _nbytes(ws), _stream(stream)))


# ----------------------------------------------------------------- embeddings, dropout


def _ref(s):
    return None if s is None else C.byref(s)


def _handle(stream) -> int:
    """A stream's raw handle as it is, else the handle of a stream or of the current one."""
    return stream if type(stream) is int else _stream(stream)


def ia_dropout(x, dtype: int, rows: int, cols: int, ldx: int, drop: Drop, out, ldo: int, stream=None):
    _check(load().ia_dropout(x.data_ptr(), dtype, rows, cols, ldx, C.byref(drop), out.data_ptr(), ldo, _handle(stream)))


def ia_embedding(table, dtype: int, entries: int, dim: int, ld: int, index, index_bytes: int, n: int, index_stride: int,
                 scale: float, drop: Drop | None, out_dtype: int, out, ldo: int, stream=None):
    _check(load().ia_embedding(table.data_ptr(), dtype, entries, dim, ld, index.data_ptr(), index_bytes, n, index_stride,
                               scale, _ref(drop), out_dtype, out.data_ptr(), ldo, _handle(stream)))


def ia_embedding_mx4(table: Mx4, index, index_bytes: int, n: int, index_stride: int, scale: float, drop: Drop | None,
                     out_dtype: int, out, ldo: int, stream=None):
    _check(load().ia_embedding_mx4(C.byref(table), index.data_ptr(), index_bytes, n, index_stride, scale, _ref(drop),
                                   out_dtype, out.data_ptr(), ldo, _handle(stream)))


@functools.lru_cache(maxsize=256)  # a shape has one size
def ia_embedding_backward_workspace_size(n: int, entries: int, dim: int) -> int:
    b = C.c_size_t()
    _check(load().ia_embedding_backward_workspace_size(n, entries, dim, C.byref(b)))
    return b.value


def ia_embedding_backward(dy, dtype: int, dim: int, lddy: int, index, index_bytes: int, n: int, index_stride: int,
                          entries: int, scale: float, drop: Drop | None, grad, ws=None, stream=None):
    _check(load().ia_embedding_backward(dy.data_ptr(), dtype, dim, lddy, index.data_ptr(), index_bytes, n, index_stride,
                                        entries, scale, _ref(drop), grad.data_ptr(), _ptr(ws), _nbytes(ws),
                                        _handle(stream)))


# ----------------------------------------------------------------- group-scaled 4 bits


def q4(codes, words, rows: int, cols: int, group: int) -> Q4:
    return Q4(_ptr(codes), _ptr(words), rows, cols, group)


def ia_q4_quantize(x, dtype: int, ldx: int, out: Q4, stream=None):
    _check(load().ia_q4_quantize(x.data_ptr(), dtype, ldx, C.byref(out), _handle(stream)))


def ia_q4_dequantize(q: Q4, dtype: int, x, ldx: int, stream=None):
    _check(load().ia_q4_dequantize(C.byref(q), dtype, x.data_ptr(), ldx, _handle(stream)))


@functools.lru_cache(maxsize=256)  # a shape has one size
def ia_q4_linear_workspace_size(dtype: int, M: int, K: int, N: int) -> int:
    n = C.c_size_t()
    _check(load().ia_q4_linear_workspace_size(dtype, M, K, N, C.byref(n)))
    return n.value


def ia_q4_linear(x, dtype: int, M: int, ldx: int, w: Q4, bias, act: int, y, ldy: int, ws=None, stream=None):
    _check(load().ia_q4_linear(x.data_ptr(), dtype, M, ldx, C.byref(w), _ptr(bias), act, y.data_ptr(), ldy, _ptr(ws),
                               _nbytes(ws), _handle(stream)))


# ----------------------------------------------------------------- diagnostics


def ia_profile_enable(on: bool = True):
    _check(load().ia_profile_enable(1 if on else 0))


def ia_profile_reset():
    load().ia_profile_reset()


def ia_profile_report() -> dict:
    """{kernel name: (calls, total ms)} since the last reset (waits for the events)."""
    import json

    need = C.c_size_t()
    load().ia_profile_report(None, 0, C.byref(need))
    buf = C.create_string_buffer(int(need.value) + 64)
    _check(load().ia_profile_report(buf, len(buf), None))
    return {k: (int(v[0]), float(v[1])) for k, v in json.loads(buf.value.decode()).items()}
