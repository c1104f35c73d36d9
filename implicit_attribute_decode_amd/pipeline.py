"""Convenience objects over the C ABI: Decoder, HexPlane, Renderer, Adam,
gradient clipping and 4-bit (MXFP4) matrices and layers.

Argument marshalling only (torch tensors in, torch tensors out); the work is
done by libia.so.  Parameter objects are duck-typed like the ones in
scenes.py (DecoderParams, HexPlaneParams, Camera).
"""
from __future__ import annotations

import math

import numpy as np
import torch

from . import ia


def _dev(a, dtype=None, device="cuda"):
    t = torch.as_tensor(np.ascontiguousarray(a), device=device)
    return t if dtype is None else t.to(dtype)


class _Workspace:
    """A device byte buffer that grows on demand and hands out 256-byte
    aligned views of the requested size (None for zero bytes)."""

    def __init__(self, device):
        self.device = device
        self.buf = None

    def get(self, nbytes: int):
        if nbytes <= 0:
            return None
        if self.buf is None or self.buf.numel() < nbytes + 256:
            self.buf = None
            self.buf = torch.empty(nbytes + 256, dtype=torch.uint8, device=self.device)
        off = (-self.buf.data_ptr()) % 256
        return self.buf[off:off + nbytes]


class Decoder:
    """Hash encoder + decoder MLP handle (SPIN-4DGS §3.3)."""

    def __init__(self, params, device="cuda"):
        h, m = params.hash, params.mlp
        f16 = bool(m.f16)
        hd = ia.HashDesc(int(h.L), int(h.F), int(h.log2T), float(h.base_res), float(h.growth), int(h.temporal_res),
                         ia.IA_DTYPE_F16 if h.table_f16 else ia.IA_DTYPE_F32, float(h.t_min), float(h.t_max))
        hidden = list(m.dims[1:-1])
        self.sh = int(m.dims[-1]) == 56  # SH colour (48 coefficients)
        branches = bool(getattr(m, "branches", False))
        md = ia.MLPDesc(int(m.dims[0]), len(hidden), (ia.C.c_int32 * 4)(*(hidden + [0] * (4 - len(hidden)))),
                        ia.IA_ACT_GELU if m.act == "gelu" else ia.IA_ACT_RELU,
                        ia.IA_DTYPE_F16 if f16 else ia.IA_DTYPE_F32,
                        ia.IA_COLOR_SH3 if self.sh else ia.IA_COLOR_RGB,
                        ia.IA_BRANCHES_PER_ATTRIBUTE if branches else ia.IA_BRANCHES_SHARED)
        self._destroy = ia.ia_decoder_destroy
        self.handle = ia.ia_decoder_create(hd, md)
        self.device = device
        self._tables = _dev(params.tables, device=device)
        self._W = [_dev(w, device=device) for w in params.weights]
        self._b = [_dev(b, torch.float32, device=device) for b in params.biases]
        ia.ia_decoder_set_params(self.handle, self._tables, self._W, self._b)
        torch.cuda.current_stream().synchronize()
        # this object's scratch (the handle holds only parameters) and a second
        # stream (default priority) for the MLP of one chunk beside the next gather
        self._ws = _Workspace(device)
        self._bwd_ws = _Workspace(device)
        self.side = torch.cuda.Stream(device=device)

    def workspace(self, N: int):
        """Aligned scratch view for a decode of N Gaussians (None if none is needed)."""
        return self._ws.get(ia.ia_decode_workspace_size(self.handle, N))

    def _out(self, N, out):
        if out is None:
            out = dict(scales=torch.empty((N, 3), dtype=torch.float32, device=self.device),
                       quats=torch.empty((N, 4), dtype=torch.float32, device=self.device),
                       opacity=torch.empty((N,), dtype=torch.float32, device=self.device))
            if self.sh:
                out["sh"] = torch.empty((N, 16, 3), dtype=torch.float32, device=self.device)
            else:
                out["colors"] = torch.empty((N, 3), dtype=torch.float32, device=self.device)
        return out

    def _gaussians(self, out):
        return ia.gaussians(scales=out["scales"], quats=out["quats"], colors=out.get("colors"), sh=out.get("sh"),
                            opacity=out["opacity"], sh_degree=3 if self.sh else -1)

    def decode(self, xyz: torch.Tensor, t: float, out: dict | None = None) -> dict:
        """Decoded attributes: scales, quats, opacity and colors [N,3] (RGB
        head) or sh [N,16,3] (SH head)."""
        N = int(xyz.shape[0])
        out = self._out(N, out)
        ia.ia_decode(self.handle, xyz, N, t, self._gaussians(out), self.workspace(N), self.side)
        return out

    def decode_xyzt(self, xyzt: torch.Tensor, out: dict | None = None) -> dict:
        N = int(xyzt.shape[0])
        out = self._out(N, out)
        ia.ia_decode_xyzt(self.handle, xyzt, N, self._gaussians(out), self.workspace(N), self.side)
        return out

    def decode_keep(self, pos: torch.Tensor, t: float | None = None, out: dict | None = None,
                    features: torch.Tensor | None = None):
        """Decode pos ([N,3] at time t, or [N,4] xyzt) and keep the encoding
        for backward(..., features=...).  Returns (attributes, features)."""
        N, stride = int(pos.shape[0]), int(pos.shape[1])
        out = self._out(N, out)
        nbytes = ia.ia_decode_feature_bytes(self.handle, N)
        if features is None or features.numel() * features.element_size() < nbytes:
            features = torch.empty(max(nbytes, 8) // 8, dtype=torch.int64, device=self.device)
        ia.ia_decode_keep(self.handle, pos, stride, N, float(t or 0.0), self._gaussians(out), features,
                          self.workspace(N), self.side)
        return out, features

    def backward(self, pos: torch.Tensor, grad_attr: dict, t: float | None = None, grad_means=None,
                 want_pos: bool = True, features: torch.Tensor | None = None) -> dict:
        """Gradients of the decode of pos ([N,3] at time t, or [N,4] xyzt)
        for upstream dL/d{scales, quats, colors (RGB) or sh [N,16,3] (SH
        colour), opacity}.  Every fp16 decoder: the shared trunk and the
        per-attribute branches.  Returns tables [L,T,F], weights and biases
        (lists in the order of the parameters, fp32, shaped like them)
        and, with want_pos, pos [N,3] = grad_means + the decoder's share."""
        N = int(pos.shape[0])
        stride = int(pos.shape[1])
        # first: the library says whether this decoder has a backward
        ws = self._bwd_ws.get(ia.ia_decode_backward_workspace_size(self.handle, N))
        out = dict(tables=torch.empty(self._tables.shape, dtype=torch.float32, device=self.device),
                   weights=[torch.empty(w.shape, dtype=torch.float32, device=self.device) for w in self._W],
                   biases=[torch.empty(b.shape, dtype=torch.float32, device=self.device) for b in self._b])
        out["pos"] = torch.empty((N, 3), dtype=torch.float32, device=self.device) if want_pos else None
        wp = [ia._ptr(w) for w in out["weights"]] + [None] * (12 - len(out["weights"]))
        bp = [ia._ptr(b) for b in out["biases"]] + [None] * (12 - len(out["biases"]))
        G = ia.DecoderGrads(ia._ptr(out["tables"]), (ia.C.c_void_p * 12)(*wp), (ia.C.c_void_p * 12)(*bp))
        up = ia.gaussians(scales=grad_attr["scales"], quats=grad_attr["quats"], colors=grad_attr.get("colors"),
                          sh=grad_attr.get("sh"), opacity=grad_attr["opacity"])
        ia.ia_decode_backward(self.handle, pos, stride, N, float(t or 0.0), up, grad_means, out["pos"], G, features,
                              ws)
        return out

    def update_params(self):
        """Copy this object's parameter tensors (tables, weights, biases; an
        optimiser updates them in place) into the handle, stream-ordered."""
        ia.ia_decoder_update_params(self.handle, self._tables, self._W, self._b)

    # rows of the shared decoder's head block per attribute (RGB head)
    HEAD_ROWS = {"scale": (0, 3), "rotation": (3, 7), "color": (7, 10), "opacity": (10, 11)}

    def param_groups(self, rates: dict) -> dict:
        """Adam groups of the shared-trunk RGB decoder ([SPIN] §4 implementation
        details: the encoder and each attribute's decoder parameters have their
        own rates).  rates: "encoder", "scale", "rotation", "color", "opacity".
        The hash tables take the encoder rate, the trunk layers (shared by all
        attributes) the largest of the attribute rates, and the head's rows and
        biases of each attribute that attribute's rate.  fp16 tables and
        weights get fp32 master copies with this object's tensors as their fp16
        mirrors; fp32 tensors are updated in place."""
        if self.sh or len(self._W) < 2:
            raise ValueError("parameter groups are defined for the shared-trunk RGB decoder")

        def master(t):
            return (t.float(), t.view(torch.int16)) if t.dtype == torch.float16 else (t, None)

        groups = {}
        p, m = master(self._tables)
        groups["tables"] = {"param": p, "lr": rates["encoder"], "f16": m}
        trunk = max(rates[a] for a in self.HEAD_ROWS)
        for k in range(len(self._W) - 1):
            p, m = master(self._W[k])
            groups[f"w{k}"] = {"param": p, "lr": trunk, "f16": m}
            groups[f"b{k}"] = {"param": self._b[k], "lr": trunk}
        head, m_head = master(self._W[-1])
        for a, (r0, r1) in self.HEAD_ROWS.items():
            groups[f"head_w_{a}"] = {"param": head[r0:r1], "lr": rates[a],
                                     "f16": None if m_head is None else m_head[r0:r1]}
            groups[f"head_b_{a}"] = {"param": self._b[-1][r0:r1], "lr": rates[a]}
        return groups

    def group_grads(self, grads: dict) -> dict:
        """The gradients of backward() keyed like param_groups()."""
        out = {"tables": grads["tables"]}
        for k in range(len(self._W) - 1):
            out[f"w{k}"] = grads["weights"][k]
            out[f"b{k}"] = grads["biases"][k]
        for a, (r0, r1) in self.HEAD_ROWS.items():
            out[f"head_w_{a}"] = grads["weights"][-1][r0:r1]
            out[f"head_b_{a}"] = grads["biases"][-1][r0:r1]
        return out

    def __del__(self):
        # the destroy function is bound at construction: at interpreter exit
        # the module globals may already be gone
        h = getattr(self, "handle", None)
        destroy = getattr(self, "_destroy", None)
        if h is not None and h.value and destroy is not None:
            destroy(h)
            self.handle = None


class HexPlane:
    """HexPlane deformation handle ("4D Gaussian Splatting详解", §3.1-3.2)."""

    def __init__(self, params, device="cuda"):
        self._destroy = ia.ia_hexplane_destroy
        self.handle = ia.ia_hexplane_create(ia.HexPlaneDesc(int(params.res_xyz), int(params.res_t),
                                                            int(params.channels), float(params.aabb)))
        self.device = device
        self._planes = [_dev(p, device=device) for p in params.planes]
        self._W = [_dev(w, device=device) for w in params.weights]
        self._b = [_dev(b, torch.float32, device=device) for b in params.biases]
        ia.ia_hexplane_set_params(self.handle, self._planes, self._W, self._b)
        torch.cuda.current_stream().synchronize()

    def deform(self, canon: dict, t: float, out: dict | None = None) -> dict:
        N = int(canon["means"].shape[0])
        if out is None:
            out = {k: torch.empty_like(canon[k]) for k in ("means", "scales", "quats", "sh", "opacity")}
        cg = ia.gaussians(means=canon["means"], scales=canon["scales"], quats=canon["quats"], sh=canon["sh"],
                          opacity=canon["opacity"], sh_degree=3)
        og = ia.gaussians(means=out["means"], scales=out["scales"], quats=out["quats"], sh=out["sh"],
                          opacity=out["opacity"], sh_degree=3)
        ia.ia_hexplane_deform(self.handle, cg, N, t, og)
        return out

    def __del__(self):
        # the destroy function is bound at construction: at interpreter exit
        # the module globals may already be gone
        h = getattr(self, "handle", None)
        destroy = getattr(self, "_destroy", None)
        if h is not None and h.value and destroy is not None:
            destroy(h)
            self.handle = None


_VIEW_TYPES = {
    "sorted_keys": (torch.int64, 1), "sorted_vals": (torch.int32, 1), "tile_ranges": (torch.int32, 2),
    "proj_a": (torch.float32, 4), "proj_b": (torch.float32, 4), "proj_c": (torch.float32, 1),
    "depth": (torch.float32, 1), "tiles_touched": (torch.int32, 1), "tile_rect": (torch.int16, 4),
}


class Renderer:
    """Owns a render workspace (a torch uint8 tensor) and calls ia_render."""

    def __init__(self, device="cuda"):
        self.device = device
        self._ws = _Workspace(device)
        self._loss_ws = _Workspace(device)

    def workspace(self, N, frames, W, H, max_entries):
        """Aligned view of this object's render workspace for these sizes."""
        return self._ws.get(ia.ia_render_workspace_size(N, frames, W, H, max_entries))

    def render(self, g: dict, frame_offsets, cams, max_entries: int, aux: bool = False, out: dict | None = None,
               keys: bool = True, binning: int = ia.BINNING_AUTO):
        """g: means [N,k>=3], scales, quats, colors | sh, opacity (cuda tensors).
        Returns image [F,3,H,W] and, with aux, T_final, n_contrib, n_entries,
        overflow and workspace views (ranges, projections and, with keys, the
        sorted keys / values).  binning: ia.BINNING_AUTO, _TILE_SORT or
        _REGIONS (the same lists either way)."""
        fo = np.asarray(frame_offsets, np.int64)
        F, W, H = len(cams), int(cams[0].W), int(cams[0].H)
        N = int(fo[-1])
        ws = self.workspace(N, F, W, H, max_entries)
        out = out or {}
        image = out.get("image")
        if image is None:
            image = torch.empty((F, 3, H, W), dtype=torch.float32, device=self.device)
        means = g["means"]
        stride = int(means.stride(0)) if means.dim() == 2 else 3
        sh = g.get("sh")
        G = ia.gaussians(means=means, scales=g["scales"], quats=g["quats"], colors=g.get("colors"), sh=sh,
                         opacity=g["opacity"], means_stride=stride, sh_degree=3 if sh is not None else -1)
        res = {"image": image}
        A = None
        if not aux and binning != ia.BINNING_AUTO:
            A = ia.RenderAux()
            A.binning = int(binning)
        if aux:
            res["T_final"] = torch.empty((F, H, W), dtype=torch.float32, device=self.device)
            res["n_contrib"] = torch.empty((F, H, W), dtype=torch.int32, device=self.device)
            res["n_entries"] = torch.zeros(1, dtype=torch.int64, device=self.device)
            res["overflow"] = torch.zeros(1, dtype=torch.int32, device=self.device)
            A = ia.RenderAux(ia._ptr(res["T_final"]), ia._ptr(res["n_contrib"]), ia._ptr(res["n_entries"]),
                             ia._ptr(res["overflow"]))
            A.want_keys = 1 if keys else 0
            A.binning = int(binning)
        ia.ia_render(G, fo, cams, ws, max_entries, image, A)
        if aux:
            base = ws.data_ptr()
            for name, (dt, width) in _VIEW_TYPES.items():
                p = getattr(A, name)
                if p:  # sorted keys / values only when requested
                    res["_view_" + name] = (int(p) - base, dt, width)
            res["_ws"] = ws
        return res

    def backward(self, g: dict, frame_offsets, cams, max_entries: int, res: dict, grad_image):
        """Gradients of the render `res` (made by render(..., aux=True) with
        the same g, frame_offsets, cams, max_entries and this workspace) for
        dL/dimage = grad_image.  Returns dict means, scales, quats, opacity,
        colors and, for SH colours, sh [N,16,3] (cuda float32, packed rows;
        the means include the view direction's share)."""
        fo = np.asarray(frame_offsets, np.int64)
        N = int(fo[-1])
        F, W, H = len(cams), int(cams[0].W), int(cams[0].H)
        ws = self.workspace(N, F, W, H, max_entries)
        means = g["means"]
        stride = int(means.stride(0)) if means.dim() == 2 else 3
        G = ia.gaussians(means=means, scales=g["scales"], quats=g["quats"], colors=g.get("colors"), sh=g.get("sh"),
                         opacity=g["opacity"], means_stride=stride, sh_degree=3 if g.get("sh") is not None else -1)
        out = {k: torch.empty(shape, dtype=torch.float32, device=self.device)
               for k, shape in (("means", (N, 3)), ("scales", (N, 3)), ("quats", (N, 4)), ("opacity", (N,)),
                                ("colors", (N, 3)))}
        if g.get("sh") is not None:
            out["sh"] = torch.empty((N, 16, 3), dtype=torch.float32, device=self.device)
        GG = ia.GaussianGrads(*[ia._ptr(out.get(k)) for k in ("means", "scales", "quats", "opacity", "colors", "sh")])
        ia.ia_render_backward(G, fo, cams, ws, max_entries, grad_image.contiguous(), res["T_final"],
                              res["n_contrib"], GG)
        return out

    @staticmethod
    def l1_loss(image, target):
        """(loss [1] float64 on the device, dL/dimage)."""
        loss = torch.empty(1, dtype=torch.float64, device=image.device)
        grad = torch.empty_like(image)
        ia.ia_l1_loss(image.contiguous(), target.contiguous(), loss, grad)
        return loss, grad

    def image_loss(self, image, target, lam: float = 0.2):
        """Eq. 12 loss of image against target ([F, 3, H, W] device float):
        (loss [3] float64 on the device = {L, L1, SSIM}, dL/dimage)."""
        F, _, H, W = (int(d) for d in image.shape)
        ws = self._loss_ws.get(ia.ia_image_loss_workspace_size(F, H, W))  # 256-byte aligned
        loss = torch.empty(3, dtype=torch.float64, device=image.device)
        grad = torch.empty_like(image)
        ia.ia_image_loss(image.contiguous(), target.contiguous(), lam, ws, loss, grad)
        return loss, grad

    @staticmethod
    def count_entries(res: dict) -> int:
        return int(res["n_entries"].item())

    @staticmethod
    def view(res: dict, name: str, count: int) -> torch.Tensor:
        """A workspace view of `count` rows (e.g. sorted_keys of n_entries rows)."""
        off, dt, width = res["_view_" + name]
        ws = res["_ws"]
        nbytes = count * width * torch.empty((), dtype=dt).element_size()
        t = ws[off:off + nbytes].view(dt)
        return t.view(count, width) if width > 1 else t



def spatial_order(pos: torch.Tensor, frame_offsets):
    """(perm, reordered positions): every frame's Gaussians along a Morton
    curve of their normalised positions (ia_spatial_order); a one-time
    storage layout for fixed per-frame position sets."""
    fo = np.asarray(frame_offsets, np.int64)
    pos = pos.contiguous()
    N = int(pos.shape[0])
    perm = torch.empty(N, dtype=torch.int32, device=pos.device)
    out = torch.empty_like(pos)
    ws = _Workspace(pos.device).get(ia.ia_spatial_order_workspace_size(N, len(fo) - 1))
    ia.ia_spatial_order(pos, fo, perm, out, ws)
    return perm, out


def lr_at(step: int, base: float, warmup: int, total: int, final: float = 1e-7) -> float:
    """Learning rate at `step` (0-based): linear warm-up over `warmup` steps,
    then cosine decay from base to `final` at `total` ([SPIN] §4
    implementation details); evaluated by ia_lr_at."""
    return ia.ia_lr_at(base, step, warmup, total, final)


class _Moments(dict):
    """name -> (m, v), an optimiser's moments: contiguous float32 tensors of one
    size on one device, checked when they are put in."""

    def __init__(self, moments):
        super().__init__()
        self.update(moments)

    def __setitem__(self, name, moments):
        m, v = moments
        if not (m.dtype == v.dtype == torch.float32 and m.is_contiguous() and v.is_contiguous()
                and m.numel() == v.numel() and m.device == v.device):
            raise ValueError(f"group {name}: moments must be contiguous float32 tensors of one size on one device")
        super().__setitem__(name, (m, v))

    def update(self, *args, **moments):
        for name, mv in dict(*args, **moments).items():
            self[name] = mv

    def setdefault(self, name, moments=None):
        if name not in self:
            self[name] = moments
        return self[name]

    def __ior__(self, moments):
        self.update(moments)
        return self

    def __reduce__(self):
        return _Moments, (dict(self),)


class Adam:
    """Adam over named parameter groups, each an fp32 device tensor with its
    own base learning rate ([SPIN] §4 implementation details: per-group rates,
    linear warm-up then cosine decay to 1e-7).  A group may carry an fp16
    mirror (e.g. the decoder's hash table) that every step refreshes, and its
    parameter may be a [rows, dim] view with rows further apart than dim (the
    x, y, z of xyzt positions).  Every update runs in ia_adam_step or
    ia_adam_step_strided, with max_norm in ia_adam_clip_step_counted."""

    def __init__(self, groups: dict, warmup: int, total: int, beta1: float = 0.9, beta2: float = 0.999,
                 eps: float = 1e-15):
        self.groups = groups  # name -> {"param": fp32 tensor, "lr": base, optional "f16": tensor}
        self.state = {k: tuple(torch.zeros(g["param"].shape, dtype=torch.float32, device=g["param"].device)
                               for _ in range(2)) for k, g in groups.items()}
        self.warmup, self.total = warmup, total
        self.beta1, self.beta2, self.eps = beta1, beta2, eps
        self.t = 0
        # steps that changed nothing, kept by the library on the parameters' device
        self.skipped = next((torch.zeros(1, dtype=torch.int32, device=g["param"].device) for g in groups.values()),
                            None)

    @property
    def state(self):
        """name -> (m, v); may be replaced, whole or group by group."""
        return self._state

    @state.setter
    def state(self, moments):
        self._state = _Moments(moments)

    def step(self, grads: dict, max_norm: float | None = None):
        """One update of every group that has a gradient in `grads` (name -> tensor).

        With max_norm the gradients count as clipped by their global norm over
        the groups updated (they are not modified) and all groups go through
        one launch; returns its stats, a device float32 tensor {norm, factor,
        1 if the norm is finite else 0}.  A step whose norm is not finite
        changes no parameter and no moment: it counts in t, which sets the
        rates, and in `skipped` (device int32 [1]), which the bias corrections
        of the clipped steps after it leave out."""
        if max_norm is not None:
            return self._clipped_step(grads, max_norm)
        self.t += 1
        for name, g in self.groups.items():
            grad = grads.get(name)
            if grad is None:
                continue
            m, v = self.state[name]
            lr = lr_at(self.t - 1, g["lr"], self.warmup, self.total)
            p = g["param"]
            if p.is_contiguous():
                ia.ia_adam_step(p, grad.contiguous(), m, v, lr, self.beta1, self.beta2, self.eps, self.t, g.get("f16"))
            else:
                if g.get("f16") is not None:
                    raise ValueError(f"group {name}: an fp16 mirror needs a contiguous parameter")
                ia.ia_adam_step_strided(p, grad.contiguous(), m, v, lr, self.beta1, self.beta2, self.eps, self.t)

    def _clipped_step(self, grads: dict, max_norm: float):
        groups = [(k, g, grad) for k, g in self.groups.items() if (grad := grads.get(k)) is not None]
        arr = (ia.AdamGroup * len(groups))()
        at, size, pack = 0, ia.AdamGroup.PACK.size, ia.AdamGroup.PACK.pack_into
        keep, rates = [], {}  # contiguous copies live until the call has enqueued its reads
        f32, state, device = torch.float32, self._state, None
        for name, g, grad in groups:
            p, f16, lr = g["param"], g.get("f16"), g["lr"]
            m, v = state[name]
            if p.dtype is not f32 or grad.dtype is not f32 or grad.shape != p.shape:
                raise ValueError(f"group {name}: parameter and gradient must be float32 of one shape")
            nbytes, dev = grad.nbytes, grad.get_device()
            if m.nbytes != nbytes or v.nbytes != nbytes or m.get_device() != dev:  # the rest when they were put in
                raise ValueError(f"group {name}: moments of another size or device than the gradient")
            if f16 is not None and not (f16.element_size() == 2 and 2 * f16.nbytes == nbytes and f16.is_contiguous()
                                        and f16.get_device() == dev):
                raise ValueError(f"group {name}: an fp16 mirror must be contiguous 16-bit values of the parameter's "
                                 "size and device")
            if device is None:
                device = dev
            if dev < 0 or dev != device or p.get_device() != dev:
                raise ValueError(f"group {name}: parameters and gradients must be on one GPU")
            if not grad.is_contiguous():
                grad = grad.contiguous()
                keep.append(grad)
            if p.is_contiguous():
                rows, dim, stride = nbytes // 4, 1, 1
            elif p.dim() == 2 and p.stride(1) == 1 and p.shape[1] <= p.stride(0) <= _INT32_MAX and f16 is None:
                rows, dim, stride = p.shape[0], p.shape[1], p.stride(0)
            else:
                raise ValueError(f"group {name}: the parameter must be contiguous, or [rows, dim] rows of a wider "
                                 "array without an fp16 mirror")
            rate = rates.get(lr)
            if rate is None:
                rate = rates[lr] = lr_at(self.t, lr, self.warmup, self.total)
            pack(arr, at, p.data_ptr(), grad.data_ptr(), m.data_ptr(), v.data_ptr(),
                 0 if f16 is None else f16.data_ptr(), rows, dim, stride, rate)
            at += size
        device = p.device if groups else "cuda"
        stats = torch.empty(3, dtype=f32, device=device)
        ws = torch.empty(ia.ia_clip_workspace_size(len(groups)), dtype=torch.uint8, device=device)
        if self.skipped is None:
            self.skipped = torch.zeros(1, dtype=torch.int32, device=device)
        elif groups and self.skipped.get_device() != dev:
            self.skipped = self.skipped.to(device)
        ia.ia_adam_clip_step(arr, max_norm, self.beta1, self.beta2, self.eps, self.t + 1, ws, stats, None, self.skipped)
        self.t += 1  # a refused call is no step
        return stats


_INT32_MAX = 2 ** 31 - 1
_DTYPES = {torch.float32: ia.IA_DTYPE_F32, torch.float16: ia.IA_DTYPE_F16, torch.bfloat16: ia.IA_DTYPE_BF16}


def _dtype(t: torch.Tensor) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"float32, float16 or bfloat16 expected, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError("a tensor on the GPU expected")
    return d


def _one_device(t: torch.Tensor, *others):
    """Refuses tensors on several devices (None stands for no tensor)."""
    device = t.get_device()
    for o in others:
        if o is not None and o.get_device() != device:
            raise ValueError("tensors on several devices")


class GradClip:
    """Clipping of a list of gradient tensors by their global norm (Pascanu,
    Mikolov & Bengio 2013): factor = max_norm / norm where norm > max_norm,
    else 1.  The tensors (float32, float16 or bfloat16 in any mix; contiguous,
    or [rows, dim] rows of a wider array) are described once and may be filled
    anew before every call; `out` (same shapes and types) receives the clipped
    values, without it they are scaled in place.  What is written must not share
    memory with another tensor of the lists.

    clip(max_norm) clips and norm() only measures; both return a new device
    float32 tensor {norm, factor, 1 if the norm is finite else 0}."""

    def __init__(self, grads, out=None):
        self.grads = list(grads)
        self.out = None if out is None else list(out)
        if self.out is not None and len(self.out) != len(self.grads):
            raise ValueError("as many outputs as gradients expected")
        self._arr = (ia.Grad * len(self.grads))()
        for k, (d, g) in enumerate(zip(self._arr, self.grads)):
            d.dtype = _dtype(g)
            d.data = g.data_ptr()
            o = g if self.out is None else self.out[k]
            if o.dtype != g.dtype or o.shape != g.shape or o.device != g.device:
                raise ValueError(f"output {k} differs from its gradient in type, shape or device")
            if g.is_contiguous() and o.is_contiguous():
                d.rows, d.dim, d.stride, d.out_stride = g.numel(), 1, 1, 1
            elif g.dim() == 2 and all(t.shape[1] <= 1 or t.stride(1) == 1 for t in (g, o)):
                if max(g.shape[1], g.stride(0), o.stride(0)) > _INT32_MAX:  # the fields would keep the low bits
                    raise ValueError(f"gradient {k}: rows of more than 2^31 - 1 elements, or as far apart")
                d.rows, d.dim, d.stride, d.out_stride = g.shape[0], max(g.shape[1], 1), g.stride(0), o.stride(0)
                if g.shape[1] == 0:
                    d.rows, d.stride, d.out_stride = 0, 1, 1
            else:
                raise ValueError(f"gradient {k} must be contiguous or [rows, dim] with unit column stride")
            d.out = None if self.out is None else o.data_ptr()
        if self.grads:
            _one_device(*self.grads)
        self.device = self.grads[0].device if self.grads else torch.device("cuda")
        self._ws_bytes = ia.ia_clip_workspace_size(len(self.grads))

    def _call(self, fn, max_norm):
        stats = torch.empty(3, dtype=torch.float32, device=self.device)
        fn(self._arr, max_norm, torch.empty(self._ws_bytes, dtype=torch.uint8, device=self.device), stats)
        return stats

    def __call__(self, max_norm: float):
        return self._call(ia.ia_clip_grad_norm, max_norm)

    def norm(self, max_norm: float = math.inf):
        return self._call(ia.ia_grad_norm, max_norm)


def clip_grad_norm(grads, max_norm: float, out=None):
    """Clip `grads` (a list of tensors) once; see GradClip.  Returns its stats."""
    return GradClip(grads, out)(max_norm)


def densify_positions(xyzt, grad_acc, grad_count, attrs: dict, m, v, noise, grad_threshold: float,
                      scale_threshold: float, min_opacity: float):
    """Refine the positions ([SPIN] §3.2 Eq. 6; clone / split / prune, see
    ia_densify) from the decoded attributes `attrs` (scales, quats, opacity).
    Returns (xyzt', m', v') of the rows written; reading their count is the
    one host synchronisation."""
    N = int(xyzt.shape[0])
    dev = xyzt.device
    out_x = torch.empty((2 * N, 4), dtype=torch.float32, device=dev)
    out_m = torch.empty((2 * N, 3), dtype=torch.float32, device=dev)
    out_v = torch.empty((2 * N, 3), dtype=torch.float32, device=dev)
    out_n = torch.zeros(1, dtype=torch.int64, device=dev)
    ws = torch.empty(max(ia.ia_densify_workspace_size(N), 256), dtype=torch.uint8, device=dev)
    p = ia.DensifyParams(grad_threshold, scale_threshold, min_opacity)
    ia.ia_densify(xyzt.contiguous(), grad_acc, grad_count, attrs["scales"], attrs["quats"], attrs["opacity"],
                  noise.contiguous(), m.contiguous(), v.contiguous(), p, out_x, out_m, out_v, out_n, ws)
    n = int(out_n.item())
    return out_x[:n], out_m[:n], out_v[:n]


class PipelinedDecodeRender:
    """Decode + render of a batch of frames whose Gaussians are stored frame
    after frame, in `parts` consecutive groups of frames: the render of group k
    runs on a second stream (default priority) beside the decode of group
    k + 1.  The decode's gather is bound by L2 requests and the raster by VALU
    issue, so the two share the chip well.  Every group has its own render
    workspace; images and decoded attributes land in the caller's tensors.
    Results equal one decode and one render of the whole batch, bit for bit
    when every group starts at a multiple of 64 Gaussians (a decoded value's
    MFMA rounding depends on its index mod 64 within a decode call), else to
    the decoder's tolerance."""

    def __init__(self, decoder: Decoder, xyzt: torch.Tensor, frame_offsets, cams, attrs: dict,
                 image: torch.Tensor, parts: int):
        fo = np.asarray(frame_offsets, np.int64)
        F = len(cams)
        if not 1 <= parts <= F:
            raise ValueError("parts must be in 1..frames")
        self.decoder, self.xyzt = decoder, xyzt
        self.side = torch.cuda.Stream(device=xyzt.device)
        bounds = [(F * k) // parts for k in range(parts + 1)]
        self.groups = []
        for k in range(parts):
            f0, f1 = bounds[k], bounds[k + 1]
            lo, hi = int(fo[f0]), int(fo[f1])
            out = {n: v[lo:hi] for n, v in attrs.items()}
            self.groups.append(dict(lo=lo, hi=hi, fo=fo[f0:f1 + 1] - lo, cams=list(cams[f0:f1]), out=out,
                                    g=dict(means=xyzt[lo:hi, :3], **out), R=Renderer(str(xyzt.device)),
                                    image=image[f0:f1], cap=None))

    def probe(self, slack: float = 1.02) -> int:
        """Decode and render once, counting each group's tile entries (host
        synchronisation); sets the capacities.  Returns the total count."""
        total = 0
        for grp in self.groups:
            self.decoder.decode_xyzt(self.xyzt[grp["lo"]:grp["hi"]], out=grp["out"])
            n = grp["hi"] - grp["lo"]
            res = grp["R"].render(grp["g"], grp["fo"], grp["cams"], 4 * max(n, 1), aux=True,
                                  out={"image": grp["image"]})
            e = Renderer.count_entries(res)
            grp["cap"] = int(e * slack) + 4096
            total += e
        return total

    def __call__(self):
        if any(grp["cap"] is None for grp in self.groups):
            raise RuntimeError("call probe() first")
        main = torch.cuda.current_stream(self.xyzt.device)
        if len(self.groups) == 1:  # nothing to overlap: one decode, one render, one stream
            grp = self.groups[0]
            self.decoder.decode_xyzt(self.xyzt[grp["lo"]:grp["hi"]], out=grp["out"])
            grp["R"].render(grp["g"], grp["fo"], grp["cams"], grp["cap"], out={"image": grp["image"]})
            return
        for grp in self.groups:
            self.decoder.decode_xyzt(self.xyzt[grp["lo"]:grp["hi"]], out=grp["out"])
            self.side.wait_stream(main)
            with torch.cuda.stream(self.side):
                grp["R"].render(grp["g"], grp["fo"], grp["cams"], grp["cap"], out={"image": grp["image"]})
        main.wait_stream(self.side)


class FrameGraphs:
    """Per-frame decode + render replayed from HIP graphs (SPIN-4DGS page §4:
    every frame is decoded from its own position set at its own time and
    rendered on its own).

    Frame f's graph holds its ia_decode_xyzt call (normalisation, hash gather,
    decoder MLP) and its ia_render call (projection, depth sort, key emission,
    tile sort, ranges, raster; the camera and frame offsets travel as kernel
    arguments of upload kernels, clears are fill kernels: no memset or memcpy
    node).  A replay submits the frame's ~45 kernels in one call instead of
    one launch each.  The graphs keep the addresses they were captured with:
    positions, attribute and image buffers, and the decoder's and renderer's
    workspaces must stay allocated and in place while they are used, and the
    decoder's parameters may be updated in place (set_params) but not
    reallocated.

    xyzt: [N, 4] device positions of all frames, frame f at
    frame_offsets[f]:frame_offsets[f+1]; attrs: decoder output buffers [N, ...];
    image: [F, 3, H, W]; max_entries: the tile-entry capacity of one frame."""

    def __init__(self, decoder: "Decoder", renderer: "Renderer", xyzt: torch.Tensor, frame_offsets, cams,
                 max_entries: int, attrs: dict, image: torch.Tensor):
        self.D, self.R = decoder, renderer
        self.xyzt, self.cams, self.cap = xyzt, list(cams), int(max_entries)
        self.fo = np.asarray(frame_offsets, np.int64)
        self.attrs, self.image = attrs, image
        F = len(self.cams)
        # one eager pass: sizes both workspaces (no allocation happens while
        # capturing) and fills the one-time caches of the launch code
        for f in range(F):
            self.frame(f)
        torch.cuda.synchronize()
        self.graphs = []
        pool = None
        for f in range(F):
            g = torch.cuda.CUDAGraph(keep_graph=True)
            with torch.cuda.graph(g, pool=pool):
                self.frame(f)
            g.instantiate()
            pool = g.pool()
            self.graphs.append(g)
        torch.cuda.synchronize()

    def frame(self, f: int):
        """Frame f eagerly: one decode and one single-frame render."""
        lo, hi = int(self.fo[f]), int(self.fo[f + 1])
        x = self.xyzt[lo:hi]
        a = self.D.decode_xyzt(x, out={k: v[lo:hi] for k, v in self.attrs.items()})
        self.R.render(dict(means=x[:, :3], **a), [0, hi - lo], [self.cams[f]], self.cap,
                      out={"image": self.image[f:f + 1]})

    def replay(self, frames=None):
        """Replay the graphs of `frames` (default: all) in order on the current stream."""
        for f in (range(len(self.graphs)) if frames is None else frames):
            self.graphs[f].replay()


_ACTS = {"none": ia.IA_ACT_NONE, "relu": ia.IA_ACT_RELU}


def _matrix(t: torch.Tensor, name: str):
    """(dtype, rows, cols, row stride) of a 2-D tensor with unit column stride; a row stride of 0 repeats one row."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be [rows, cols]")
    (rows, cols), (ld, step) = t.shape, t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must have unit column stride")
    return _dtype(t), rows, cols, (ld if rows > 1 else cols)


def _bytes(n: int, device):
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


class Mx4Tensor:
    """A [rows, cols] matrix in MXFP4: codes uint8 [rows, 16 ceil(cols / 32)]
    (two E2M1 codes a byte, the earlier value in the low half), scales uint8
    [rows, ceil(cols / 32)] (2^(byte - 127), 255 = NaN).  The tensors are not
    replaced, nor are the sizes; their values may change (quantised anew)."""

    __slots__ = ("_codes", "_scales", "_rows", "_cols", "c")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, cols: int):
        blocks = (cols + 31) // 32
        rows = codes.shape[0]
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or not codes.is_cuda or not scales.is_cuda:
            raise ValueError("codes and scales must be uint8 tensors on the GPU")
        _one_device(codes, scales)
        if (codes.shape != (rows, 16 * blocks) or scales.shape != (rows, blocks)
                or not codes.is_contiguous() or not scales.is_contiguous()):
            raise ValueError(f"codes [{rows}, {16 * blocks}] and scales [{rows}, {blocks}] expected, contiguous")
        self._codes, self._scales, self._rows, self._cols = codes, scales, rows, cols
        self.c = ia.mx4(codes, scales, rows, cols)

    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)
    rows = property(lambda self: self._rows)
    cols = property(lambda self: self._cols)

    @classmethod
    def empty(cls, rows: int, cols: int, device="cuda"):
        blocks = (cols + 31) // 32
        return cls(torch.empty((rows, 16 * blocks), dtype=torch.uint8, device=device),
                   torch.empty((rows, blocks), dtype=torch.uint8, device=device), cols)

    def dequantize(self, dtype=torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
        """The values, rounded once to dtype (float32, float16 or bfloat16)."""
        if out is None:
            out = torch.empty((self.rows, self.cols), dtype=dtype, device=self._codes.device)
        d, rows, cols, ld = _matrix(out, "out")
        if (rows, cols) != (self.rows, self.cols):
            raise ValueError("out has another shape")
        _one_device(out, self._codes)
        ia.ia_mx4_dequantize(self.c, d, out, ld)
        return out


def mx4_quantize(x: torch.Tensor, transpose: bool = False, out: Mx4Tensor | None = None) -> Mx4Tensor:
    """x [rows, cols] in MXFP4, blocks along its rows; with transpose the
    matrix [cols, rows] of its columns, blocks along them."""
    d, rows, cols, ld = _matrix(x, "x")
    if out is None:
        out = Mx4Tensor.empty(cols, rows, x.device) if transpose else Mx4Tensor.empty(rows, cols, x.device)
    else:
        _one_device(x, out._codes)
    ia.ia_mx4_quantize(x, d, rows, cols, ld, transpose, out.c)
    return out


def _bias(bias, n: int):
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (n,) or not bias.is_contiguous()
                             or not bias.is_cuda):
        raise ValueError(f"bias must be a contiguous float32 [{n}] on the GPU")
    return bias


def mx4_matmul(a: Mx4Tensor, b: Mx4Tensor, bias: torch.Tensor | None = None, act: str = "none",
               dtype=torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """act(a b^T + bias): a [M, K], b [N, K] -> [M, N] of dtype; act "none" or "relu"."""
    if out is None:
        out = torch.empty((a.rows, b.rows), dtype=dtype, device=a.codes.device)
    d, rows, cols, ld = _matrix(out, "out")
    if (rows, cols) != (a.rows, b.rows):
        raise ValueError("out has another shape")
    _one_device(out, a._codes, b._codes, bias)
    ws = _bytes(ia.ia_mx4_matmul_workspace_size(a.rows, b.rows, a.cols), out.device)
    ia.ia_mx4_matmul(a.c, b.c, _bias(bias, b.rows), _ACTS[act], d, out, ld, ws)
    return out


def mx4_linear(x: torch.Tensor, w: Mx4Tensor, bias: torch.Tensor | None = None, act: str = "none",
               out: torch.Tensor | None = None) -> torch.Tensor:
    """A linear layer with MXFP4 weights: act(Q(x) w^T + bias), x [M, K]
    quantised along its rows, w [N, K]; returns [M, N] of x's type."""
    d, M, K, ldx = _matrix(x, "x")
    N = w.rows
    if K != w.cols:
        raise ValueError(f"x has {K} columns, the weights {w.cols}")
    if out is None:
        out, ldy = torch.empty((M, N), dtype=x.dtype, device=x.device), N
    else:
        do, rows, cols, ldy = _matrix(out, "out")
        if (do, rows, cols) != (d, M, N):
            raise ValueError("out has another shape or type")
    _one_device(x, w._codes, bias, out)
    ws = _bytes(ia.ia_mx4_linear_workspace_size(M, K, N), x.device)
    ia.ia_mx4_linear(x, d, M, ldx, w.c, _bias(bias, N), _ACTS[act], out, ldy, ws)
    return out


def mx4_linear_backward(dy: torch.Tensor, x: torch.Tensor, wt: Mx4Tensor | None, y: torch.Tensor | None = None,
                        want_x: bool = True) -> dict:
    """Gradients of mx4_linear for upstream dy [M, N]: x [M, K] of x's type
    (with want_x), weight [N, K] and bias [N] in float32.  wt: the [N, K]
    weights quantised along their outputs (mx4_quantize(w, transpose=True), so
    [K, N]); y: the layer's output when its activation was ReLU."""
    d, M, N, lddy = _matrix(dy, "dy")
    dx_, Mx, K, ldx = _matrix(x, "x")
    if dx_ != d or Mx != M:
        raise ValueError("dy and x must have one type and number of rows")
    ldy = 0
    if y is not None:
        dt, My, Ny, ldy = _matrix(y, "y")
        if (dt, My, Ny) != (d, M, N):
            raise ValueError("y must have dy's type and shape")
    if want_x and (wt is None or (wt.rows, wt.cols) != (K, N)):
        raise ValueError(f"wt must be [{K}, {N}]")
    _one_device(dy, x, y, wt._codes if want_x else None)
    dx = torch.empty((M, K), dtype=x.dtype, device=x.device) if want_x else None
    dw = torch.empty((N, K), dtype=torch.float32, device=x.device)
    db = torch.empty(N, dtype=torch.float32, device=x.device)
    ws = _bytes(ia.ia_mx4_linear_backward_workspace_size(M, N, K), x.device)
    ia.ia_mx4_linear_backward(dy, lddy, y, ldy, x, ldx, d, M, N, K, wt.c if want_x else None, dx, K, dw, db, ws)
    return {"x": dx, "weight": dw, "bias": db}


class Mx4Linear:
    """A linear layer trained with its products in MXFP4: fp32 master weight
    [N, K] and bias [N] (an optimiser updates them in place, then update()
    quantises them again) and the weight's two 4-bit forms, along its inputs
    (forward) and along its outputs (the input's gradient)."""

    def __init__(self, weight: torch.Tensor, bias: torch.Tensor | None = None, act: str = "none"):
        if act not in _ACTS:
            raise ValueError("act must be 'none' or 'relu'")
        self.weight, self.bias, self.act = weight, _bias(bias, weight.shape[0]), act
        N, K = weight.shape
        self.w = Mx4Tensor.empty(N, K, weight.device)
        self.wt = Mx4Tensor.empty(K, N, weight.device)
        self.update()

    def update(self):
        mx4_quantize(self.weight, out=self.w)
        mx4_quantize(self.weight, transpose=True, out=self.wt)

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        return mx4_linear(x, self.w, self.bias, self.act)

    def backward(self, x: torch.Tensor, dy: torch.Tensor, y: torch.Tensor | None = None, want_x: bool = True) -> dict:
        """Gradients {x, weight, bias} for upstream dy; y is this layer's output (needed for ReLU)."""
        if self.act == "relu" and y is None:
            raise ValueError("a ReLU layer's backward needs its output y")
        return mx4_linear_backward(dy, x, self.wt, y if self.act == "relu" else None, want_x)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _here(*tensors):
    """The current stream's raw handle (None where torch has no call for it); refuses tensors that are not on the
    current GPU (None stands for no tensor)."""
    device = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError("the tensors must be on the current device")
    return None if _raw_stream is None else _raw_stream(device)


class Dropout:
    """Dropout with probability p whose mask is computed from the place of a
    value and stored nowhere: value (r, c) is kept, and divided by 1 - p, where
    word c mod 4 of Philox4x32-10 (counter (c // 4, r, offset), key seed) is at
    least p 2^32.  The same p, seed and offset give the same mask: each layer and
    each step takes an offset of its own, and the backward that of its forward.

    step: a device int64 tensor of one element that is added to offset when the
    work runs (not when it is enqueued), for captured graphs that are replayed.

    None of the four can be assigned: another p or offset is another Dropout."""

    __slots__ = ("_step", "c")

    def __init__(self, p: float, seed: int, offset: int = 0, step: torch.Tensor | None = None):
        if not 0.0 <= p <= 1.0:
            raise ValueError("p must be in [0, 1]")
        if not (0 <= seed < 2 ** 64 and 0 <= offset < 2 ** 64):
            raise ValueError("seed and offset must be in [0, 2^64)")
        if step is not None and (step.dtype != torch.int64 or step.numel() != 1 or not step.is_cuda):
            raise ValueError("step must be an int64 tensor of one element on the GPU")
        self._step, self.c = step, ia.Drop(p, seed, offset, None if step is None else step.data_ptr())

    # what the kernels read
    p = property(lambda self: self.c.p)
    seed = property(lambda self: self.c.seed)
    offset = property(lambda self: self.c.offset)
    step = property(lambda self: self._step)

    def __call__(self, x: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
        """x [rows, cols] (float32, float16 or bfloat16) with dropout; out may be x."""
        d, rows, cols, ldx = _matrix(x, "x")
        if out is None:
            out, ldo = x.new_empty((rows, cols)), cols
        else:
            do, r, c, ldo = _matrix(out, "out")
            if (do, r, c) != (d, rows, cols):
                raise ValueError("out has another shape or type")
        stream = _here(x, out, self._step)
        ia.ia_dropout(x, d, rows, cols, ldx, self.c, out, ldo, stream)
        return out

    def backward(self, dy: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
        """The input's gradient for upstream dy: the same values kept, the same factor."""
        return self(dy, out)


_INDEX_BYTES = {torch.int32: 4, torch.int64: 8}


def _index(index: torch.Tensor):
    """(bytes of an index, their number, their stride)."""
    b = _INDEX_BYTES.get(index.dtype)
    if b is None or index.dim() != 1 or not index.is_cuda:
        raise ValueError("index must be a 1-D int32 or int64 tensor on the GPU")
    return b, index.shape[0], index.stride(0)


def embedding(table, index: torch.Tensor, scale: float = 1.0, dtype=None, dropout: Dropout | None = None,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """scale * table[index], with dropout of the result where asked: [n, dim] of
    dtype (the table's type by default, float32 for an Mx4Tensor).  table is a
    [entries, dim] tensor (float32, float16 or bfloat16) or an Mx4Tensor, whose
    picked rows alone are read back.  An index outside [0, entries) gives a row
    of zeros."""
    b, n, between = _index(index)
    if packed := isinstance(table, Mx4Tensor):
        entries, dim, memory, own = table._rows, table._cols, table._codes, torch.float32
    else:
        d, entries, dim, ld = _matrix(table, "table")
        memory, own = table, table.dtype
    if out is None:
        out, ldo = memory.new_empty((n, dim), dtype=dtype or own), dim
        do = _dtype(out)
    else:
        do, rows, cols, ldo = _matrix(out, "out")
        if (rows, cols) != (n, dim) or dtype not in (None, out.dtype):
            raise ValueError("out has another shape or type")
    step, drop = (None, None) if dropout is None else (dropout._step, dropout.c)
    stream = _here(index, memory, out, step)
    if packed:
        ia.ia_embedding_mx4(table.c, index, b, n, between, scale, drop, do, out, ldo, stream)
    else:
        ia.ia_embedding(table, d, entries, dim, ld, index, b, n, between, scale, drop, do, out, ldo, stream)
    return out


def embedding_backward(dy: torch.Tensor, index: torch.Tensor, entries: int, scale: float = 1.0,
                       dropout: Dropout | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """The table's gradient [entries, dim] (float32, dense) of embedding(table,
    index, scale, dropout=dropout) for upstream dy [n, dim]: the sum of the rows
    that picked an entry, zeros where none did; the same on every run."""
    b, n, between = _index(index)
    d, rows, dim, ld = _matrix(dy, "dy")
    if rows != n:
        raise ValueError(f"dy has {rows} rows for {n} indices")
    if out is None:
        out = dy.new_empty((entries, dim), dtype=torch.float32)
    elif out.dtype != torch.float32 or out.shape != (entries, dim) or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous float32 [{entries}, {dim}]")
    step, drop = (None, None) if dropout is None else (dropout._step, dropout.c)
    stream = _here(index, dy, out, step)
    ws = _bytes(ia.ia_embedding_backward_workspace_size(n, entries, dim), dy.device)
    ia.ia_embedding_backward(dy, d, dim, ld, index, b, n, between, entries, scale, drop, out, ws, stream)
    return out


class Q4Tensor:
    """A [rows, cols] matrix in 4 bits with a scale and a zero for each group of
    32, 64 or 128 values of a row, which stand for scale * (code - zero): codes
    uint8 [rows, groups * group / 2] (two a byte, the earlier one in the low
    half), words int32 [rows, groups rounded up to 4] (the bits of the scale as a
    float32 whose lowest byte is zero, and in that byte the zero, 0..15).  The
    tensors and sizes are not replaced; the tensors' values may change (quantised anew)."""

    __slots__ = ("_codes", "_words", "_rows", "_cols", "_group", "c")

    def __init__(self, codes: torch.Tensor, words: torch.Tensor, cols: int, group: int):
        shapes = self._shapes(codes.shape[0], cols, group)
        if codes.dtype != torch.uint8 or words.dtype != torch.int32 or not codes.is_cuda or not words.is_cuda:
            raise ValueError("codes must be uint8 and words int32 tensors on the GPU")
        _one_device(codes, words)
        if (codes.shape, words.shape) != shapes or not codes.is_contiguous() or not words.is_contiguous():
            raise ValueError(f"codes {list(shapes[0])} and words {list(shapes[1])} expected, contiguous")
        self._set(codes, words, cols, group)

    @staticmethod
    def _shapes(rows: int, cols: int, group: int):
        if group not in (32, 64, 128):
            raise ValueError("groups are of 32, 64 or 128 values")
        groups = (cols + group - 1) // group
        return (rows, groups * group // 2), (rows, (groups + 3) // 4 * 4)

    def _set(self, codes, words, cols, group):
        self._codes, self._words, self._rows, self._cols, self._group = codes, words, codes.shape[0], cols, group
        self.c = ia.q4(codes, words, self._rows, cols, group)

    codes = property(lambda self: self._codes)
    words = property(lambda self: self._words)
    rows = property(lambda self: self._rows)
    cols = property(lambda self: self._cols)
    group = property(lambda self: self._group)

    @classmethod
    def empty(cls, rows: int, cols: int, group: int = 128, device="cuda"):
        codes, words = cls._shapes(rows, cols, group)
        q = cls.__new__(cls)
        q._set(torch.empty(codes, dtype=torch.uint8, device=device), torch.empty(words, dtype=torch.int32, device=device),
               cols, group)
        return q

    @classmethod
    def from_parts(cls, codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | int, cols: int, group: int):
        """From codes and [rows, groups] tensors of scales (NaN or, rounded to 16
        significant bits, finite floats, so exact for float16 and bfloat16) and of
        zeros in 0..15 (or one zero for all).  Looks at both on the host: it waits
        for the GPU."""
        (rows, _), _ = cls._shapes(codes.shape[0], cols, group)
        shape = (rows, (cols + group - 1) // group)
        if scales.shape != shape:  # the constructor sees the padded words only
            raise ValueError(f"scales {list(shape)} expected, got {list(scales.shape)}")
        bits = scales.to(torch.float32).contiguous().view(torch.int32)
        bits = torch.where(torch.isnan(scales), 0x7fc00000, (bits + 127 + ((bits >> 8) & 1)) & ~255)
        if bool(torch.isinf(bits.view(torch.float32)).any()):
            raise ValueError("scales must be NaN or finite as floats of 16 significant bits")
        zeros = torch.as_tensor(zeros, device=scales.device)
        if zeros.dtype.is_floating_point or bool(((zeros < 0) | (zeros > 15)).any()):
            raise ValueError("zeros must be whole numbers in 0..15")
        if any(z not in (1, n) for z, n in zip(zeros.shape[::-1], shape[::-1])) or zeros.dim() > 2:
            raise ValueError(f"zeros {list(shape)} or one for all expected, got {list(zeros.shape)}")
        words = bits | zeros.to(torch.int32)
        return cls(codes, torch.nn.functional.pad(words, (0, -words.shape[1] % 4)).contiguous(), cols, group)

    @property
    def scales(self) -> torch.Tensor:
        """[rows, groups] float32."""
        return (self._words[:, :(self.cols + self.group - 1) // self.group] & ~255).view(torch.float32)

    @property
    def zeros(self) -> torch.Tensor:
        """[rows, groups] int32."""
        return self._words[:, :(self.cols + self.group - 1) // self.group] & 255

    def dequantize(self, dtype=torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
        """The values, rounded once to dtype (float32, float16 or bfloat16)."""
        if out is None:
            out, ld = self._codes.new_empty((self._rows, self._cols), dtype=dtype), self._cols
            d = _dtype(out)
        else:
            d, rows, cols, ld = _matrix(out, "out")
            if (rows, cols) != (self.rows, self.cols):
                raise ValueError("out has another shape")
        stream = _here(out, self._codes)
        ia.ia_q4_dequantize(self.c, d, out, ld, stream)
        return out


def q4_quantize(x: torch.Tensor, group: int = 128, out: Q4Tensor | None = None) -> Q4Tensor:
    """x [rows, cols] in 4 bits with a scale and a zero for each group of a row:
    scale = (greatest - least) / 15, zero included, codes rounded to nearest.
    With out (whose groups count) its tensors are filled anew."""
    d, rows, cols, ld = _matrix(x, "x")
    if out is None:
        out = Q4Tensor.empty(rows, cols, group, x.device)
    elif (out.rows, out.cols) != (rows, cols):
        raise ValueError("out has another shape")
    stream = _here(x, out._codes)
    ia.ia_q4_quantize(x, d, ld, out.c, stream)
    return out


def q4_linear(x: torch.Tensor, w: Q4Tensor, bias: torch.Tensor | None = None, act: str = "none",
              out: torch.Tensor | None = None) -> torch.Tensor:
    """A linear layer with 4-bit weights and its input as it is: act(x w^T +
    bias), x [M, K], w [N, K]; returns [M, N] of x's type; act "none" or "relu"."""
    d, M, K, ldx = _matrix(x, "x")
    N = w._rows
    if K != w._cols:
        raise ValueError(f"x has {K} columns, the weights {w._cols}")
    if out is None:
        out, ldy = x.new_empty((M, N)), N
    else:
        do, rows, cols, ldy = _matrix(out, "out")
        if (do, rows, cols) != (d, M, N):
            raise ValueError("out has another shape or type")
    stream = _here(x, w._codes, bias, out)
    ws = _bytes(ia.ia_q4_linear_workspace_size(d, M, K, N), x.device)
    ia.ia_q4_linear(x, d, M, ldx, w.c, _bias(bias, N), _ACTS[act], out, ldy, ws, stream)
    return out
