"""Python binding of libzopt: one rank's ZeRO-style optimizer step on MI355X.

Argument marshalling only.  Every step of the computation runs in the HIP
kernels of ``libzopt.so`` (built from ``csrc/`` by ``build.py``); this module
checks tensor dtypes, devices and sizes (the C ABI takes plain pointers and
cannot), passes pointers and the current HIP stream, and turns status codes
into exceptions.  PyTorch only supplies device memory and streams.  If the
library is not built, importing the entry points raises -- there is no
fallback.

Entry points (same names as the C ABI in include/zopt.h):
  adamw_shard_step   fused AdamW over a flat bucketed fp32 shard
  muon_step          Muon on a batch of same-shape matrices
  muon_workspace_bytes / muon_output_view
  muon_step_groups   Muon on several such batches in one call (shared launches);
                     with ns_guard: zopt_muon_step_groups_guarded (health checks)
  MuonGraph          a Muon call captured once (zopt_muon_graph_*), replayed per step
                     with lr / momentum / weight decay read from device memory
  muon_groups_workspace_bytes / muon_groups_output_view
  round_bf16         fp32 -> bf16 round-to-nearest-even
  shard_len          the shard length the layout derives (zopt_shard_len)
  grad_sq_norm       sum of squares of a rank's real gradient elements
  grad_sq_norm_noalloc  the same with the library's own scratch (allocates nothing)
  grad_clip_stats    clip statistics (device scalars) from summed squares
  adamw_shard_step_clipped   AdamW taking grad_scale from the clip statistics
  linear_xent_loss / linear_xent_grad   cross entropy of a vocabulary projection,
                     alone or with its gradients, from x and w (zopt_linear_xent)
  glu_forward / glu_backward   the gated feed-forward block's gate / up part
  act8_pack / act8_unpack / act8_wgrad   activation checkpoints in 8 bits (Act8)

Every entry point stands outside autograd: it records nothing, whatever
requires_grad says of its arguments, and the caller passes gradients on.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libzopt.so")

ZOPT_OK, ZOPT_ERR_NULL, ZOPT_ERR_SIZE, ZOPT_ERR_HYPER, ZOPT_ERR_WORKSPACE, ZOPT_ERR_DEVICE = range(6)
# layout of the clip statistics (ZOPT_CLIP_* in zopt.h)
CLIP_TOTAL_NORM, CLIP_COEF, CLIP_CLIPPED, CLIP_FOUND_INF, CLIP_GRAD_SCALE, CLIP_STATS = range(6)
MAX_BATCH = 64
MAX_GROUPS = 16


class ZoptError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib_or_raise().zopt_status_string(status).decode()
        super().__init__(f"{where}: {msg}")


_lib = None


def _lib_or_raise() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is not built; run `python -m sharded_optimizer_step_adamw_amd.build` "
                "(or __graft_entry__.build()). There is no CPU fallback.")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
        L.zopt_status_string.argtypes = [ctypes.c_int]
        L.zopt_status_string.restype = ctypes.c_char_p
        L.zopt_adamw_shard_step.argtypes = [vp, vp, vp, vp, vp, i64, i64, i32, i32, i64,
                                            f32, f32, f32, f32, f32, i64, f32, vp]
        L.zopt_adamw_shard_step.restype = ctypes.c_int
        L.zopt_adamw_shard_step_clipped.argtypes = [vp, vp, vp, vp, vp, i64, i64, i32, i32,
                                                    i64, f32, f32, f32, f32, f32, i64, vp, i32,
                                                    vp]
        L.zopt_adamw_shard_step_clipped.restype = ctypes.c_int
        L.zopt_grad_sq_norm.argtypes = [vp, i64, i64, i32, i32, i64, vp, vp,
                                        ctypes.POINTER(ctypes.c_size_t), vp]
        L.zopt_grad_sq_norm.restype = ctypes.c_int
        L.zopt_grad_sq_norm_noalloc.argtypes = [vp, i64, i64, i32, i32, i64, vp, vp]
        L.zopt_grad_sq_norm_noalloc.restype = ctypes.c_int
        L.zopt_grad_clip_stats.argtypes = [vp, i32, f32, f32, vp, vp]
        L.zopt_grad_clip_stats.restype = ctypes.c_int
        L.zopt_shard_len.argtypes = [i64, i64, i32]
        L.zopt_shard_len.restype = i64
        L.zopt_round_bf16.argtypes = [vp, vp, i64, vp]
        L.zopt_round_bf16.restype = ctypes.c_int
        L.zopt_set_ns_workgroup_limit.argtypes = [i32]
        L.zopt_set_ns_workgroup_limit.restype = ctypes.c_int
        L.zopt_set_ns_form.argtypes = [i32]
        L.zopt_set_ns_form.restype = ctypes.c_int
        pp = ctypes.POINTER(vp)
        L.zopt_muon_step.argtypes = [i32, i64, i64, pp, pp, pp, pp, f32, f32, i32, f32, i32,
                                     f32, f32, f32, f32, i32, vp,
                                     ctypes.POINTER(ctypes.c_size_t), vp]
        L.zopt_muon_step.restype = ctypes.c_int
        L.zopt_muon_output_view.argtypes = [i32, i64, i64, i32, vp, i32, pp,
                                            ctypes.POINTER(i64)]
        L.zopt_muon_output_view.restype = ctypes.c_int
        pi32, pi64 = ctypes.POINTER(i32), ctypes.POINTER(i64)
        L.zopt_muon_step_groups.argtypes = [i32, pi32, pi64, pi64, pp, pp, pp, pp, f32, f32, i32,
                                            f32, i32, f32, f32, f32, f32, i32, vp,
                                            ctypes.POINTER(ctypes.c_size_t), vp]
        L.zopt_muon_step_groups.restype = ctypes.c_int
        L.zopt_muon_step_groups_guarded.argtypes = [
            i32, pi32, pi64, pi64, pp, pp, pp, pp, f32, f32, i32, f32, i32, f32, f32, f32, f32,
            i32, f32, vp, vp, ctypes.POINTER(ctypes.c_size_t), vp]
        L.zopt_muon_step_groups_guarded.restype = ctypes.c_int
        L.zopt_muon_graph_create.argtypes = [
            i32, pi32, pi64, pi64, pp, pp, pp, pp, vp, i32, i32, f32, f32, f32, f32, i32, f32,
            vp, vp, ctypes.c_size_t, ctypes.POINTER(vp)]
        L.zopt_muon_graph_create.restype = ctypes.c_int
        L.zopt_muon_graph_launch.argtypes = [vp, vp]
        L.zopt_muon_graph_launch.restype = ctypes.c_int
        L.zopt_muon_graph_destroy.argtypes = [vp]
        L.zopt_muon_graph_destroy.restype = ctypes.c_int
        L.zopt_muon_groups_output_view.argtypes = [i32, pi32, pi64, pi64, i32, vp, i32, i32, pp,
                                                   pi64]
        L.zopt_muon_groups_output_view.restype = ctypes.c_int
        size_p = ctypes.POINTER(ctypes.c_size_t)
        L.zopt_linear_xent.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, i32, f32, vp, vp,
                                       vp, i64, vp, i64, vp, size_p, vp]
        L.zopt_act8_pack.argtypes = [i64, i64, vp, i64, vp, vp, vp]
        L.zopt_act8_unpack.argtypes = [i64, i64, vp, vp, vp, i64, vp]
        L.zopt_act8_wgrad.argtypes = [i64, i64, i64, vp, i64, vp, vp, vp, i64, vp, size_p, vp]
        L.zopt_glu_forward.argtypes = [i64, i64, i64, vp, i64, vp, vp, i64, i32, vp, i64, vp, vp,
                                       vp, vp, vp, size_p, vp]
        L.zopt_glu_backward.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, vp, vp, vp, i64, i32,
                                        vp, vp, vp, vp, vp, i64, vp, i64, vp, vp, i64, vp, size_p,
                                        vp]
        for f in (L.zopt_linear_xent, L.zopt_act8_pack, L.zopt_act8_unpack, L.zopt_act8_wgrad,
                  L.zopt_glu_forward, L.zopt_glu_backward):
            f.restype = ctypes.c_int
        _lib = L
    return _lib


def lib() -> ctypes.CDLL:
    """The loaded libzopt (raises ImportError if it is not built)."""
    return _lib_or_raise()


def _stream(device: torch.device, stream) -> int:
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _need(t: torch.Tensor, dtype, numel: int, name: str, device=None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, need {dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name}: has {t.numel()} elements, needs {numel}")


def _check(status: int, where: str) -> None:
    if status != ZOPT_OK:
        raise ZoptError(status, where)


def shard_len(n: int, bucket: int, world: int) -> int:
    """Shard length every rank holds (zopt_shard_len)."""
    v = lib().zopt_shard_len(n, bucket, world)
    if v < 0:
        raise ValueError("shard_len: need n, bucket, world >= 1")
    return int(v)


def adamw_shard_step(master, exp_avg, exp_avg_sq, grad, weight, n, bucket, world, rank,
                     lr, beta1, beta2, eps, weight_decay, step, grad_scale=1.0,
                     shard_len_=None, stream=None) -> None:
    """One fused AdamW step over rank `rank`'s shard (zopt_adamw_shard_step).
    master/exp_avg/exp_avg_sq: fp32 [shard_len]; grad: bf16 [n]; weight:
    bf16 [n] or None."""
    sl = shard_len(n, bucket, world) if shard_len_ is None else shard_len_
    dev = master.device
    _need(master, torch.float32, sl, "master")
    _need(exp_avg, torch.float32, sl, "exp_avg", dev)
    _need(exp_avg_sq, torch.float32, sl, "exp_avg_sq", dev)
    _need(grad, torch.bfloat16, n, "grad", dev)
    if weight is not None:
        _need(weight, torch.bfloat16, n, "weight", dev)
    st = lib().zopt_adamw_shard_step(
        master.data_ptr(), exp_avg.data_ptr(), exp_avg_sq.data_ptr(), grad.data_ptr(),
        None if weight is None else weight.data_ptr(), n, bucket, world, rank, sl,
        lr, beta1, beta2, eps, weight_decay, step, grad_scale, _stream(dev, stream))
    _check(st, "zopt_adamw_shard_step")


def adamw_shard_step_clipped(master, exp_avg, exp_avg_sq, grad, weight, n, bucket, world, rank,
                             lr, beta1, beta2, eps, weight_decay, step, clip_stats,
                             skip_nonfinite=False, shard_len_=None, stream=None) -> None:
    """adamw_shard_step with grad_scale read from the device clip statistics
    (fp32 [CLIP_STATS]) when the kernel runs (zopt_adamw_shard_step_clipped)."""
    sl = shard_len(n, bucket, world) if shard_len_ is None else shard_len_
    dev = master.device
    _need(master, torch.float32, sl, "master")
    _need(exp_avg, torch.float32, sl, "exp_avg", dev)
    _need(exp_avg_sq, torch.float32, sl, "exp_avg_sq", dev)
    _need(grad, torch.bfloat16, n, "grad", dev)
    _need(clip_stats, torch.float32, CLIP_STATS, "clip_stats", dev)
    if weight is not None:
        _need(weight, torch.bfloat16, n, "weight", dev)
    st = lib().zopt_adamw_shard_step_clipped(
        master.data_ptr(), exp_avg.data_ptr(), exp_avg_sq.data_ptr(), grad.data_ptr(),
        None if weight is None else weight.data_ptr(), n, bucket, world, rank, sl,
        lr, beta1, beta2, eps, weight_decay, step, clip_stats.data_ptr(), int(skip_nonfinite),
        _stream(dev, stream))
    _check(st, "zopt_adamw_shard_step_clipped")


def grad_sq_norm_workspace_bytes(n: int, bucket: int, world: int, rank: int = 0) -> int:
    size = ctypes.c_size_t(0)
    st = lib().zopt_grad_sq_norm(None, n, bucket, world, rank, shard_len(n, bucket, world),
                                 None, None, ctypes.byref(size), None)
    _check(st, "zopt_grad_sq_norm(workspace query)")
    return int(size.value)


def grad_sq_norm(grad, n, bucket, world, rank, out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Sum of squares of rank `rank`'s real gradient elements, as a float64
    [1] device tensor (zopt_grad_sq_norm); nothing is read back."""
    dev = grad.device
    _need(grad, torch.bfloat16, n, "grad")
    if out is None:
        out = _On(dev, stream).empty(1, torch.float64)
    _need(out, torch.float64, 1, "out", dev)
    need = grad_sq_norm_workspace_bytes(n, bucket, world, rank)
    if workspace is None:
        workspace = _On(dev, stream).empty(need, torch.uint8)
    _need(workspace, torch.uint8, need, "workspace", dev)
    size = ctypes.c_size_t(workspace.numel())
    st = lib().zopt_grad_sq_norm(grad.data_ptr(), n, bucket, world, rank,
                                 shard_len(n, bucket, world), out.data_ptr(),
                                 workspace.data_ptr(), ctypes.byref(size), _stream(dev, stream))
    _check(st, "zopt_grad_sq_norm")
    return out


def grad_sq_norm_noalloc(grad, n, bucket, world, rank, out: torch.Tensor,
                         stream=None) -> torch.Tensor:
    """grad_sq_norm with the library's own 16 KiB scratch per GPU instead of
    a workspace (zopt_grad_sq_norm_noalloc): `out` is a float64 [1] device
    tensor the caller provides, and the call allocates nothing.  Calls that
    overlap on one GPU race on the scratch."""
    _need(grad, torch.bfloat16, n, "grad")
    _need(out, torch.float64, 1, "out", grad.device)
    st = lib().zopt_grad_sq_norm_noalloc(grad.data_ptr(), n, bucket, world, rank,
                                         shard_len(n, bucket, world), out.data_ptr(),
                                         _stream(grad.device, stream))
    _check(st, "zopt_grad_sq_norm_noalloc")
    return out


def grad_clip_stats(sq: torch.Tensor, max_norm: float, inv_scale: float = 1.0,
                    out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Clip statistics (fp32 [CLIP_STATS] device tensor: total_norm,
    clip_coef, clipped, found_inf, grad_scale) from the float64 sums of
    squares in `sq`, added in order (zopt_grad_clip_stats)."""
    dev = sq.device
    _need(sq, torch.float64, 1, "sq")
    if out is None:
        out = _On(dev, stream).empty(CLIP_STATS, torch.float32)
    _need(out, torch.float32, CLIP_STATS, "out", dev)
    st = lib().zopt_grad_clip_stats(sq.data_ptr(), sq.numel(), max_norm, inv_scale,
                                    out.data_ptr(), _stream(dev, stream))
    _check(st, "zopt_grad_clip_stats")
    return out


def round_bf16(src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    """dst = bf16(src), round to nearest even (zopt_round_bf16)."""
    n = src.numel()
    _need(src, torch.float32, n, "src")
    _need(dst, torch.bfloat16, n, "dst", src.device)
    st = lib().zopt_round_bf16(src.data_ptr(), dst.data_ptr(), n, _stream(src.device, stream))
    _check(st, "zopt_round_bf16")


def set_ns_workgroup_limit(n: int) -> None:
    """Caps the workgroups the persistent Newton-Schulz B X launches keep
    resident (0: a full round of the device); process-wide
    (zopt_set_ns_workgroup_limit)."""
    _check(lib().zopt_set_ns_workgroup_limit(int(n)), "zopt_set_ns_workgroup_limit")


NS_FORM_AUTO, NS_FORM_PLAIN, NS_FORM_GRAM_BF16 = 0, 1, 2


def set_ns_form(form: int) -> None:
    """Newton-Schulz form of later calls: NS_FORM_AUTO (segments on the Gram
    matrix for groups with n >= 2 m, m <= 4096 and batch m^2 (n - m) >= 2^29, the m x m
    chain in fp16 where the coefficients allow), NS_FORM_PLAIN (plain
    iterations throughout) or NS_FORM_GRAM_BF16 (as AUTO, chain in bf16)
    (zopt_set_ns_form)."""
    _check(lib().zopt_set_ns_form(int(form)), "zopt_set_ns_form")


def _ptr_array(tensors) -> ctypes.Array:
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def _check_matrices(lists, shape, device, prefix=""):
    """Every tensor of `lists` [(tensors, dtype, name)] is a contiguous GPU
    tensor of that dtype and `shape` on `device`: one combined test per
    tensor, and the detailed checks (for the error message) only where it
    fails."""
    index = device.index if device.type == "cuda" else -2
    for tensors, dt, nm in lists:
        for i, t in enumerate(tensors):
            if not (isinstance(t, torch.Tensor) and t.dtype == dt and t.is_cuda
                    and t.get_device() == index and t.shape == shape and t.is_contiguous()):
                name = f"{prefix}{nm}[{i}]"
                _need(t, dt, shape[0] * shape[1], name, device)
                raise ValueError(f"{name}: shape {tuple(t.shape)}, need {tuple(shape)}")


def muon_workspace_bytes(batch: int, rows: int, cols: int) -> int:
    size = ctypes.c_size_t(0)
    st = lib().zopt_muon_step(batch, rows, cols, None, None, None, None, 0.0, 0.0, 0, 0.0, 0,
                              0.0, 0.0, 0.0, 0.0, 0, None, ctypes.byref(size), None)
    _check(st, "zopt_muon_step(workspace query)")
    return int(size.value)


def muon_step(master: Sequence[torch.Tensor], momentum: Sequence[torch.Tensor],
              grad: Sequence[torch.Tensor], weight: Optional[Sequence[torch.Tensor]],
              lr: float, momentum_beta: float = 0.95, nesterov: bool = True,
              weight_decay: float = 0.1, ns_steps: int = 5,
              ns_coeffs=(3.4445, -4.7750, 2.0315), ns_eps: float = 1e-7,
              adjust_lr: int = 1, workspace: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """One Muon step on a batch of same-shape [rows, cols] matrices
    (zopt_muon_step).  master, momentum: fp32; grad, weight: bf16.  Returns
    the workspace (allocated with torch if not given), which holds the
    orthogonalised updates (see muon_output_view)."""
    batch = len(master)
    if not (1 <= batch <= MAX_BATCH) or len(momentum) != batch or len(grad) != batch or (
            weight is not None and len(weight) != batch):
        raise ValueError("muon_step: need 1..64 matrices and equal-length lists")
    shape = master[0].shape
    rows, cols = shape
    dev = master[0].device
    _check_matrices(((master, torch.float32, "master"), (momentum, torch.float32, "momentum"),
                     (grad, torch.bfloat16, "grad"))
                    + (((weight, torch.bfloat16, "weight"),) if weight is not None else ()),
                    shape, dev)
    need = muon_workspace_bytes(batch, rows, cols)
    if workspace is None:
        workspace = _On(dev, stream).empty(need, torch.uint8)
    _need(workspace, torch.uint8, need, "workspace", dev)
    size = ctypes.c_size_t(workspace.numel())
    a, b, c = (float(x) for x in ns_coeffs)
    st = lib().zopt_muon_step(
        batch, rows, cols, _ptr_array(master), _ptr_array(momentum), _ptr_array(grad),
        None if weight is None else _ptr_array(weight), lr, momentum_beta, int(nesterov),
        weight_decay, ns_steps, a, b, c, ns_eps, adjust_lr, workspace.data_ptr(),
        ctypes.byref(size), _stream(dev, stream))
    _check(st, "zopt_muon_step")
    return workspace


def muon_output_view(workspace: torch.Tensor, batch: int, rows: int, cols: int,
                     ns_steps: int, index: int) -> torch.Tensor:
    """The bf16 [rows, cols] orthogonalised update of matrix `index` inside a
    workspace filled by muon_step (a strided view, not a copy)."""
    out = ctypes.c_void_p(0)
    ld = ctypes.c_int64(0)
    st = lib().zopt_muon_output_view(batch, rows, cols, ns_steps, workspace.data_ptr(), index,
                                     ctypes.byref(out), ctypes.byref(ld))
    _check(st, "zopt_muon_output_view")
    off = out.value - workspace.data_ptr()
    assert off % 2 == 0 and off >= 0
    flat = workspace.view(torch.bfloat16)
    return flat.as_strided((rows, cols), (ld.value, 1), off // 2)


def _shape_arrays(shapes):
    n = len(shapes)
    if not (1 <= n <= MAX_GROUPS):
        raise ValueError(f"need 1..{MAX_GROUPS} groups, got {n}")
    b = (ctypes.c_int32 * n)(*[int(x[0]) for x in shapes])
    r = (ctypes.c_int64 * n)(*[int(x[1]) for x in shapes])
    c = (ctypes.c_int64 * n)(*[int(x[2]) for x in shapes])
    return n, b, r, c


def muon_groups_workspace_bytes(shapes: Sequence[tuple]) -> int:
    """Workspace bytes of a zopt_muon_step_groups call over groups given as
    (batch, rows, cols)."""
    n, b, r, c = _shape_arrays(shapes)
    size = ctypes.c_size_t(0)
    st = lib().zopt_muon_step_groups(n, b, r, c, None, None, None, None, 0.0, 0.0, 0, 0.0, 0,
                                     0.0, 0.0, 0.0, 0.0, 0, None, ctypes.byref(size), None)
    _check(st, "zopt_muon_step_groups(workspace query)")
    return int(size.value)


def muon_step_groups(groups: Sequence[tuple], lr: float, momentum_beta: float = 0.95,
                     nesterov: bool = True, weight_decay: float = 0.1, ns_steps: int = 5,
                     ns_coeffs=(3.4445, -4.7750, 2.0315), ns_eps: float = 1e-7,
                     adjust_lr: int = 1, workspace: Optional[torch.Tensor] = None,
                     stream=None, ns_guard: Optional[float] = None,
                     ns_health: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One Muon step on several groups of same-shape matrices in one call
    (zopt_muon_step_groups).  Each group is (master, momentum, grad, weight)
    with lists of equal length; weight may be None for every group or for
    none.  Returns the workspace (see muon_groups_output_view).

    With ns_guard (and ns_health, fp32 [2 + 3 * matrices] on the device) the
    call is zopt_muon_step_groups_guarded: ns_health receives the number of
    rejected matrices, the worst passing ratio and [ratio, absmax, rejected]
    per matrix, and a rejected matrix is not updated."""
    shapes, M, Mo, G, W, with_w, dev = _muon_group_tables(groups)
    need = muon_groups_workspace_bytes(shapes)
    if workspace is None:
        workspace = _On(dev, stream).empty(need, torch.uint8)
    _need(workspace, torch.uint8, need, "workspace", dev)
    n, b, r, c = _shape_arrays(shapes)
    size = ctypes.c_size_t(workspace.numel())
    ca, cb, cc = (float(x) for x in ns_coeffs)
    common = (n, b, r, c, _ptr_array(M), _ptr_array(Mo), _ptr_array(G),
              _ptr_array(W) if with_w else None, lr, momentum_beta, int(nesterov), weight_decay,
              ns_steps, ca, cb, cc, ns_eps, adjust_lr)
    if ns_guard is None:
        if ns_health is not None:
            raise ValueError("muon_step_groups: ns_health needs ns_guard")
        st = lib().zopt_muon_step_groups(*common, workspace.data_ptr(), ctypes.byref(size),
                                         _stream(dev, stream))
        _check(st, "zopt_muon_step_groups")
        return workspace
    if ns_health is None:
        raise ValueError("muon_step_groups: ns_guard needs an ns_health tensor")
    _need(ns_health, torch.float32, 2 + 3 * len(M), "ns_health", dev)
    st = lib().zopt_muon_step_groups_guarded(*common, ns_guard, ns_health.data_ptr(),
                                             workspace.data_ptr(), ctypes.byref(size),
                                             _stream(dev, stream))
    _check(st, "zopt_muon_step_groups_guarded")
    return workspace


def _muon_group_tables(groups):
    """Checks the (master, momentum, grad, weight) groups of a Muon call and
    flattens them: (shapes, masters, momenta, grads, weights, with_weights,
    device)."""
    if not groups:
        raise ValueError("muon_step_groups: no groups")
    with_w = groups[0][3] is not None
    shapes, M, Mo, G, W = [], [], [], [], []
    dev = groups[0][0][0].device
    for gi, (master, momentum, grad, weight) in enumerate(groups):
        batch = len(master)
        if not (1 <= batch <= MAX_BATCH) or len(momentum) != batch or len(grad) != batch:
            raise ValueError(f"group {gi}: need 1..64 matrices and equal-length lists")
        if (weight is not None) != with_w or (weight is not None and len(weight) != batch):
            raise ValueError(f"group {gi}: weight lists must be given for all groups or none")
        shape = master[0].shape
        rows, cols = shape
        _check_matrices(((master, torch.float32, "master"), (momentum, torch.float32, "momentum"),
                         (grad, torch.bfloat16, "grad"))
                        + (((weight, torch.bfloat16, "weight"),) if weight is not None else ()),
                        shape, dev, f"group {gi} ")
        shapes.append((batch, rows, cols))
        M += list(master)
        Mo += list(momentum)
        G += list(grad)
        if with_w:
            W += list(weight)
    return shapes, M, Mo, G, W, with_w, dev


class MuonGraph:
    """One Muon call over `groups` captured as a hipGraph
    (zopt_muon_graph_create), replayed by launch() (zopt_muon_graph_launch).
    lr, momentum_beta and weight_decay are read from `scalars` (fp32 [3] on
    the device) each time the graph runs: write new values there (a copy or
    fill on the stream) to change them.  The tensors given are kept alive
    while the graph exists; close() (or garbage collection) synchronises the
    device and frees the graph."""

    def __init__(self, groups, scalars: torch.Tensor, nesterov: bool = True, ns_steps: int = 5,
                 ns_coeffs=(3.4445, -4.7750, 2.0315), ns_eps: float = 1e-7, adjust_lr: int = 1,
                 workspace: Optional[torch.Tensor] = None, ns_guard: Optional[float] = None,
                 ns_health: Optional[torch.Tensor] = None):
        shapes, M, Mo, G, W, with_w, dev = _muon_group_tables(groups)
        _need(scalars, torch.float32, 3, "scalars", dev)
        need = muon_groups_workspace_bytes(shapes)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        _need(workspace, torch.uint8, need, "workspace", dev)
        if (ns_guard is None) != (ns_health is None):
            raise ValueError("MuonGraph: give ns_guard and ns_health together")
        if ns_health is not None:
            _need(ns_health, torch.float32, 2 + 3 * len(M), "ns_health", dev)
        n, b, r, c = _shape_arrays(shapes)
        ca, cb, cc = (float(x) for x in ns_coeffs)
        handle = ctypes.c_void_p()
        st = lib().zopt_muon_graph_create(
            n, b, r, c, _ptr_array(M), _ptr_array(Mo), _ptr_array(G),
            _ptr_array(W) if with_w else None, scalars.data_ptr(), int(nesterov), ns_steps,
            ca, cb, cc, ns_eps, adjust_lr, 0.0 if ns_guard is None else ns_guard,
            None if ns_health is None else ns_health.data_ptr(), workspace.data_ptr(),
            workspace.numel(), ctypes.byref(handle))
        _check(st, "zopt_muon_graph_create")
        self._handle = handle
        self.device = dev
        self.shapes = shapes
        self.ns_steps = ns_steps
        self.workspace = workspace
        self._keep = (groups, scalars, ns_health)

    def launch(self, stream=None) -> None:
        if self._handle is None:
            raise RuntimeError("MuonGraph: closed")
        _check(lib().zopt_muon_graph_launch(self._handle, _stream(self.device, stream)),
               "zopt_muon_graph_launch")

    def close(self) -> None:
        if getattr(self, "_handle", None) is not None:
            torch.cuda.synchronize(self.device)
            _check(lib().zopt_muon_graph_destroy(self._handle), "zopt_muon_graph_destroy")
            self._handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def muon_groups_output_view(workspace: torch.Tensor, shapes: Sequence[tuple], ns_steps: int,
                            group: int, index: int) -> torch.Tensor:
    """The bf16 [rows, cols] orthogonalised update of matrix `index` of group
    `group` inside a workspace filled by muon_step_groups (a strided view)."""
    n, b, r, c = _shape_arrays(shapes)
    out = ctypes.c_void_p(0)
    ld = ctypes.c_int64(0)
    st = lib().zopt_muon_groups_output_view(n, b, r, c, ns_steps, workspace.data_ptr(), group,
                                            index, ctypes.byref(out), ctypes.byref(ld))
    _check(st, "zopt_muon_groups_output_view")
    off = out.value - workspace.data_ptr()
    assert off % 2 == 0 and off >= 0
    rows, cols = int(shapes[group][1]), int(shapes[group][2])
    return workspace.view(torch.bfloat16).as_strided((rows, cols), (ld.value, 1), off // 2)


__all__ = ["adamw_shard_step", "adamw_shard_step_clipped", "grad_sq_norm", "grad_sq_norm_noalloc",
           "grad_sq_norm_workspace_bytes", "grad_clip_stats", "muon_step", "muon_workspace_bytes",
           "muon_output_view", "muon_step_groups", "muon_groups_workspace_bytes",
           "muon_groups_output_view", "MuonGraph", "set_ns_workgroup_limit", "set_ns_form",
           "linear_xent_loss", "linear_xent_grad", "glu_forward", "glu_backward", "act8_pack",
           "act8_unpack", "act8_wgrad", "Act8", "ACTIVATIONS", "round_bf16", "shard_len", "lib",
           "ZoptError", "LIB_PATH", "MAX_BATCH", "MAX_GROUPS"]


# ------------------------------------------------------ operators of the gradients

ACTIVATIONS = {"silu": 0, "gelu": 1}


class Act8(NamedTuple):
    """A bf16 matrix [rows, cols] kept in 8 bits: q, float8_e4m3fn [rows,
    cols], and scale, uint8 [rows, ceil(cols / 32)]; an element is
    q * 2^(scale - 127) (zopt_act8_pack)."""
    q: torch.Tensor
    scale: torch.Tensor


def _need_rows(t, dtype, rows, cols, name, device=None) -> int:
    """Checks that t is a GPU matrix [rows, cols] of dtype with contiguous
    rows (None: any size there) and returns its row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, need {dtype}")
    shape = t.shape
    if len(shape) != 2 or (rows is not None and shape[0] != rows) or (
            cols is not None and shape[1] != cols):
        want = tuple("any" if s is None else s for s in (rows, cols))
        raise ValueError(f"{name}: shape {tuple(shape)}, need {want}")
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"{name}: must be a GPU tensor")
    if device is not None and dev != device:
        raise ValueError(f"{name}: on {dev}, expected {device}")
    r, c = shape
    if c == 0:
        raise ValueError(f"{name}: rows are empty")
    s0, s1 = t.stride()
    if c > 1 and s1 != 1 or r > 1 and s0 < c:
        raise ValueError(f"{name}: strides {(s0, s1)}, need contiguous rows that do not overlap")
    return s0 if r > 1 else c


def _need_act8(a, rows, cols, name, device=None) -> None:
    if not isinstance(a, Act8):
        raise TypeError(f"{name}: expected an Act8")
    _need_rows(a.q, torch.float8_e4m3fn, rows, cols, f"{name}.q", device)
    r, c = a.q.shape
    _need_rows(a.scale, torch.uint8, r, (c + 31) // 32, f"{name}.scale", a.q.device)
    if not a.q.is_contiguous() or not a.scale.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _ptr(t):
    return None if t is None else t.data_ptr()


class _On:
    """The stream of a call, and where its outputs and workspace come from when
    the caller gives none: memory of the call's own stream, so that the
    allocator reuses it only after the call."""

    def __init__(self, device, stream):
        self.device = device
        current = torch._C._cuda_getCurrentRawStream(device.index)
        self.handle = current if stream is None else _stream(device, stream)
        self.other = self.handle != current

    def empty(self, shape, dtype, ld=None):
        """(ld: the row stride of a matrix, its width if not given)"""
        if not self.other:
            return self._empty(shape, dtype, ld)
        # (the default stream's handle is 0, and an ExternalStream of 0 is a new
        # stream of torch's own pool, whose memory the call does not order)
        stream = (torch.cuda.ExternalStream(self.handle, device=self.device) if self.handle else
                  torch.cuda.default_stream(self.device))
        with torch.cuda.stream(stream):
            return self._empty(shape, dtype, ld)

    def _empty(self, shape, dtype, ld):
        if ld is None or ld == shape[1]:
            return torch.empty(shape, dtype=dtype, device=self.device)
        return torch.empty_strided(shape, (ld, 1), dtype=dtype, device=self.device)


def _sized(fn, args, where, on, workspace):
    """Runs fn(*args, workspace, size, stream), with a workspace of the size
    that the same call asks for if none is given."""
    size = ctypes.c_size_t(0)
    if workspace is None:
        _check(fn(*args, None, ctypes.byref(size), None), where)
        if size.value == 0:  # any address will do
            _check(fn(*args, 256, ctypes.byref(size), on.handle), where)
            return
        workspace = on.empty(size.value, torch.uint8)
    else:
        _need(workspace, torch.uint8, 0, "workspace", on.device)
        size.value = workspace.numel()
    _check(fn(*args, workspace.data_ptr(), ctypes.byref(size), on.handle), where)


def _linear_xent(x, w, target, ignore_index, mean, grad_scale, loss, row_loss, dx, dw, want_dx,
                 want_dw, workspace, stream):
    ldx = _need_rows(x, torch.bfloat16, None, None, "x")
    dev = x.device
    T, D = x.shape
    ldw = _need_rows(w, torch.bfloat16, None, D, "w", dev)
    V = w.shape[0]
    _need(target, torch.int64, T, "target", dev)
    if target.dim() != 1 or target.shape[0] != T:
        raise ValueError(f"target: shape {tuple(target.shape)}, need ({T},)")
    on = _On(dev, stream)
    if loss is None:
        loss = on.empty(1, torch.float32)
    if row_loss is None:
        row_loss = on.empty(T, torch.float32)
    _need(loss, torch.float32, 1, "loss", dev)
    _need(row_loss, torch.float32, T, "row_loss", dev)
    if dx is None and want_dx:
        dx = on.empty((T, D), torch.bfloat16)
    if dw is None and want_dw:
        dw = on.empty((V, D), torch.bfloat16)
    lddx = D if dx is None else _need_rows(dx, torch.bfloat16, T, D, "dx", dev)
    lddw = D if dw is None else _need_rows(dw, torch.bfloat16, V, D, "dw", dev)
    # (a tensor of no rows has no address; the call takes NULL for "not wanted")
    args = (T, D, V, _ptr(x), ldx, _ptr(w), ldw, _ptr(target), int(ignore_index), int(mean),
            float(grad_scale), _ptr(loss), _ptr(row_loss), _ptr(dx), lddx, _ptr(dw), lddw)
    _sized(lib().zopt_linear_xent, args, "zopt_linear_xent", on, workspace)
    return loss, row_loss, dx, dw


def linear_xent_loss(x, w, target, ignore_index: int = -100, mean: bool = True,
                     loss: Optional[torch.Tensor] = None,
                     row_loss: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """Softmax cross entropy of the projection x w^T (zopt_linear_xent): x
    bf16 [T, D], w bf16 [V, D], target int64 [T].  Returns (loss, row_loss),
    fp32 [1] and [T]: the rows' losses, 0 where target is ignore_index, and
    their sum, or mean over the rows not ignored."""
    return _linear_xent(x, w, target, ignore_index, mean, 1.0, loss, row_loss, None, None, False,
                        False, workspace, stream)[:2]


def linear_xent_grad(x, w, target, ignore_index: int = -100, mean: bool = True,
                     grad_scale: float = 1.0, want_dx: bool = True, want_dw: bool = True,
                     loss: Optional[torch.Tensor] = None,
                     row_loss: Optional[torch.Tensor] = None,
                     dx: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """linear_xent_loss with the gradients of grad_scale * loss: returns
    (loss, row_loss, dx, dw), dx bf16 [T, D] and dw bf16 [V, D] (None where
    not wanted).  dw may be a [V, D] view of a flat gradient vector."""
    return _linear_xent(x, w, target, ignore_index, mean, grad_scale, loss, row_loss, dx, dw,
                        want_dx, want_dw, workspace, stream)


def _act8_empty(rows, cols, on) -> Act8:
    return Act8(on.empty((rows, cols), torch.float8_e4m3fn),
                on.empty((rows, (cols + 31) // 32), torch.uint8))


def act8_pack(x, out: Optional[Act8] = None, stream=None) -> Act8:
    """The 8-bit checkpoint of x, bf16 [rows, cols] (zopt_act8_pack)."""
    ldx = _need_rows(x, torch.bfloat16, None, None, "x")
    rows, cols = x.shape
    on = _On(x.device, stream)
    if out is None:
        out = _act8_empty(rows, cols, on)
    _need_act8(out, rows, cols, "out", x.device)
    _check(lib().zopt_act8_pack(rows, cols, _ptr(x), ldx, _ptr(out.q), _ptr(out.scale), on.handle),
           "zopt_act8_pack")
    return out


def act8_unpack(a: Act8, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The bf16 matrix that a checkpoint stands for (zopt_act8_unpack)."""
    _need_act8(a, None, None, "a")
    rows, cols = a.q.shape
    on = _On(a.q.device, stream)
    if out is None:
        out = on.empty((rows, cols), torch.bfloat16)
    ld = _need_rows(out, torch.bfloat16, rows, cols, "out", a.q.device)
    _check(lib().zopt_act8_unpack(rows, cols, _ptr(a.q), _ptr(a.scale), _ptr(out), ld, on.handle),
           "zopt_act8_unpack")
    return out


def act8_wgrad(dy, a: Act8, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dy^T x, bf16 [N, D], of dy bf16 [T, N] and the checkpoint a of x [T, D]:
    a linear layer's weight gradient (zopt_act8_wgrad)."""
    lddy = _need_rows(dy, torch.bfloat16, None, None, "dy")
    T, N = dy.shape
    _need_act8(a, T, None, "a", dy.device)
    D = a.q.shape[1]
    on = _On(dy.device, stream)
    if out is None:
        out = on.empty((N, D), torch.bfloat16)
    ld = _need_rows(out, torch.bfloat16, N, D, "out", dy.device)
    _sized(lib().zopt_act8_wgrad, (T, N, D, _ptr(dy), lddy, _ptr(a.q), _ptr(a.scale), _ptr(out), ld),
           "zopt_act8_wgrad", on, workspace)
    return out


def _glu_weights(w_gate, w_up, D, dev):
    ldw = _need_rows(w_gate, torch.bfloat16, None, D, "w_gate", dev)
    F = w_gate.shape[0]
    if _need_rows(w_up, torch.bfloat16, F, D, "w_up", dev) != ldw:
        raise ValueError("w_up: row stride differs from w_gate's")
    if F == 0:
        raise ValueError("w_gate: no rows")
    return F, ldw


def _act_id(act):
    if act not in ACTIVATIONS:
        raise ValueError(f"act: {act!r}, need one of {sorted(ACTIVATIONS)}")
    return ACTIVATIONS[act]


def glu_forward(x, w_gate, w_up, act: str = "silu", checkpoint=False,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                stream=None):
    """h = act(x w_gate^T) * (x w_up^T), bf16 [T, F] (zopt_glu_forward): x bf16
    [T, D], w_gate and w_up bf16 [F, D] with one row stride, act "silu" or
    "gelu" (the tanh form, torch's approximate="tanh").  With checkpoint=True, or a pair of Act8 to fill,
    returns (h, (g, u)) with the two products kept in 8 bits for
    glu_backward."""
    ldx = _need_rows(x, torch.bfloat16, None, None, "x")
    T, D = x.shape
    dev = x.device
    F, ldw = _glu_weights(w_gate, w_up, D, dev)
    on = _On(dev, stream)
    if out is None:
        out = on.empty((T, F), torch.bfloat16)
    ldh = _need_rows(out, torch.bfloat16, T, F, "out", dev)
    kept = None
    if checkpoint is True:
        kept = (_act8_empty(T, F, on), _act8_empty(T, F, on))
    elif checkpoint:
        kept = checkpoint
    if kept is not None:
        _need_act8(kept[0], T, F, "checkpoint[0]", dev)
        _need_act8(kept[1], T, F, "checkpoint[1]", dev)
    c = [None] * 4 if kept is None else [_ptr(t) for a in kept for t in a]
    _sized(lib().zopt_glu_forward, (T, D, F, _ptr(x), ldx, _ptr(w_gate), _ptr(w_up), ldw,
                                    _act_id(act), _ptr(out), ldh, *c),
           "zopt_glu_forward", on, workspace)
    return out if kept is None else (out, kept)


def glu_backward(dh, x, w_gate, w_up, act: str = "silu", checkpoint=None,
                 dx: Optional[torch.Tensor] = None, dw_gate: Optional[torch.Tensor] = None,
                 dw_up: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients (dx, dw_gate, dw_up) of glu_forward from dh, bf16 [T, F]
    (zopt_glu_backward).  x is the forward's input or its Act8; checkpoint the
    pair that glu_forward returned, or None to compute g and u again.  h, if
    given, receives act(g) u."""
    lddh = _need_rows(dh, torch.bfloat16, None, None, "dh")
    T, dev = dh.shape[0], dh.device
    if isinstance(x, Act8):
        _need_act8(x, T, None, "x", dev)
        D, xa = x.q.shape[1], (None, x.q.shape[1], _ptr(x.q), _ptr(x.scale))
    else:
        ldx = _need_rows(x, torch.bfloat16, T, None, "x", dev)
        D, xa = x.shape[1], (_ptr(x), ldx, None, None)
    F, ldw = _glu_weights(w_gate, w_up, D, dev)
    _need_rows(dh, torch.bfloat16, T, F, "dh", dev)
    c = [None] * 4
    if checkpoint is not None:
        _need_act8(checkpoint[0], T, F, "checkpoint[0]", dev)
        _need_act8(checkpoint[1], T, F, "checkpoint[1]", dev)
        c = [_ptr(t) for a in checkpoint for t in a]
    on = _On(dev, stream)
    if dx is None:
        dx = on.empty((T, D), torch.bfloat16)
    # (the weight gradients have one row stride; one that is not given takes the other's)
    lddw = D
    for t, name in ((dw_up, "dw_up"), (dw_gate, "dw_gate")):
        if t is not None:
            lddw = _need_rows(t, torch.bfloat16, F, D, name, dev)
    if dw_gate is None:
        dw_gate = on.empty((F, D), torch.bfloat16, lddw)
    if dw_up is None:
        dw_up = on.empty((F, D), torch.bfloat16, lddw)
    lddx = _need_rows(dx, torch.bfloat16, T, D, "dx", dev)
    if _need_rows(dw_up, torch.bfloat16, F, D, "dw_up", dev) != lddw:
        raise ValueError("dw_up: row stride differs from dw_gate's")
    ldh = F if h is None else _need_rows(h, torch.bfloat16, T, F, "h", dev)
    _sized(lib().zopt_glu_backward, (T, D, F, _ptr(dh), lddh, *xa, _ptr(w_gate), _ptr(w_up), ldw,
                                     _act_id(act), *c, _ptr(h), ldh, _ptr(dx), lddx, _ptr(dw_gate),
                                     _ptr(dw_up), lddw),
           "zopt_glu_backward", on, workspace)
    return dx, dw_gate, dw_up
