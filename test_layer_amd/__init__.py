"""VGG-T^3 test-time-training layer on MI355X (gfx950).

Thin binding over the C ABI in include/vggt3.h (libvggt3.so, built from
test_layer_amd/csrc). Every function marshals torch tensors (device memory and
the current stream) into the C calls; all layer arithmetic runs in the HIP
kernels. There is no CPU or PyTorch fallback: without the built library, or
without a GPU, calls raise.

    Vp    = shortconv(V, w, n_views, grid_h, grid_w, n_special)
    theta = ttt_write(K, Vp, theta, lr, steps, n_heads)        # in place
    O     = ttt_read(Q, theta, n_heads)
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Union

import torch

from . import _lib

BF16 = 0
F32 = 1
MX4 = 2

OK, EINVAL, EUNSUPPORTED, EWORKSPACE, EHIP = 0, -1, -2, -3, -4


class Vggt3Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        lib = _lib.load()
        detail = lib.vggt3_last_error().decode()
        super().__init__(f"{fn}: {lib.vggt3_status_str(status).decode()} ({status}): {detail}")
        self.status = status


def lib():
    return _lib.load()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype}; token tensors are bfloat16 or float32")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check_dev(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must live on the GPU (HIP device memory)")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _check_tokens(name: str, t: torch.Tensor) -> None:
    if t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D [tokens, channels] tensor, got shape {tuple(t.shape)}")
    _dtype_code(t)


def _check_same(name: str, t: Optional[torch.Tensor], ref: torch.Tensor, ref_name: str) -> None:
    if t is None:
        return
    if t.shape != ref.shape or t.dtype != ref.dtype:
        raise ValueError(f"{name} {tuple(t.shape)} {t.dtype} does not match {ref_name} {tuple(ref.shape)} {ref.dtype}")


def _check_f32(name: str, t: Optional[torch.Tensor], numel: int, at_least: bool = False) -> None:
    if t is None:
        return
    if t.dtype != torch.float32:
        raise ValueError(f"{name} must be float32, got {t.dtype}")
    if (t.numel() < numel) if at_least else (t.numel() != numel):
        raise ValueError(f"{name} has {t.numel()} elements, {'at least ' if at_least else ''}{numel} expected")


def _check_theta(theta: torch.Tensor, n_heads: int, d: int, m: int) -> None:
    _check_f32("theta", theta, n_heads * 3 * d * m)


def _call(name: str, *args) -> int:
    rc = getattr(lib(), name)(*args)
    if rc != OK:
        raise Vggt3Error(name, rc)
    return rc


def shortconv(V: torch.Tensor, w: torch.Tensor, n_views: int, grid_h: int, grid_w: int, n_special: int,
              out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """V' = depthwise k x k ShortConv2D of each view's patch grid (k = w.shape[-1],
    3 or 5); special tokens copied."""
    _check_tokens("V", V)
    if w.dtype != torch.float32 or w.dim() != 3 or w.shape[1] != w.shape[2]:
        raise TypeError("conv weights are float32 [C, k, k]")
    if w.shape[0] != V.shape[1]:
        raise ValueError(f"conv weights have {w.shape[0]} channels, V has {V.shape[1]}")
    if V.shape[0] != n_views * (n_special + grid_h * grid_w):
        raise ValueError(f"V has {V.shape[0]} tokens, {n_views} views x ({n_special} + {grid_h}x{grid_w}) expected")
    _check_same("out", out, V, "V")
    if out is None:
        out = torch.empty_like(V)
    _check_dev(V, w, out)
    k = int(w.shape[-1])
    if k == 3:
        _call("vggt3_shortconv", _ptr(V), _ptr(out), _ptr(w), n_views, grid_h, grid_w, n_special, V.shape[1],
              _dtype_code(V), _stream())
    else:
        _call("vggt3_shortconv_ex", _ptr(V), _ptr(out), _ptr(w), n_views, grid_h, grid_w, n_special, V.shape[1], k,
              _dtype_code(V), _stream())
    return out


def workspace_bytes(n_tokens: int, n_heads: int, d_head: int, d_hidden: int, dtype_code: int) -> int:
    return int(lib().vggt3_ttt_workspace_bytes(n_tokens, n_heads, d_head, d_hidden, dtype_code))


def make_workspace(n_tokens: int, n_heads: int, d_head: int, d_hidden: int, dtype_code: int,
                   device="cuda") -> Optional[torch.Tensor]:
    nb = workspace_bytes(n_tokens, n_heads, d_head, d_hidden, dtype_code)
    if nb == 0:
        return None
    return torch.empty(nb, dtype=torch.uint8, device=device)


def _mlp_dims(theta: torch.Tensor, X: torch.Tensor, n_heads: int, d_hidden: Optional[int]):
    C = X.shape[1]
    if C % n_heads:
        raise ValueError("channels not divisible by n_heads")
    d = C // n_heads
    per = theta.shape[-1] if theta.dim() == 2 else theta.numel() // n_heads
    m = d_hidden if d_hidden is not None else per // (3 * d)
    return d, m


LOSS_MSE, LOSS_DOT = 0, 1
OPT_GD, OPT_MUON = 0, 1
_LOSSES = {"mse": LOSS_MSE, "dot": LOSS_DOT}
_OPTS = {"gd": OPT_GD, "muon": OPT_MUON}


def _loss_code(loss) -> int:
    return _LOSSES[loss] if isinstance(loss, str) else int(loss)


def _opt_code(opt) -> int:
    return _OPTS[opt] if isinstance(opt, str) else int(opt)


def ttt_write(K: torch.Tensor, Vp: torch.Tensor, theta: torch.Tensor, lr: float, steps: int, n_heads: int,
              d_hidden: Optional[int] = None, workspace: Optional[torch.Tensor] = None,
              loss_out: Optional[torch.Tensor] = None, loss="mse", optimizer="gd", ns_steps: int = 5) -> torch.Tensor:
    """`steps` write steps of the inner loss; theta (fp32) is updated in place.

    loss: "mse" (default) or "dot"; optimizer: "gd" (default) or "muon" with
    `ns_steps` Newton-Schulz iterations.
    """
    _check_tokens("K", K)
    _check_same("Vp", Vp, K, "K")
    d, m = _mlp_dims(theta, K, n_heads, d_hidden)
    _check_theta(theta, n_heads, d, m)
    _check_f32("loss_out", loss_out, max(int(steps), 0) * n_heads, at_least=True)
    _check_dev(K, Vp, theta, workspace, loss_out)
    dt = _dtype_code(K)
    if workspace is None:
        workspace = make_workspace(K.shape[0], n_heads, d, m, dt, K.device)
    nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    lc, oc = _loss_code(loss), _opt_code(optimizer)
    if lc == LOSS_MSE and oc == OPT_GD:
        _call("vggt3_ttt_write", _ptr(K), _ptr(Vp), _ptr(theta), K.shape[0], n_heads, d, m, float(lr), int(steps),
              dt, _ptr(workspace), nb, _ptr(loss_out), _stream())
    else:
        _call("vggt3_ttt_write_ex", _ptr(K), _ptr(Vp), _ptr(theta), K.shape[0], n_heads, d, m, float(lr),
              int(steps), lc, oc, int(ns_steps), dt, _ptr(workspace), nb, _ptr(loss_out), _stream())
    return theta


NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024


def ttt_write_noalloc(K: torch.Tensor, Vp: torch.Tensor, theta: torch.Tensor, lr: float, steps: int, n_heads: int,
                      d_hidden: Optional[int] = None, loss_out: Optional[torch.Tensor] = None, loss="mse",
                      optimizer="gd", ns_steps: int = 5) -> torch.Tensor:
    """ttt_write through vggt3_ttt_write_noalloc: no workspace, nothing allocated
    (the library's fixed per-GPU scratch array serves as the workspace)."""
    _check_tokens("K", K)
    _check_same("Vp", Vp, K, "K")
    d, m = _mlp_dims(theta, K, n_heads, d_hidden)
    _check_theta(theta, n_heads, d, m)
    _check_f32("loss_out", loss_out, max(int(steps), 0) * n_heads, at_least=True)
    _check_dev(K, Vp, theta, loss_out)
    _call("vggt3_ttt_write_noalloc", _ptr(K), _ptr(Vp), _ptr(theta), K.shape[0], n_heads, d, m, float(lr),
          int(steps), _loss_code(loss), _opt_code(optimizer), int(ns_steps), _dtype_code(K), _ptr(loss_out),
          _stream())
    return theta


def ttt_write_conv(K: torch.Tensor, V: torch.Tensor, conv_w: torch.Tensor, n_views: int, grid_h: int, grid_w: int,
                   n_special: int, theta: torch.Tensor, lr: float, steps: int, n_heads: int,
                   Vp_out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   loss_out: Optional[torch.Tensor] = None, loss="mse", optimizer="gd",
                   ns_steps: int = 5) -> torch.Tensor:
    """ShortConv2D + write with the 3x3 conv formed inside each gradient pass
    (vggt3_ttt_write_conv): V' never has to exist in device memory. With
    Vp_out, the first step also writes V' there and later steps read it.
    bf16, (d_head, d_hidden) = (64, 128); theta is updated in place."""
    _check_tokens("K", K)
    _check_same("V", V, K, "K")
    if conv_w.dtype != torch.float32 or tuple(conv_w.shape) != (K.shape[1], 3, 3):
        raise ValueError(f"conv_w must be float32 [{K.shape[1]}, 3, 3]")
    if K.shape[0] != n_views * (n_special + grid_h * grid_w):
        raise ValueError(f"K has {K.shape[0]} tokens, {n_views} views x ({n_special} + {grid_h}x{grid_w}) expected")
    _check_same("Vp_out", Vp_out, K, "K")
    d, m = _mlp_dims(theta, K, n_heads, None)
    _check_theta(theta, n_heads, d, m)
    _check_f32("loss_out", loss_out, max(int(steps), 0) * n_heads, at_least=True)
    _check_dev(K, V, conv_w, theta, Vp_out, workspace, loss_out)
    dt = _dtype_code(K)
    if workspace is None:
        workspace = make_workspace(K.shape[0], n_heads, d, m, dt, K.device)
    nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _call("vggt3_ttt_write_conv", _ptr(K), _ptr(V), _ptr(conv_w), n_views, grid_h, grid_w, n_special, _ptr(theta),
          n_heads, d, m, float(lr), int(steps), _loss_code(loss), _opt_code(optimizer), int(ns_steps),
          _ptr(Vp_out), _ptr(workspace), nb, _ptr(loss_out), _stream())
    return theta


def ttt_grad(K: torch.Tensor, Vp: torch.Tensor, theta: torch.Tensor, n_heads: int,
             grad: Optional[torch.Tensor] = None, accumulate: bool = False, d_hidden: Optional[int] = None,
             workspace: Optional[torch.Tensor] = None, loss_out: Optional[torch.Tensor] = None,
             loss="mse") -> torch.Tensor:
    """Gradient of the inner loss at theta (Eq. 5 split: accumulate=True adds to grad)."""
    _check_tokens("K", K)
    _check_same("Vp", Vp, K, "K")
    d, m = _mlp_dims(theta, K, n_heads, d_hidden)
    _check_theta(theta, n_heads, d, m)
    _check_f32("grad", grad, n_heads * 3 * d * m)
    _check_f32("loss_out", loss_out, n_heads, at_least=True)
    if grad is None:
        grad = torch.empty_like(theta)
    _check_dev(K, Vp, theta, grad, workspace, loss_out)
    dt = _dtype_code(K)
    if workspace is None:
        workspace = make_workspace(K.shape[0], n_heads, d, m, dt, K.device)
    nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    lc = _loss_code(loss)
    if lc == LOSS_MSE:
        _call("vggt3_ttt_grad", _ptr(K), _ptr(Vp), _ptr(theta), _ptr(grad), int(bool(accumulate)), K.shape[0],
              n_heads, d, m, dt, _ptr(workspace), nb, _ptr(loss_out), _stream())
    else:
        _call("vggt3_ttt_grad_ex", _ptr(K), _ptr(Vp), _ptr(theta), _ptr(grad), int(bool(accumulate)), K.shape[0],
              n_heads, d, m, lc, dt, _ptr(workspace), nb, _ptr(loss_out), _stream())
    return grad


REDUCE_APPLY, REDUCE_STORE, REDUCE_ACCUMULATE = 0, 1, 2


def ttt_grad_partials(K: torch.Tensor, Vp: torch.Tensor, theta: torch.Tensor, n_heads: int,
                      workspace: torch.Tensor, d_hidden: Optional[int] = None, loss="mse",
                      want_loss: bool = True) -> None:
    """Per-(head, chunk) gradient and loss partials into `workspace` (Eq. 5 inner sums).
    With want_loss=False the loss partials are not computed (a later reduce's loss is NaN)."""
    _check_tokens("K", K)
    _check_same("Vp", Vp, K, "K")
    d, m = _mlp_dims(theta, K, n_heads, d_hidden)
    _check_theta(theta, n_heads, d, m)
    _check_dev(K, Vp, theta, workspace)
    lc = _loss_code(loss)
    if lc == LOSS_MSE and want_loss:
        _call("vggt3_ttt_grad_partials", _ptr(K), _ptr(Vp), _ptr(theta), K.shape[0], n_heads, d, m,
              _dtype_code(K), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream())
    else:
        _call("vggt3_ttt_grad_partials_ex", _ptr(K), _ptr(Vp), _ptr(theta), K.shape[0], n_heads, d, m, lc,
              int(bool(want_loss)), _dtype_code(K), _ptr(workspace), workspace.numel() * workspace.element_size(),
              _stream())


def muon_workspace_bytes(n_heads: int, d_head: int, d_hidden: int) -> int:
    return int(lib().vggt3_ttt_muon_workspace_bytes(n_heads, d_head, d_hidden))


def ttt_muon_apply(theta: torch.Tensor, grad: torch.Tensor, lr: float, n_heads: int, d_head: int,
                   d_hidden: int, ns_steps: int = 5, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """theta -= lr * NS(grad) per head and weight matrix (Muon update), in place
    (the full-width 1024 -> 4096 MLP takes a workspace)."""
    _check_theta(theta, n_heads, d_head, d_hidden)
    _check_f32("grad", grad, n_heads * 3 * d_head * d_hidden)
    _check_dev(theta, grad, workspace)
    need = muon_workspace_bytes(n_heads, d_head, d_hidden)
    if need == 0 and workspace is None:
        _call("vggt3_ttt_muon_apply", _ptr(theta), _ptr(grad), float(lr), n_heads, d_head, d_hidden, int(ns_steps),
              _stream())
        return theta
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=theta.device)
    _call("vggt3_ttt_muon_apply_ex", _ptr(theta), _ptr(grad), float(lr), n_heads, d_head, d_hidden, int(ns_steps),
          _ptr(workspace), workspace.numel() * workspace.element_size(), _stream())
    return theta


def ttt_reduce(workspace: torch.Tensor, n_tokens: int, n_heads: int, d_head: int, d_hidden: int, dtype_code: int,
               mode: int, dst: torch.Tensor, lr: float = 0.0, loss_out: Optional[torch.Tensor] = None) -> None:
    """Fixed-tree sum of the partials, then apply to theta / store / accumulate into dst."""
    _check_f32("dst", dst, n_heads * 3 * d_head * d_hidden)
    _check_f32("loss_out", loss_out, n_heads, at_least=True)
    _check_dev(workspace, dst, loss_out)
    _call("vggt3_ttt_reduce", _ptr(workspace), workspace.numel() * workspace.element_size(), n_tokens, n_heads,
          d_head, d_hidden, dtype_code, mode, _ptr(dst), float(lr), _ptr(loss_out), _stream())


def ttt_apply(theta: torch.Tensor, grad: torch.Tensor, lr: float, n_heads: int, d_head: int,
              d_hidden: int) -> torch.Tensor:
    _check_theta(theta, n_heads, d_head, d_hidden)
    _check_f32("grad", grad, n_heads * 3 * d_head * d_hidden)
    _check_dev(theta, grad)
    _call("vggt3_ttt_apply", _ptr(theta), _ptr(grad), float(lr), n_heads, d_head, d_hidden, _stream())
    return theta


def read_workspace_bytes(n_tokens: int, n_heads: int, d_head: int, d_hidden: int, dtype_code: int) -> int:
    return int(lib().vggt3_ttt_read_workspace_bytes(n_tokens, n_heads, d_head, d_hidden, dtype_code))


def ttt_read(Q: torch.Tensor, theta: torch.Tensor, n_heads: int, d_hidden: Optional[int] = None,
             out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """O = T_theta(Q) per head (the full-width 1024 -> 4096 MLP reads through a workspace)."""
    _check_tokens("Q", Q)
    _check_same("out", out, Q, "Q")
    d, m = _mlp_dims(theta, Q, n_heads, d_hidden)
    _check_theta(theta, n_heads, d, m)
    if out is None:
        out = torch.empty_like(Q)
    _check_dev(Q, theta, out, workspace)
    dt = _dtype_code(Q)
    need = read_workspace_bytes(Q.shape[0], n_heads, d, m, dt)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=Q.device)
    nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    # vggt3_ttt_read_ex serves every shape (the per-head ones ignore the workspace)
    _call("vggt3_ttt_read_ex", _ptr(Q), _ptr(theta), _ptr(out), Q.shape[0], n_heads, d, m, dt, _ptr(workspace), nb,
          _stream())
    return out


def ttt_layer(K, V, Q, theta, conv_w, n_views, grid_h, grid_w, n_special, n_heads, lr, steps,
              workspace=None, loss_out=None, Vp=None, O=None, loss="mse", optimizer="gd", ns_steps=5,
              conv_k=None):
    """The whole layer: V' = ShortConv2D(V); write theta (in place); O = read(Q).

    conv_w may be [C, 3, 3] (the pages' ShortConv2D) or [C, 5, 5] (their "V-5"
    variant); conv_k, if given, convolves the keys as well before the write
    (their "KV-3" variant, with its own filters)."""
    Vp = shortconv(V, conv_w, n_views, grid_h, grid_w, n_special, out=Vp)
    if conv_k is not None:
        K = shortconv(K, conv_k, n_views, grid_h, grid_w, n_special)
    ttt_write(K, Vp, theta, lr, steps, n_heads, workspace=workspace, loss_out=loss_out, loss=loss,
              optimizer=optimizer, ns_steps=ns_steps)
    return ttt_read(Q, theta, n_heads, out=O), Vp


# ---------------------------------------------------------------------------
# Streamed (offloaded) write and read over host-resident token tensors
# ---------------------------------------------------------------------------

_side_streams = {}


def _side_stream(device: torch.device, key: str) -> torch.cuda.Stream:
    """A per-device copy stream of default priority, created once."""
    idx = device.index if device.index is not None else torch.cuda.current_device()
    s = _side_streams.get((idx, key))
    if s is None:
        s = torch.cuda.Stream(device=idx)
        _side_streams[(idx, key)] = s
    return s


def _check_host(*ts):
    for t in ts:
        if t.is_cuda:
            raise ValueError("streamed token tensors live in host memory (pinned for overlap)")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def stage_bytes(chunk_tokens: int, n_heads: int, d_head: int, dtype_code: int) -> int:
    """Device staging a streamed call needs: two slots of two token chunks."""
    return int(lib().vggt3_ttt_stream_stage_bytes(chunk_tokens, n_heads, d_head, dtype_code))


def ttt_write_streamed(K_host: torch.Tensor, Vp_host: torch.Tensor, theta: torch.Tensor, lr: float, steps: int,
                       n_heads: int, chunk_tokens: int, d_hidden: Optional[int] = None,
                       stage: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                       loss_out: Optional[torch.Tensor] = None, loss="mse", optimizer="gd", ns_steps: int = 5,
                       copy_stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """ttt_write over host-resident K and V' streamed in chunks of `chunk_tokens`
    (Eq. 5 offload schedule); theta is a device tensor updated in place.

    The copies run on `copy_stream` (default: a side stream of this device)
    while the kernels run on the current stream; the host tensors must stay
    untouched until the current stream has been synchronised."""
    _check_tokens("K_host", K_host)
    _check_same("Vp_host", Vp_host, K_host, "K_host")
    d, m = _mlp_dims(theta, K_host, n_heads, d_hidden)
    _check_theta(theta, n_heads, d, m)
    _check_f32("loss_out", loss_out, max(int(steps), 0) * n_heads, at_least=True)
    _check_host(K_host, Vp_host)
    _check_dev(theta, stage, workspace, loss_out)
    dt = _dtype_code(K_host)
    n = K_host.shape[0]
    ct = max(1, min(int(chunk_tokens), n))
    if stage is None:
        stage = torch.empty(stage_bytes(ct, n_heads, d, dt), dtype=torch.uint8, device=theta.device)
    if workspace is None:
        workspace = make_workspace(ct, n_heads, d, m, dt, theta.device)
    if copy_stream is None:
        copy_stream = _side_stream(theta.device, "h2d")
    ws_nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _call("vggt3_ttt_write_streamed", _ptr(K_host), _ptr(Vp_host), _ptr(theta), n, n_heads, d, m, float(lr),
          int(steps), _loss_code(loss), _opt_code(optimizer), int(ns_steps), dt, int(chunk_tokens), _ptr(stage),
          stage.numel() * stage.element_size(), _ptr(workspace), ws_nb, _ptr(loss_out), _stream(),
          ctypes.c_void_p(copy_stream.cuda_stream))
    return theta


def ttt_read_streamed(Q_host: torch.Tensor, theta: torch.Tensor, n_heads: int, chunk_tokens: int,
                      d_hidden: Optional[int] = None, out: Optional[torch.Tensor] = None,
                      stage: Optional[torch.Tensor] = None, h2d_stream: Optional[torch.cuda.Stream] = None,
                      d2h_stream: Optional[torch.cuda.Stream] = None,
                      workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """O = T_theta(Q) for host-resident Q, written to a host tensor (query mode
    over a frozen theta), streamed in chunks of `chunk_tokens`. `out` defaults
    to a new pinned tensor; read it after synchronising the current stream."""
    _check_tokens("Q_host", Q_host)
    _check_same("out", out, Q_host, "Q_host")
    d, m = _mlp_dims(theta, Q_host, n_heads, d_hidden)
    _check_theta(theta, n_heads, d, m)
    if out is None:
        out = torch.empty(Q_host.shape, dtype=Q_host.dtype, pin_memory=True)
    _check_host(Q_host, out)
    _check_dev(theta, stage)
    dt = _dtype_code(Q_host)
    n = Q_host.shape[0]
    ct = max(1, min(int(chunk_tokens), n))
    if stage is None:
        stage = torch.empty(stage_bytes(ct, n_heads, d, dt), dtype=torch.uint8, device=theta.device)
    if h2d_stream is None:
        h2d_stream = _side_stream(theta.device, "h2d")
    if d2h_stream is None:
        d2h_stream = _side_stream(theta.device, "d2h")
    if workspace is None:
        need = read_workspace_bytes(ct, n_heads, d, m, dt)
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=theta.device)
    _check_dev(workspace)
    nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _call("vggt3_ttt_read_streamed_ex", _ptr(Q_host), _ptr(theta), _ptr(out), n, n_heads, d, m, dt,
          int(chunk_tokens), _ptr(stage), stage.numel() * stage.element_size(), _ptr(workspace), nb, _stream(),
          ctypes.c_void_p(h2d_stream.cuda_stream), ctypes.c_void_p(d2h_stream.cuda_stream))
    return out


# ---------------------------------------------------------------------------
# Microscaled 4-bit matrices: quantisation, products, and the read of fast
# weights frozen in 4 bits
# ---------------------------------------------------------------------------

def _pointers(*ts):
    """The GPU that a call's tensors (contiguous, None where absent) share, and their addresses."""
    dev, out = None, []
    for t in ts:
        if t is None:
            out.append(None)
            continue
        d = t.get_device()
        if d != dev:
            if d < 0:
                raise ValueError("tensors must live on the GPU (HIP device memory)")
            if dev is not None:
                raise ValueError(f"tensors live on different devices: cuda:{dev} and cuda:{d}")
            dev = d
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        out.append(t.data_ptr())
    return dev, out


# The current stream of a GPU as the address that the C calls take, without the
# Stream object round it (which costs as much host time as a launch), and the
# current GPU. Both are private to torch, so a build without them takes the
# public calls.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_gpu = getattr(torch._C, "_cuda_getDevice", None)
if _raw_stream is None or _current_gpu is None:
    def _raw_stream(dev: int) -> int:
        return torch.cuda.current_stream(dev).cuda_stream

    def _current_gpu() -> int:
        return torch.cuda.current_device()


def _run(name: str, dev: int, *args) -> None:
    """Call `name` on GPU `dev`'s current stream, whichever device is current."""
    fn = getattr(_lib.load(), name)
    if dev == _current_gpu():
        rc = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev))
    if rc != OK:
        raise Vggt3Error(name, rc)


class Mx4(NamedTuple):
    """A 4-bit matrix [rows, k] (include/vggt3.h, "Microscaled 4-bit matrices"):
    codes uint8 [rows, kp / 2] and scales uint8 [ceil(rows / 64), kp / 128, 64, 4],
    kp = k rounded up to 128."""

    codes: torch.Tensor
    scales: torch.Tensor
    k: int

    @property
    def rows(self) -> int:
        return self.codes.shape[0]


class FrozenMx4(NamedTuple):
    """The full-width fast weights in 4 bits: gate and up [4096, 1024], down [1024, 4096]."""

    gate: Mx4
    up: Mx4
    down: Mx4


def _check_width(name: str, k: int) -> None:
    if k > 0x7FFFFFFF:  # ctypes would pass on its low 32 bits
        raise ValueError(f"{name} has {k} columns, which do not fit 32 bits")


def _mx4_shapes(rows: int, k: int):
    nb = (k + 127) // 128
    return (rows, nb * 64), ((rows + 63) // 64, nb, 64, 4)


def _mx4_empty(rows: int, k: int, device) -> Mx4:
    cs, ss = _mx4_shapes(rows, k)
    return Mx4(torch.empty(cs, dtype=torch.uint8, device=device), torch.empty(ss, dtype=torch.uint8, device=device), k)


def _check_mx4(name: str, a: Mx4, rows: Optional[int] = None, k: Optional[int] = None) -> None:
    if not isinstance(a, Mx4):
        raise TypeError(f"{name} must be an Mx4 (codes, scales, k), got {type(a).__name__}")
    codes, scales, ak = a
    if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise TypeError(f"{name}: codes and scales must be uint8, got {codes.dtype} and {scales.dtype}")
    if codes.dim() != 2 or ak < 1:
        raise ValueError(f"{name}: codes are [rows, kp / 2] and k >= 1, got {tuple(codes.shape)} and k = {ak}")
    _check_width(name, ak)
    n = codes.shape[0]
    if (rows is not None and n != rows) or (k is not None and ak != k):
        raise ValueError(f"{name} is [{n}, {ak}], [{n if rows is None else rows}, {ak if k is None else k}] expected")
    cs, ss = _mx4_shapes(n, ak)
    if codes.shape != cs or scales.shape != ss:
        raise ValueError(f"{name} [{n}, {ak}] has codes {tuple(codes.shape)} and scales {tuple(scales.shape)}, "
                         f"{cs} and {ss} expected")


def _type_code(dtype: torch.dtype) -> int:
    if dtype == torch.bfloat16:
        return BF16
    if dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {dtype}; bfloat16 or float32")


def _check_out(out: Optional[torch.Tensor], shape, dtype: torch.dtype) -> None:
    if out is not None and (tuple(out.shape) != tuple(shape) or out.dtype != dtype):
        raise ValueError(f"out {tuple(out.shape)} {out.dtype}, {tuple(shape)} {dtype} expected")


def _ws(workspace: Optional[torch.Tensor], need: int, device):
    """(workspace, its bytes), allocated where none was given and one is needed."""
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return workspace, 0 if workspace is None else workspace.numel() * workspace.element_size()


def mx4_quantize(X: torch.Tensor, transpose: bool = False, out: Optional[Mx4] = None) -> Mx4:
    """X [rows, k] (or, with transpose, X [k, rows]) in 4 bits, blocks of 32 along k."""
    _check_tokens("X", X)
    k, rows = X.shape if transpose else (X.shape[1], X.shape[0])
    if k < 1:
        raise ValueError("X has no columns to contract over")
    _check_width("X", k)
    if out is not None:
        _check_mx4("out", out, rows, k)
    else:
        out = _mx4_empty(rows, k, X.device)
    dev, (x, c, s) = _pointers(X, out.codes, out.scales)
    _run("vggt3_mx4_quantize", dev, x, int(bool(transpose)), c, s, rows, k, _dtype_code(X))
    return out


def mx4_dequantize(A: Mx4, dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values [rows, k] that A stands for."""
    _check_mx4("A", A)
    dt = _type_code(dtype)
    _check_out(out, (A.rows, A.k), dtype)
    if out is None:
        out = torch.empty((A.rows, A.k), dtype=dtype, device=A.codes.device)
    dev, (c, s, o) = _pointers(A.codes, A.scales, out)
    _run("vggt3_mx4_dequantize", dev, c, s, o, A.rows, A.k, dt)
    return out


def mx4_matmul_workspace_bytes(m: int, n: int, k: int, a_type: int) -> int:
    return int(lib().vggt3_mx4_matmul_workspace_bytes(m, n, k, a_type))


def mx4_matmul(A: Union[Mx4, torch.Tensor], W: Mx4, dtype: torch.dtype = torch.bfloat16,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A W^T [m, n] with W [n, k] in 4 bits; tokens A [m, k] are quantised on the way."""
    _check_mx4("W", W)
    if isinstance(A, Mx4):
        _check_mx4("A", A, k=W.k)
        m, a_type, data, scales = A.rows, MX4, A.codes, A.scales
    else:
        _check_tokens("A", A)
        if A.shape[1] != W.k:
            raise ValueError(f"A has {A.shape[1]} columns, W is [{W.rows}, {W.k}]")
        m, a_type, data, scales = A.shape[0], _dtype_code(A), A, None
    dt = _type_code(dtype)
    _check_out(out, (m, W.rows), dtype)
    if out is None:
        out = torch.empty((m, W.rows), dtype=dtype, device=data.device)
    workspace, nb = _ws(workspace, mx4_matmul_workspace_bytes(m, W.rows, W.k, a_type), data.device)
    dev, (a, a_s, w, w_s, o, ws) = _pointers(data, scales, W.codes, W.scales, out, workspace)
    _run("vggt3_mx4_matmul", dev, a, a_s, a_type, w, w_s, o, m, W.rows, W.k, dt, ws, nb)
    return out


def ttt_freeze_mx4(theta: torch.Tensor, d_head: int = 1024, d_hidden: int = 4096,
                   out: Optional[FrozenMx4] = None) -> FrozenMx4:
    """Freeze the full-width theta* in 4 bits for ttt_read_mx4 (6.7 MB for its 50 MB)."""
    _check_theta(theta, 1, d_head, d_hidden)
    shapes = ((d_hidden, d_head), (d_hidden, d_head), (d_head, d_hidden))
    if out is None:
        out = FrozenMx4(*(_mx4_empty(r, k, theta.device) for r, k in shapes))
    parts = []
    for name, a, (r, k) in zip(FrozenMx4._fields, out, shapes):
        _check_mx4(name, a, r, k)
        parts += [a.codes, a.scales]
    dev, ptrs = _pointers(theta, *parts)
    _run("vggt3_ttt_freeze_mx4", dev, *ptrs, 1, d_head, d_hidden)
    return out


def read_mx4_workspace_bytes(n_tokens: int, d_head: int, d_hidden: int, q_type: int) -> int:
    return int(lib().vggt3_ttt_read_mx4_workspace_bytes(n_tokens, 1, d_head, d_hidden, q_type))


def ttt_read_mx4(Q: Union[Mx4, torch.Tensor], frozen: FrozenMx4, out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """O = T_theta*(Q) with the full-width fast weights frozen in 4 bits (query mode).
    Q: bf16 tokens [n, 1024], quantised on the way, or an Mx4; O is bf16."""
    if not isinstance(frozen, FrozenMx4):
        raise TypeError(f"frozen must be a FrozenMx4 (ttt_freeze_mx4), got {type(frozen).__name__}")
    d, m = frozen.down.rows, frozen.gate.rows
    if isinstance(Q, Mx4):
        _check_mx4("Q", Q, k=d)
        n, q_type, data, scales = Q.rows, MX4, Q.codes, Q.scales
    else:
        _check_tokens("Q", Q)
        if Q.shape[1] != d:
            raise ValueError(f"Q has {Q.shape[1]} channels, the frozen weights {d}")
        n, q_type, data, scales = Q.shape[0], _dtype_code(Q), Q, None
    parts = []
    for name, a, (r, k) in zip(FrozenMx4._fields, frozen, ((m, d), (m, d), (d, m))):
        _check_mx4(name, a, r, k)
        parts += [a.codes, a.scales]
    _check_out(out, (n, d), torch.bfloat16)
    if out is None:
        out = torch.empty((n, d), dtype=torch.bfloat16, device=data.device)
    workspace, nb = _ws(workspace, read_mx4_workspace_bytes(n, d, m, q_type), data.device)
    dev, (q, q_s, *weights, o, ws) = _pointers(data, scales, *parts, out, workspace)
    _run("vggt3_ttt_read_mx4", dev, q, q_s, q_type, *weights, o, n, 1, d, m, ws, nb)
    return out


# ---------------------------------------------------------------------------
# Block join: norm after a block, gate, residual scale, residual, norm before
# the next block; and its gradient
# ---------------------------------------------------------------------------

NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2
_NORMS = {None: NORM_NONE, "none": NORM_NONE, "rms": NORM_RMS, "layer": NORM_LAYER}


def _norm_code(kind) -> int:
    if kind is not None and not isinstance(kind, str):
        return int(kind)
    if kind not in _NORMS:
        raise KeyError(f"unknown norm {kind!r}; None, 'none', 'rms' or 'layer'")
    return _NORMS[kind]


def _check_gate(gate: Optional[torch.Tensor], gate_tokens: int, x: torch.Tensor) -> int:
    """Tokens that share a gate row, at most all of them (so that the count fits the C call's 64 bits)."""
    if gate is None:
        return 1
    per = int(gate_tokens)
    if per < 1:
        raise ValueError(f"gate_tokens = {gate_tokens} < 1")
    n = x.shape[0]
    want = (-(-n // per), x.shape[1])
    if tuple(gate.shape) != want or gate.dtype != x.dtype:
        raise ValueError(f"gate {tuple(gate.shape)} {gate.dtype}, {want} {x.dtype} expected")
    return min(per, max(n, 1))


def _check_channels(C: int, **params) -> None:
    for name, p in params.items():
        if p is not None and (p.dtype != torch.float32 or p.numel() != C):
            _check_f32(name, p, C)


def block_join(x: torch.Tensor, f: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
               gate_tokens: int = 1, scale: Optional[torch.Tensor] = None, post=None,
               post_w: Optional[torch.Tensor] = None, post_b: Optional[torch.Tensor] = None, pre=None,
               pre_w: Optional[torch.Tensor] = None, pre_b: Optional[torch.Tensor] = None, eps: float = 1e-6,
               mx4: bool = False, r: Optional[torch.Tensor] = None, y: Union[torch.Tensor, Mx4, None] = None):
    """(r, y): r = x + scale * gate * post(f), y = pre(r).

    post, pre: None, "rms" or "layer". Without f, y = pre(x) and r is None;
    without pre, y is None. Row t // gate_tokens of gate serves token t. With
    mx4, y comes in 4 bits (the operand of mx4_matmul and ttt_read_mx4). r and y
    may be given as outputs; r may be x (in place)."""
    _check_tokens("x", x)
    _check_same("f", f, x, "x")
    per = _check_gate(gate, gate_tokens, x)
    n, C = x.shape
    _check_width("x", C)
    _check_channels(C, scale=scale, post_w=post_w, post_b=post_b, pre_w=pre_w, pre_b=pre_b)
    post, pre = _norm_code(post), _norm_code(pre)
    if f is not None:
        _check_same("r", r, x, "x")
        if r is None:
            r = torch.empty_like(x)
    elif r is not None:
        raise ValueError("r goes with a block output f")
    codes = scales = None
    if pre == NORM_NONE:
        if y is not None or mx4:
            raise ValueError("y goes with a norm before the next block")
    elif mx4:
        if y is None:
            y = _mx4_empty(n, C, x.device)
        _check_mx4("y", y, n, C)
        codes, scales = y.codes, y.scales
    else:
        if y is None:
            y = torch.empty_like(x)
        elif isinstance(y, Mx4):
            raise TypeError("y is an Mx4, which goes with mx4=True")
        _check_same("y", y, x, "x")
    plain = None if mx4 else y
    dev, (px, pf, pg, ps, *norms, pr, py, pc, psc) = _pointers(x, f, gate, scale, post_w, post_b, pre_w, pre_b, r,
                                                               plain, codes, scales)
    _run("vggt3_block_join", dev, px, pf, pg, per, ps, post, norms[0], norms[1], pre, norms[2], norms[3],
         float(eps), pr, py, pc, psc, n, C, _dtype_code(x))
    return r, y


class BlockJoinGrads(NamedTuple):
    """Gradients of block_join's inputs; None for those that are absent or not wanted."""

    dx: Optional[torch.Tensor] = None
    df: Optional[torch.Tensor] = None
    dgate: Optional[torch.Tensor] = None
    dscale: Optional[torch.Tensor] = None
    dpost_w: Optional[torch.Tensor] = None
    dpost_b: Optional[torch.Tensor] = None
    dpre_w: Optional[torch.Tensor] = None
    dpre_b: Optional[torch.Tensor] = None


def block_join_grad_workspace_bytes(n_tokens: int, channels: int, dtype_code: int) -> int:
    return int(lib().vggt3_block_join_grad_workspace_bytes(n_tokens, channels, dtype_code))


def block_join_grad(r: torch.Tensor, f: Optional[torch.Tensor] = None, dr: Optional[torch.Tensor] = None,
                    dy: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, gate_tokens: int = 1,
                    scale: Optional[torch.Tensor] = None, post=None, post_w: Optional[torch.Tensor] = None,
                    post_b: Optional[torch.Tensor] = None, pre=None, pre_w: Optional[torch.Tensor] = None,
                    pre_bias: bool = False, eps: float = 1e-6, out: Optional[BlockJoinGrads] = None,
                    workspace: Optional[torch.Tensor] = None) -> BlockJoinGrads:
    """Gradient of block_join at its stored r (without f: its x) and f, from the
    gradients dr of r and dy of y.

    Gradients of what was given are returned (pre_bias: there was a pre_b, whose
    value does not enter). With `out`, exactly its tensors are written; out.dx
    may be dr."""
    _check_tokens("r", r)
    for name, t in (("f", f), ("dr", dr), ("dy", dy)):
        _check_same(name, t, r, "r")
    per = _check_gate(gate, gate_tokens, r)
    n, C = r.shape
    _check_width("r", C)
    _check_channels(C, scale=scale, post_w=post_w, post_b=post_b, pre_w=pre_w)
    post, pre = _norm_code(post), _norm_code(pre)
    if out is None:
        # the channel vectors are rows of one allocation, 16-byte aligned
        wanted = [scale is not None, post_w is not None, post_b is not None, pre_w is not None, bool(pre_bias)]
        rows = iter(torch.empty((sum(wanted), (C + 3) // 4 * 4), dtype=torch.float32, device=r.device).unbind(0))
        vecs = [(next(rows) if C % 4 == 0 else next(rows)[:C]) if w else None for w in wanted]
        out = BlockJoinGrads(torch.empty_like(r), None if f is None else torch.empty_like(f),
                             None if gate is None else torch.empty_like(gate), *vecs)
    else:
        _check_same("dx", out.dx, r, "r")
        _check_same("df", out.df, r, "r")
        if out.dgate is not None and gate is None:
            raise ValueError("dgate without a gate")
        _check_same("dgate", out.dgate, gate, "gate")
        for name in BlockJoinGrads._fields[3:]:
            _check_f32(name, getattr(out, name), C)
    workspace, nb = _ws(workspace, block_join_grad_workspace_bytes(n, C, _dtype_code(r)), r.device)
    dev, (pr, pf, pg, ps, pw, pb, w, ws, *grads) = _pointers(r, f, gate, scale, post_w, post_b, pre_w, workspace, dr, dy,
                                                             *out)
    _run("vggt3_block_join_grad", dev, pr, pf, pg, per, ps, post, pw, pb, pre, w, float(eps), *grads, n, C,
         _dtype_code(r), ws, nb)
    return out
