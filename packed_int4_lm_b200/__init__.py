"""ARCHead packed LM-head logits on NVIDIA B200 (sm_100a).

The GPU path is libarchead.so (include/archead.h); this module only marshals torch
tensors (device memory, streams) into its C ABI.  Every step of the logit and NLL path
runs in the library's CUDA kernels; there is no CPU fallback, and calling a GPU entry
point without the built library raises.

    head  = pack.build_head(W, H_cal, r_c, r_r, g, p, lam)     # offline, Algorithm 1
    dh    = DeviceHead.from_canonical(head, "cuda")             # upload + repack
    Y     = logits(H_bf16, dh)                                  # N x V float32
    nlls  = nll(H_bf16, dh, targets)                            # N float32, no logits

and, to train what feeds the (frozen) head:

    nlls, lse = nll_lse(H_bf16, dh, targets)                    # forward
    out = policy_loss(nlls, nlls_old, advantages)               # or preference_loss(...)
    dH  = nll_grad(H_bf16, dh, targets, nlls, lse, out["dnll"]) # N x D bf16: H.backward(dH)

All of them take a `stream` to run on instead of the current one.  The caller then orders the two: the
inputs (and an `out` that is given) have to be ready on that stream, e.g. by stream.wait_stream,
and the results are ready there.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import numpy as np
import torch

from . import _lib, pack
from ._lib import ArcheadError, ArcheadHead

__all__ = ["DeviceHead", "logits", "nll", "nll_lse", "nll_grad", "logits_grad", "policy_loss",
           "preference_loss", "agreement", "logits_host", "nll_host", "dequant", "check",
           "last_launches", "profile", "profile_read", "ArcheadError", "pack"]

_KEYS = ("r_nib", "r_code", "r_super", "Ac", "sAc", "Bc", "sBc", "Aw", "sAw", "Bw", "sBw")


def _stream_handle(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None or t.numel() == 0:
        return None
    return t.data_ptr()


FMT_SC4, FMT_ROW8 = 0, 1  # archead_format


class DeviceHead:
    """A head resident in device memory: the packed ARCHead head in the library's device
    layout, or (format "row8") the Row INT8 baseline head."""

    def __init__(self, meta: dict, tensors: dict):
        self.V, self.D = int(meta["V"]), int(meta["D"])
        self.r_c, self.r_r, self.g = int(meta["r_c"]), int(meta["r_r"]), int(meta["g"])
        self.format = FMT_ROW8 if meta.get("format") == "row8" else FMT_SC4
        self.tensors = tensors  # keeps the device buffers alive
        s = ArcheadHead()
        s.V, s.D, s.r_c, s.r_r, s.g = self.V, self.D, self.r_c, self.r_r, self.g
        s.format = self.format
        for k in _KEYS:
            setattr(s, k, _ptr(tensors.get(k)))
        s.row_scale = _ptr(tensors.get("row_scale"))
        self.struct = s

    @property
    def shape_args(self):
        return (self.V, self.D, self.r_c, self.r_r, self.g)

    def nbytes(self) -> int:
        return int(sum(t.numel() * t.element_size() for t in self.tensors.values()))

    @classmethod
    def from_canonical(cls, head: dict, device="cuda", stream=None) -> "DeviceHead":
        dev = torch.device(device)
        if head.get("format") == "row8":  # INT8 V x D row-major and FP32 row scales
            up = {"r_nib": torch.from_numpy(np.ascontiguousarray(head["q8"]).view(np.uint8)).to(dev),
                  "row_scale": torch.from_numpy(np.ascontiguousarray(head["row_scale"])).to(dev)}
            return cls(head, up)
        up = {}
        Vpad = (int(head["V"]) + 127) // 128 * 128
        for k in _KEYS:
            a = np.ascontiguousarray(head[k])
            if k == "r_code" and a.shape[0] != Vpad:
                # the device code array holds whole 128-row tiles (rows >= V are zero)
                a = np.concatenate([a, np.zeros((Vpad - a.shape[0], a.shape[1]), a.dtype)])
            if a.dtype == np.uint16:
                t = torch.from_numpy(a.view(np.int16))
            else:
                t = torch.from_numpy(a)
            up[k] = t.to(dev, non_blocking=False)
        canon = up["r_nib"]
        V, D = int(head["V"]), int(head["D"])
        # device layout: rows padded to a multiple of 128 (see archead_repack_residual)
        devnib = torch.empty((V + 127) // 128 * 128, D // 2, dtype=torch.uint8, device=dev)
        st = _stream_handle(stream)
        _lib.check(_lib.lib().archead_repack_residual(canon.data_ptr(), devnib.data_ptr(),
                                                      int(head["V"]), int(head["D"]), st),
                   "archead_repack_residual")
        torch.cuda.current_stream(dev).synchronize() if stream is None else stream.synchronize()
        up["r_nib"] = devnib
        return cls(head, up)


def _check_H(H: torch.Tensor, dh: DeviceHead):
    if H.dtype != torch.bfloat16 or H.dim() != 2 or H.shape[1] != dh.D:
        raise ValueError(f"H must be a bf16 N x {dh.D} tensor, got {H.dtype} {tuple(H.shape)}")
    if not H.is_cuda or not H.is_contiguous():
        raise ValueError("H must be a contiguous CUDA tensor")


def _optional(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _run(name: str, dev: torch.device, stream, tensors, *args):
    """One call into the library for tensors on dev: that device is made current around it (the
    library works on the current device), the stream is the given one or dev's current one, and
    on a stream other than the current one the tensors are recorded (their memory may not be
    handed out again before that stream is done with it).  A call through a head lists the head's."""
    # (torch.cuda.current_stream builds a Stream object first: 2 us, a fifth of a small call)
    current = torch._C._cuda_getCurrentRawStream(dev.index)
    handle = current if stream is None else stream.cuda_stream
    call = getattr(_lib.lib(), name)
    if torch._C._cuda_getDevice() == dev.index:
        status = call(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = call(*args, handle)
    if status:
        _lib.check(status, name)
    if handle != current:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _outputs(dev: torch.device, stream, make):
    """The tensors that make() allocates for the results of a call on `stream`.  Where that is not
    the current stream they are memory of its own pool: memory of the current stream's may still be
    in use by work queued there.  The current stream is recorded as a user of them."""
    if stream is None or stream.cuda_stream == torch._C._cuda_getCurrentRawStream(dev.index):
        return make()
    current = torch.cuda.current_stream(dev)
    with torch.cuda.stream(stream):
        out = make()
    for t in out:
        t.record_stream(current)
    return out


def logits(H: torch.Tensor, dh: DeviceHead, out: Optional[torch.Tensor] = None,
           stream=None) -> torch.Tensor:
    """Y = H W_d^T + (H B_w^T) A_w^T (N x V float32), asynchronous on the stream."""
    _check_H(H, dh)
    N, dev = H.shape[0], H.device
    if out is None:
        out, = _outputs(dev, stream, lambda: [torch.empty(N, dh.V, device=dev, dtype=torch.float32)])
    _run("archead_logits", dev, stream, (H, out, *dh.tensors.values()), H.data_ptr(),
         ctypes.byref(dh.struct), out.data_ptr() if N else None, N, *dh.shape_args)
    return out


def nll(H: torch.Tensor, dh: DeviceHead, targets: torch.Tensor,
        out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Per-token NLL (nats) = logsumexp(Y[n]) - Y[n, target[n]], without writing Y."""
    _check_H(H, dh)
    N = H.shape[0]
    if targets.dtype != torch.int32 or targets.shape != (N,) or not targets.is_cuda:
        raise ValueError("targets must be an int32 CUDA tensor of shape (N,)")
    if out is None:
        out, = _outputs(H.device, stream, lambda: [torch.empty(N, device=H.device, dtype=torch.float32)])
    targets, = _outputs(H.device, stream, lambda: [targets.contiguous()])
    _run("archead_nll", H.device, stream, (H, targets, out, *dh.tensors.values()), H.data_ptr(),
         ctypes.byref(dh.struct), targets.data_ptr(), out.data_ptr() if N else None, N,
         *dh.shape_args)
    return out


def nll_partials(H: torch.Tensor, dh: DeviceHead, targets: torch.Tensor, v_begin: int,
                 v_total: int, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """archead_nll_partials: this vocabulary shard's (max, sum exp, target logit) per token
    (N x 3 float32).  dh holds rows [v_begin, v_begin + dh.V) of a v_total-row head."""
    _check_H(H, dh)
    N = H.shape[0]
    if targets.dtype != torch.int32 or targets.shape != (N,) or not targets.is_cuda:
        raise ValueError("targets must be an int32 CUDA tensor of shape (N,)")
    if out is None:
        out, = _outputs(H.device, stream, lambda: [torch.empty(N, 3, device=H.device, dtype=torch.float32)])
    targets, = _outputs(H.device, stream, lambda: [targets.contiguous()])
    _run("archead_nll_partials", H.device, stream, (H, targets, out, *dh.tensors.values()),
         H.data_ptr(), ctypes.byref(dh.struct), targets.data_ptr(), int(v_begin), int(v_total),
         out.data_ptr() if N else None, N, *dh.shape_args)
    return out


def nll_merge(partials: torch.Tensor, out: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """archead_nll_merge: per-token NLL from G shards' partials (G x N x 3 float32 CUDA)."""
    if (partials.dtype != torch.float32 or partials.dim() != 3 or partials.shape[2] != 3
            or not partials.is_cuda):
        raise ValueError("partials must be a float32 CUDA tensor of shape (G, N, 3)")
    G, N = int(partials.shape[0]), int(partials.shape[1])
    dev = partials.device
    p, = _outputs(dev, stream, lambda: [partials.contiguous()])
    if out is None:
        out, = _outputs(dev, stream, lambda: [torch.empty(N, device=dev, dtype=torch.float32)])
    _run("archead_nll_merge", dev, stream, (p, out), p.data_ptr(), G, N, out.data_ptr() if N else None)
    return out


def vocab_parallel_nll(H: torch.Tensor, dh: DeviceHead, targets: torch.Tensor, v_begin: int,
                       v_total: int, group=None) -> torch.Tensor:
    """Per-token NLL of a head whose vocabulary rows are sharded over the ranks of `group`
    (rank k holds dh = rows [v_begin, v_begin + dh.V)): each rank reduces its shard to
    (max, sum exp, target logit) per token, one all-gather exchanges the N x 3 partials,
    and every rank merges them in rank order.  H and targets are the same on every rank."""
    import torch.distributed as dist
    part = nll_partials(H, dh, targets, v_begin, v_total)
    if not (dist.is_available() and dist.is_initialized()):  # one process holds the head
        return nll_merge(part[None])
    G = dist.get_world_size(group)
    if dist.get_backend(group) == "gloo":  # host collectives (tests without NCCL)
        host = part.cpu()
        gathered = [torch.empty_like(host) for _ in range(G)]
        dist.all_gather(gathered, host, group=group)
        return nll_merge(torch.stack(gathered).to(part.device))
    gathered = [torch.empty_like(part) for _ in range(G)]
    dist.all_gather(gathered, part, group=group)
    return nll_merge(torch.stack(gathered))


def agreement(H: torch.Tensor, dh: DeviceHead, Y_dense: torch.Tensor, k: int = 10,
              stream=None) -> dict:
    """archead_agreement: per token the ids of the k largest packed logits ("topk", N x k
    int32, decreasing, equal logits by smaller id), the dense argmax ("top1_dense", N),
    KL(P_dense || P_packed) in nats ("kl", N) and the packed log-sum-exp ("lse", N), all
    on the device.  Y_dense: N x V float32 reference logits on the same device."""
    _check_H(H, dh)
    N = H.shape[0]
    if (Y_dense.dtype != torch.float32 or tuple(Y_dense.shape) != (N, dh.V)
            or not Y_dense.is_cuda or not Y_dense.is_contiguous()):
        raise ValueError(f"Y_dense must be a contiguous float32 CUDA tensor of shape ({N}, {dh.V})")
    dev = H.device
    names = ("topk", "top1_dense", "kl", "lse")
    out = dict(zip(names, _outputs(dev, stream, lambda: [
        torch.empty(N, k, dtype=torch.int32, device=dev), torch.empty(N, dtype=torch.int32, device=dev),
        torch.empty(N, dtype=torch.float32, device=dev), torch.empty(N, dtype=torch.float32, device=dev)])))
    _run("archead_agreement", dev, stream, (H, Y_dense, *out.values(), *dh.tensors.values()),
         H.data_ptr(), ctypes.byref(dh.struct), Y_dense.data_ptr(), int(k),
         *[out[x].data_ptr() if N else None for x in names], N, *dh.shape_args)
    return out


def _float_arrays(N: int, dev, **arrays):
    """Checks that each given array is a contiguous float32 CUDA tensor of shape (N,) on dev."""
    for name, t in arrays.items():
        if t is not None and (t.dtype is not torch.float32 or t.shape != (N,) or t.device != dev
                              or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 tensor of shape ({N},) on {dev}")


def _int_array(name: str, t: torch.Tensor, shape, dev):
    if (t.dtype != torch.int32 or tuple(t.shape) != shape or t.device != dev
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {shape} on {dev}")


def _head_on(dh: DeviceHead, dev: torch.device):
    if dh.tensors["r_nib"].device != dev:
        raise ValueError(f"the head is on {dh.tensors['r_nib'].device}, the inputs are on {dev}")


def _grad_out(out: Optional[torch.Tensor], N: int, dh: DeviceHead, dev, stream) -> torch.Tensor:
    if out is None:
        return _outputs(dev, stream, lambda: [torch.empty((N, dh.D), device=dev, dtype=torch.bfloat16)])[0]
    if (out.dtype != torch.bfloat16 or tuple(out.shape) != (N, dh.D) or out.device != dev
            or not out.is_contiguous()):
        raise ValueError(f"out must be a contiguous bf16 tensor of shape ({N}, {dh.D}) on {dev}")
    return out


def nll_lse(H: torch.Tensor, dh: DeviceHead, targets: torch.Tensor, stream=None):
    """The per-token NLL, as nll gives it, and log-sum-exp of the logits (N float32 each):
    what nll_grad takes.  Every token needs a target in [0, V) here, also one that the loss masks
    (another id makes its NLL NaN and check() reports it)."""
    _check_H(H, dh)
    N, dev = H.shape[0], H.device
    _head_on(dh, dev)
    _int_array("targets", targets, (N,), dev)
    out, lse = _outputs(dev, stream, lambda: [torch.empty(N, device=dev, dtype=torch.float32) for _ in range(2)])
    _run("archead_nll_lse", dev, stream, (H, targets, out, lse, *dh.tensors.values()), H.data_ptr(),
         ctypes.byref(dh.struct), targets.data_ptr(), out.data_ptr(), lse.data_ptr(), N,
         *dh.shape_args)
    return out, lse


def nll_grad(H: torch.Tensor, dh: DeviceHead, targets: torch.Tensor, nll: torch.Tensor,
             lse: torch.Tensor, dnll: torch.Tensor, out: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
    """dH (N x D bf16): the gradient by the hidden states of a loss whose gradient by the
    per-token NLLs is dnll (N float32), through the packed head.  nll, lse: from nll_lse on the
    same H, head and targets.  Tokens with dnll = 0 are masked: their rows are zero, whatever
    their target."""
    _check_H(H, dh)
    N, dev = H.shape[0], H.device
    _head_on(dh, dev)
    _int_array("targets", targets, (N,), dev)
    _float_arrays(N, dev, nll=nll, lse=lse, dnll=dnll)
    out = _grad_out(out, N, dh, dev, stream)
    _run("archead_nll_grad", dev, stream, (H, targets, nll, lse, dnll, out, *dh.tensors.values()),
         H.data_ptr(), ctypes.byref(dh.struct), targets.data_ptr(), nll.data_ptr(), lse.data_ptr(),
         dnll.data_ptr(), out.data_ptr(), N, *dh.shape_args)
    return out


def logits_grad(dY: torch.Tensor, dh: DeviceHead, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """dH = dY W (N x D bf16): the gradient by the hidden states of a loss whose gradient by the
    logits is dY (N x V float32), through the packed head."""
    if (dY.dtype != torch.float32 or dY.dim() != 2 or dY.shape[1] != dh.V or not dY.is_cuda
            or not dY.is_contiguous()):
        raise ValueError(f"dY must be a contiguous float32 CUDA tensor of shape (N, {dh.V})")
    N, dev = dY.shape[0], dY.device
    _head_on(dh, dev)
    out = _grad_out(out, N, dh, dev, stream)
    _run("archead_logits_grad", dev, stream, (dY, out, *dh.tensors.values()), dY.data_ptr(),
         ctypes.byref(dh.struct), out.data_ptr(), N, *dh.shape_args)
    return out


REDUCTIONS = {"token": 0, "sequence": 1, "sum": 2}        # archead_reduction
PREFERENCES = {"sigmoid": 0, "hinge": 1, "ipo": 2}        # archead_preference


def _loss_inputs(nll: torch.Tensor, cu_seqlens: Optional[torch.Tensor]):
    if nll.dim() != 1 or not nll.is_cuda:
        raise ValueError("nll must be a float32 CUDA tensor of shape (N,)")
    N, dev = nll.shape[0], nll.device
    B = 0
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
            raise ValueError("cu_seqlens must hold B + 1 offsets")
        B = cu_seqlens.shape[0] - 1
        _int_array("cu_seqlens", cu_seqlens, (B + 1,), dev)
    return N, B, dev


def policy_loss(nll: torch.Tensor, nll_old: torch.Tensor, advantages: torch.Tensor, *,
                nll_ref: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None,
                cu_seqlens: Optional[torch.Tensor] = None, per_sequence: bool = False,
                clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0,
                reduction: str = "token", stream=None) -> dict:
    """archead_policy_loss: the clipped policy loss with a KL term on per-token NLLs (N float32
    each) and its gradient.  advantages: one per token, or with per_sequence one per sequence
    of cu_seqlens (B + 1 int32 offsets).  weights: 0 masks a token.  reduction: "token",
    "sequence" (needs cu_seqlens) or "sum".  Returns "stats" (4 float32: loss, surrogate, KL
    term, clipped share) and "dnll" (N float32, for nll_grad)."""
    if reduction not in REDUCTIONS:
        raise ValueError(f"reduction must be one of {sorted(REDUCTIONS)}, got {reduction!r}")
    N, B, dev = _loss_inputs(nll, cu_seqlens)
    if cu_seqlens is None and (per_sequence or reduction == "sequence"):
        raise ValueError("per_sequence advantages and the sequence reduction need cu_seqlens")
    _float_arrays(N, dev, nll=nll, nll_old=nll_old, nll_ref=nll_ref, weights=weights)
    _float_arrays(B if per_sequence else N, dev, advantages=advantages)
    dnll, stats = _outputs(dev, stream, lambda: [nll.new_empty(N), nll.new_empty(4)])
    _run("archead_policy_loss", dev, stream,
         (nll, nll_old, nll_ref, advantages, weights, cu_seqlens, dnll, stats),
         nll.data_ptr(), nll_old.data_ptr(), _optional(nll_ref), advantages.data_ptr(),
         _optional(weights), _optional(cu_seqlens), dnll.data_ptr(), stats.data_ptr(), N, B,
         per_sequence, clip_low, clip_high, kl_coef, REDUCTIONS[reduction])
    return {"stats": stats, "dnll": dnll}


def preference_loss(nll: torch.Tensor, cu_seqlens: torch.Tensor, pairs: torch.Tensor, *,
                    nll_ref: Optional[torch.Tensor] = None,
                    weights: Optional[torch.Tensor] = None, beta: float = 0.1,
                    kind: str = "sigmoid", label_smoothing: float = 0.0, margin: float = 0.0,
                    average: bool = False, stream=None) -> dict:
    """archead_preference_loss: the loss of preference pairs (P x 2 int32 sequence indices, the
    preferred one first) on per-token NLLs (N float32) of the sequences of cu_seqlens, and its
    gradient.  kind: "sigmoid", "hinge" or "ipo"; average: scores per weighted token.  Returns
    "loss" (1 float32, the mean), "pair_loss" (P), "rewards" (P x 2) and "dnll" (N, for
    nll_grad)."""
    if kind not in PREFERENCES:
        raise ValueError(f"kind must be one of {sorted(PREFERENCES)}, got {kind!r}")
    if cu_seqlens is None:
        raise ValueError("cu_seqlens must hold B + 1 offsets")
    N, B, dev = _loss_inputs(nll, cu_seqlens)
    _float_arrays(N, dev, nll=nll, nll_ref=nll_ref, weights=weights)
    if pairs.dim() != 2:
        raise ValueError("pairs must be an int32 tensor of shape (P, 2)")
    P = pairs.shape[0]
    _int_array("pairs", pairs, (P, 2), dev)
    dnll, loss, pair_loss, rewards = _outputs(
        dev, stream, lambda: [nll.new_empty(N), nll.new_empty(1), nll.new_empty(P), nll.new_empty(P, 2)])
    _run("archead_preference_loss", dev, stream,
         (nll, nll_ref, weights, cu_seqlens, pairs, dnll, loss, pair_loss, rewards),
         nll.data_ptr(), _optional(nll_ref), _optional(weights), cu_seqlens.data_ptr(),
         pairs.data_ptr(), dnll.data_ptr(), loss.data_ptr(), pair_loss.data_ptr(),
         rewards.data_ptr(), N, B, P, PREFERENCES[kind], average, beta, label_smoothing, margin)
    return {"loss": loss, "pair_loss": pair_loss, "rewards": rewards, "dnll": dnll}


def logits_host(H: torch.Tensor, dh: DeviceHead, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """archead_logits_host: host H in, host Y out (copies inside the call, synchronous)."""
    if H.dtype != torch.bfloat16 or H.is_cuda or not H.is_contiguous():
        raise ValueError("H must be a contiguous host bf16 tensor")
    N = H.shape[0]
    if out is None:
        out = torch.empty(N, dh.V, dtype=torch.float32, pin_memory=True)
    _lib.check(_lib.lib().archead_logits_host(H.data_ptr(), ctypes.byref(dh.struct),
                                              out.data_ptr(), N, *dh.shape_args,
                                              _stream_handle(stream)), "archead_logits_host")
    return out


def nll_host(H: torch.Tensor, dh: DeviceHead, targets: torch.Tensor,
             out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    if H.dtype != torch.bfloat16 or H.is_cuda or not H.is_contiguous():
        raise ValueError("H must be a contiguous host bf16 tensor")
    N = H.shape[0]
    if out is None:
        out = torch.empty(N, dtype=torch.float32, pin_memory=True)
    _lib.check(_lib.lib().archead_nll_host(H.data_ptr(), ctypes.byref(dh.struct),
                                           targets.contiguous().data_ptr(), out.data_ptr(),
                                           N, *dh.shape_args, _stream_handle(stream)),
               "archead_nll_host")
    return out


def dequant(dh: DeviceHead, row0: int = 0, nrows: Optional[int] = None, stream=None) -> dict:
    """FP32 dequantised components via the archead_dequant hook (for bit-exact checks)."""
    nrows = dh.V - row0 if nrows is None else nrows
    dev = dh.tensors["r_nib"].device
    shapes = {"R": (nrows, dh.D), "Ac": (nrows, dh.r_c), "Aw": (nrows, dh.r_r), "Bc": (dh.r_c, dh.D),
              "Bw": (dh.r_r, dh.D)}
    out = dict(zip(shapes, _outputs(dev, stream, lambda: [torch.empty(s, device=dev) for s in shapes.values()])))
    _run("archead_dequant", dev, stream, (*out.values(), *dh.tensors.values()), ctypes.byref(dh.struct),
         row0, nrows, *[_ptr(x) for x in out.values()])
    return out


def check(stream=None) -> None:
    """Synchronise the stream and raise if a kernel flagged an error (archead_check)."""
    _lib.check(_lib.lib().archead_check(_stream_handle(stream)), "archead_check")


def last_launches() -> int:
    """Kernels launched by the most recent archead_logits / archead_nll on this thread."""
    return int(_lib.lib().archead_last_launches())


def profile(enable: bool) -> None:
    """Start (clearing the record) or stop recording events around the main kernel."""
    _lib.check(_lib.lib().archead_profile(1 if enable else 0), "archead_profile")


def profile_read():
    """(total milliseconds, launches) of the main kernel since profile(True)."""
    ms = ctypes.c_double(0)
    n = ctypes.c_int(0)
    _lib.check(_lib.lib().archead_profile_read(ctypes.byref(ms), ctypes.byref(n)),
               "archead_profile_read")
    return float(ms.value), int(n.value)
