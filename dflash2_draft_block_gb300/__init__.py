"""DFlash2 draft-block head on one GB300: Python binding of libdflash2.

Argument marshalling only: every step runs in the library's CUDA kernels.
Tensors are torch CUDA tensors (bf16 weights/activations as torch.bfloat16),
contiguous and row-major; calls are asynchronous on the current torch stream.
Autograd records none of them: outputs do not require gradients, whatever the inputs
do, and gradients come from the *_grad calls.

    ids, vals, G = unary_topk(h, W_lm, K, W_H)          # logits never leave the chip
    path, scores = selector_walk(anchors, ids, vals, G, A, Bc, block_size)
    s = selector_pair_scores(pred, ids, vals, G, A, Bc)  # teacher-forced
    loss, label = selector_ce(s, ids, targets, V)      # the selector's K-way CE
    y, dyn = conv_prepare(x, block_size, taps, group, W_proj, base)
    y2 = conv_finish(z, block_size, taps, group, dyn, base)
    loss, lse, dh, dW = unary_loss_grad(h, W_lm, targets)  # full-vocabulary CE, gradients
    y = dropout(x, rate, seed, step)                    # dropout_grad: the same mask
"""
from __future__ import annotations

import ctypes as ct
import functools
import operator

import torch

from . import _abi

DF2_DTYPE_BF16 = 0
DF2_DTYPE_F32 = 1
DF2_ERR_UNSUPPORTED = 2
DF2_STATUS_ID_OUT_OF_RANGE = 0x1
DF2_STATUS_WAIT_TIMEOUT = 0x2
DF2_HEAD_PATH_STREAM = 0
DF2_HEAD_PATH_GEMM = 1
DF2_HEAD_PATH_CUDA_CORE = 2


class DFlash2Error(RuntimeError):
    def __init__(self, call: str, code: int):
        self.code = code
        super().__init__(f"{call}: {status_string(code)}")


def lib():
    return _abi._lib or _abi.load()


def kernels_launched() -> int:
    """Kernels this library has launched in this process so far."""
    return int(lib().dflash2_kernels_launched())


def unary_topk_path(P, D, V, K) -> int:
    """DF2_HEAD_PATH_* of the head kernels for these shapes (-1: shapes rejected)."""
    return int(lib().dflash2_unary_topk_path(P, D, V, K))


def status_string(code: int) -> str:
    return lib().dflash2_status_string(int(code)).decode()


def _p(t):
    return ct.c_void_p(t.data_ptr() if t is not None else 0)


def _on_device(t):
    return t.is_cuda


def _stream(stream, device):
    """The CUDA stream handle of `stream` (default: the current one), which must
    belong to the device of the call's tensors."""
    if stream is None and _raw_stream is not None and device.index is not None:
        return ct.c_void_p(_raw_stream(device.index))  # the handle alone, in a tenth of the time
    s = stream if stream is not None else torch.cuda.current_stream()
    if s.device != device:
        raise ValueError(f"the stream is on {s.device}, the call's tensors on {device}")
    return ct.c_void_p(s.cuda_stream)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _capturing(stream, device):
    """Whether what is launched on `stream` (default: the current one) goes into a graph."""
    if device.type != "cuda":
        return False
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _need(t, name, dtype, ndim=None):
    if not isinstance(t, torch.Tensor) or not _on_device(t):
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")


def _device(first, **others):
    """The device of the call: `first`'s, which every other given tensor shares and
    which is the current CUDA device (the library launches on the current device)."""
    dev = first.device
    for name, t in others.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the call's tensors on {dev}")
    if dev.type == "cuda" and dev.index is not None and dev.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {dev} but the current CUDA device is "
                         f"cuda:{torch.cuda.current_device()} (torch.cuda.set_device first)")
    return dev


def _out(t, name, dtype, numel, dev):
    """A caller-given output: a contiguous tensor of the call's device, dtype and
    element count (the kernels write numel elements through its pointer)."""
    _need(t, name, dtype)
    if t.numel() != numel:
        raise ValueError(f"{name} must hold {numel} elements, got shape {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the call's tensors on {dev}")
    return t


def _status(st, dev):
    """dev_status: None, or one int32 word (at least) on the call's device."""
    if st is not None:
        _need(st, "dev_status", torch.int32)
        if st.numel() < 1 or st.device != dev:
            raise ValueError("dev_status must hold an int32 word on the call's device")
    return st


def _check(call, rc):
    if rc != 0:
        raise DFlash2Error(call, rc)


def _empty(shape, dtype, dev, stream):
    """Memory for a call to write, of its stream's own: what the current stream's allocations
    left free may have work queued there, which another stream does not wait for."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _made(shape, dtype, dev, stream):
    """An output that the call makes: kept from other uses until the work of the current stream,
    where the caller goes on with it, is done, too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    t = _empty(shape, dtype, dev, stream)
    t.record_stream(torch.cuda.current_stream(dev))
    return t


def _workspace(nbytes, workspace, device, stream=None):
    if nbytes == 0 and workspace is None:
        return None
    if workspace is None:
        return _empty(nbytes, torch.uint8, device, stream)
    _need(workspace, "workspace", workspace.dtype)
    if workspace.device != device:
        raise ValueError(f"workspace is on {workspace.device}, the call's tensors on {device}")
    if _nbytes(workspace) < nbytes:
        raise ValueError(f"workspace too small: need {nbytes} bytes")
    return workspace


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def unary_topk_workspace_size(P, D, V, K, r=0) -> int:
    return int(lib().dflash2_unary_topk_workspace_size(P, D, V, K, r))


def unary_topk(h, W_lm, K, W_H=None, *, output_multiplier=1.0, final_logit_softcapping=0.0,
               workspace=None, dev_status=None, out=None, stream=None):
    """Top-K unary logits per row of h, and G = h W_H^T.  Returns (ids, vals, G).

    output_multiplier m and final_logit_softcapping c map each logit u to
    c*tanh(m*u/c) (m*u when c = 0) before the selection; the defaults leave it."""
    _need(h, "h", torch.bfloat16, 2)
    _need(W_lm, "W_lm", torch.bfloat16, 2)
    P, D = h.shape
    V = W_lm.shape[0]
    if W_lm.shape[1] != D:
        raise ValueError("W_lm must be [V, D]")
    r = 0
    if W_H is not None:
        _need(W_H, "W_H", torch.bfloat16, 2)
        r = W_H.shape[0]
        if W_H.shape[1] != D:
            raise ValueError("W_H must be [r, D]")
    dev = _device(h, W_lm=W_lm, W_H=W_H)
    if out is None:
        ids = _made((P, K), torch.int32, dev, stream)
        vals = _made((P, K), torch.float32, dev, stream)
        G = _made((P, r), torch.float32, dev, stream) if r else None
    else:
        ids, vals, G = out
        _out(ids, "ids", torch.int32, P * K, dev)
        _out(vals, "vals", torch.float32, P * K, dev)
        if r:
            _out(G, "G", torch.float32, P * r, dev)
    _status(dev_status, dev)
    ws = _workspace(unary_topk_workspace_size(P, D, V, K, r), workspace, dev, stream)
    rc = lib().dflash2_unary_topk(_p(h), P, D, _p(W_lm), V, int(K), float(output_multiplier),
                                  float(final_logit_softcapping), _p(W_H), r, _p(G), _p(ids),
                                  _p(vals), _p(ws), _nbytes(ws),
                                  _p(dev_status), _stream(stream, dev))
    _check("dflash2_unary_topk", rc)
    return ids, vals, G


def unary_topk_noalloc(h, W_lm, K, W_H=None, *, output_multiplier=1.0, final_logit_softcapping=0.0,
                       dev_status=None, out=None, stream=None):
    """unary_topk without a workspace: for callers that may not allocate device
    memory during a call.  Scratch comes from a fixed array inside the library
    (DF2_NOALLOC_SCRATCH_BYTES per GPU), shared by every call, so calls must not
    overlap on the GPU.  Outputs are allocated here unless `out` is given."""
    _need(h, "h", torch.bfloat16, 2)
    _need(W_lm, "W_lm", torch.bfloat16, 2)
    P, D = h.shape
    if W_lm.shape[1] != D:
        raise ValueError("W_lm must be [V, D]")
    r = 0
    if W_H is not None:
        _need(W_H, "W_H", torch.bfloat16, 2)
        r = W_H.shape[0]
        if W_H.shape[1] != D:
            raise ValueError("W_H must be [r, D]")
    dev = _device(h, W_lm=W_lm, W_H=W_H)
    if out is None:
        ids = _made((P, K), torch.int32, dev, stream)
        vals = _made((P, K), torch.float32, dev, stream)
        G = _made((P, r), torch.float32, dev, stream) if r else None
    else:
        ids, vals, G = out
        _out(ids, "ids", torch.int32, P * K, dev)
        _out(vals, "vals", torch.float32, P * K, dev)
        if r:
            _out(G, "G", torch.float32, P * r, dev)
    _status(dev_status, dev)
    rc = lib().dflash2_unary_topk_noalloc(_p(h), P, D, _p(W_lm), W_lm.shape[0], int(K),
                                          float(output_multiplier), float(final_logit_softcapping), _p(W_H), r,
                                          _p(G), _p(ids), _p(vals), _p(dev_status), _stream(stream, dev))
    _check("dflash2_unary_topk_noalloc", rc)
    return ids, vals, G


def selector_walk(anchors, topk_ids, topk_vals, G, A, Bc, block_size, *, dev_status=None,
                  out=None, stream=None):
    """Greedy walk per request.  Returns (path [R, B-1] int32, path_scores [R, B-1] f32)."""
    _need(anchors, "anchors", torch.int32, 1)
    _need(topk_ids, "topk_ids", torch.int32)
    _need(topk_vals, "topk_vals", torch.float32)
    _need(G, "G", torch.float32)
    _need(A, "A", torch.bfloat16, 2)
    _need(Bc, "Bc", torch.bfloat16, 2)
    R = anchors.shape[0]
    B = int(block_size)
    K = topk_ids.shape[-1]
    V, r = A.shape
    if topk_ids.numel() != R * B * K or topk_vals.numel() != R * B * K or G.numel() != R * B * r:
        raise ValueError("candidate / gate shapes do not match [R*B, K] / [R*B, r]")
    if tuple(Bc.shape) != (V, r):
        raise ValueError("Bc must be [V, r] like A")
    dev = _device(anchors, topk_ids=topk_ids, topk_vals=topk_vals, G=G, A=A, Bc=Bc)
    T = max(B - 1, 0)
    if out is None:
        path = _made((R, T), torch.int32, dev, stream)
        scores = _made((R, T), torch.float32, dev, stream)
    else:
        path, scores = out
        _out(path, "path", torch.int32, R * T, dev)
        _out(scores, "path_scores", torch.float32, R * T, dev)
    _status(dev_status, dev)
    rc = lib().dflash2_selector_walk(_p(anchors), R, B, _p(topk_ids), _p(topk_vals), _p(G), _p(A),
                                     _p(Bc), V, K, r, _p(path), _p(scores), _p(dev_status),
                                     _stream(stream, dev))
    _check("dflash2_selector_walk", rc)
    return path, scores


def selector_ce(scores, topk_ids, targets, V, *, dev_status=None, out=None, stream=None):
    """The selector's K-way cross-entropy per row of teacher-forced scores [P, K]:
    (loss [P] fp32, label [P] int32); rows whose target is not a candidate give
    label -1 and NaN loss."""
    _need(scores, "scores", torch.float32)
    _need(topk_ids, "topk_ids", torch.int32)
    _need(targets, "targets", torch.int32, 1)
    P = targets.shape[0]
    K = topk_ids.shape[-1]
    if topk_ids.numel() != P * K or scores.numel() != P * K:
        raise ValueError("scores / topk_ids do not match [P, K]")
    dev = _device(scores, topk_ids=topk_ids, targets=targets)
    if out is None:
        out = (_made((P,), torch.float32, dev, stream), _made((P,), torch.int32, dev, stream))
    loss, label = out
    _out(loss, "loss", torch.float32, P, dev)
    _out(label, "label", torch.int32, P, dev)
    _status(dev_status, dev)
    rc = lib().dflash2_selector_ce(_p(scores), _p(topk_ids), _p(targets), P, K, int(V), _p(loss), _p(label),
                                   _p(dev_status), _stream(stream, dev))
    _check("dflash2_selector_ce", rc)
    return loss, label


def selector_pair_scores(pred, topk_ids, topk_vals, G, A, Bc, *, dev_status=None, out=None,
                         stream=None):
    """Teacher-forced scores [P, K]."""
    _need(pred, "pred", torch.int32, 1)
    _need(topk_ids, "topk_ids", torch.int32)
    _need(topk_vals, "topk_vals", torch.float32)
    _need(G, "G", torch.float32)
    _need(A, "A", torch.bfloat16, 2)
    _need(Bc, "Bc", torch.bfloat16, 2)
    P = pred.shape[0]
    K = topk_ids.shape[-1]
    V, r = A.shape
    if topk_ids.numel() != P * K or topk_vals.numel() != P * K or G.numel() != P * r:
        raise ValueError("candidate / gate shapes do not match [P, K] / [P, r]")
    if tuple(Bc.shape) != (V, r):
        raise ValueError("Bc must be [V, r] like A")
    dev = _device(pred, topk_ids=topk_ids, topk_vals=topk_vals, G=G, A=A, Bc=Bc)
    if out is None:
        scores = _made((P, K), torch.float32, dev, stream)
    else:
        scores = _out(out, "scores", torch.float32, P * K, dev)
    _status(dev_status, dev)
    rc = lib().dflash2_selector_pair_scores(_p(pred), P, _p(topk_ids), _p(topk_vals), _p(G), _p(A),
                                            _p(Bc), V, K, r, _p(scores), _p(dev_status),
                                            _stream(stream, dev))
    _check("dflash2_selector_pair_scores", rc)
    return scores


def draft_head_workspace_size(R, B, D, V, K, r) -> int:
    return int(lib().dflash2_draft_head_workspace_size(R, B, D, V, K, r))


def draft_head(h, W_lm, K, W_H, A, Bc, anchors, block_size, pred=None, *, output_multiplier=1.0,
               final_logit_softcapping=0.0, workspace=None, dev_status=None, out=None, stream=None):
    """Unary top-K, G = H(h), the greedy walk and (pred given) the teacher-forced
    scores of one draft block in one call.  Returns (ids, vals, G, path, path_scores,
    pair_scores or None)."""
    _need(h, "h", torch.bfloat16, 2)
    _need(W_lm, "W_lm", torch.bfloat16, 2)
    _need(W_H, "W_H", torch.bfloat16, 2)
    _need(A, "A", torch.bfloat16, 2)
    _need(Bc, "Bc", torch.bfloat16, 2)
    _need(anchors, "anchors", torch.int32, 1)
    P, D = h.shape
    V = W_lm.shape[0]
    r = W_H.shape[0]
    R = anchors.shape[0]
    B = int(block_size)
    if P != R * B or W_lm.shape[1] != D or W_H.shape[1] != D:
        raise ValueError("h must be [R*B, D] with W_lm [V, D], W_H [r, D]")
    if tuple(A.shape) != (V, r) or tuple(Bc.shape) != (V, r):
        raise ValueError("A and Bc must be [V, r]")
    if pred is not None:
        _need(pred, "pred", torch.int32, 1)
        if pred.shape[0] != P:
            raise ValueError("pred must be [R*B]")
    dev = _device(h, W_lm=W_lm, W_H=W_H, A=A, Bc=Bc, anchors=anchors, pred=pred)
    T = max(B - 1, 0)
    if out is None:
        def e(shape, dtype):
            return _made(shape, dtype, dev, stream)
        out = (e((P, K), torch.int32), e((P, K), torch.float32), e((P, r), torch.float32), e((R, T), torch.int32),
               e((R, T), torch.float32), e((P, K), torch.float32) if pred is not None else None)
    ids, vals, G, path, ps, pair = out
    _out(ids, "ids", torch.int32, P * K, dev)
    _out(vals, "vals", torch.float32, P * K, dev)
    _out(G, "G", torch.float32, P * r, dev)
    _out(path, "path", torch.int32, R * T, dev)
    _out(ps, "path_scores", torch.float32, R * T, dev)
    if pred is not None:
        _out(pair, "pair_scores", torch.float32, P * K, dev)
    _status(dev_status, dev)
    workspace = _workspace(draft_head_workspace_size(R, B, D, V, K, r), workspace, dev, stream)
    if workspace is None:  # nothing to hold (R = 0): the call still takes a buffer
        workspace = _empty(1, torch.uint8, dev, stream)
    rc = lib().dflash2_draft_head(_p(h), R, B, D, _p(W_lm), V, K, float(output_multiplier),
                                  float(final_logit_softcapping), _p(W_H), r, _p(A), _p(Bc), _p(anchors),
                                  _p(pred), _p(ids), _p(vals), _p(G), _p(path), _p(ps), _p(pair),
                                  _p(workspace), _nbytes(workspace), _p(dev_status), _stream(stream, dev))
    _check("dflash2_draft_head", rc)
    return ids, vals, G, path, ps, pair


def selector_lattice(anchors, topk_ids, topk_vals, G, A, Bc, block_size, *, dev_status=None,
                     out=None, stream=None):
    """Every adjacent candidate pair scored at once: lattice [R, B-1, K, K] f32."""
    _need(anchors, "anchors", torch.int32, 1)
    _need(topk_ids, "topk_ids", torch.int32)
    _need(topk_vals, "topk_vals", torch.float32)
    _need(G, "G", torch.float32)
    _need(A, "A", torch.bfloat16, 2)
    _need(Bc, "Bc", torch.bfloat16, 2)
    R = anchors.shape[0]
    B = int(block_size)
    K = topk_ids.shape[-1]
    V, r = A.shape
    if topk_ids.numel() != R * B * K or topk_vals.numel() != R * B * K or G.numel() != R * B * r:
        raise ValueError("candidate / gate shapes do not match [R*B, K] / [R*B, r]")
    if tuple(Bc.shape) != (V, r):
        raise ValueError("Bc must be [V, r] like A")
    dev = _device(anchors, topk_ids=topk_ids, topk_vals=topk_vals, G=G, A=A, Bc=Bc)
    T = max(B - 1, 0)
    lat = out if out is not None else _made((R, T, K, K), torch.float32, dev, stream)
    _out(lat, "lattice", torch.float32, R * T * K * K, dev)
    _status(dev_status, dev)
    rc = lib().dflash2_selector_lattice(_p(anchors), R, B, _p(topk_ids), _p(topk_vals), _p(G), _p(A),
                                        _p(Bc), V, K, r, _p(lat), _p(dev_status), _stream(stream, dev))
    _check("dflash2_selector_lattice", rc)
    return lat


def lattice_walk(lattice, topk_ids, block_size, vocab_size, *, uniforms=None, temperature=1.0,
                 dev_status=None, out=None, stream=None):
    """Greedy (uniforms None) or sampling walk over a lattice.  Returns (path [R, B-1]
    int32, path_scores [R, B-1] f32)."""
    _need(lattice, "lattice", torch.float32, 4)
    _need(topk_ids, "topk_ids", torch.int32)
    R, T, K, K2 = lattice.shape
    B = int(block_size)
    if K2 != K or T != B - 1 or topk_ids.numel() != R * B * K:
        raise ValueError("lattice must be [R, B-1, K, K] over topk_ids [R*B, K]")
    if uniforms is not None:
        _need(uniforms, "uniforms", torch.float32)
        if uniforms.numel() != R * T:
            raise ValueError("uniforms must be [R, B-1]")
    dev = _device(lattice, topk_ids=topk_ids, uniforms=uniforms)
    if out is None:
        path = _made((R, T), torch.int32, dev, stream)
        scores = _made((R, T), torch.float32, dev, stream)
    else:
        path, scores = out
        _out(path, "path", torch.int32, R * T, dev)
        _out(scores, "path_scores", torch.float32, R * T, dev)
    _status(dev_status, dev)
    rc = lib().dflash2_lattice_walk(_p(lattice), _p(topk_ids), R, B, K, int(vocab_size), _p(uniforms),
                                    float(temperature), _p(path), _p(scores), _p(dev_status),
                                    _stream(stream, dev))
    _check("dflash2_lattice_walk", rc)
    return path, scores


def _act_dtype(x):
    if x.dtype == torch.bfloat16:
        return DF2_DTYPE_BF16
    if x.dtype == torch.float32:
        return DF2_DTYPE_F32
    raise TypeError("conv activations must be bfloat16 or float32")


def _conv_shapes(C, taps, group, **named):
    """The conv's weight and correction shapes (skipped when taps or group are
    themselves invalid: the library rejects those with a status)."""
    if not (taps >= 1 and group >= 1 and C % group == 0):
        return
    G = C // group
    want = {"W_proj": (2 * taps * G, C), "base": (2, taps, C), "base_next": (2, taps, C)}
    for name, (t, P) in named.items():
        shape = (P, taps, G) if name == "dyn_out" else want[name]
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def conv_prepare_workspace_size(P, C, taps, group, dtype=DF2_DTYPE_BF16) -> int:
    return int(lib().dflash2_conv_prepare_workspace_size(P, C, taps, group, dtype))


def conv_prepare(x, block_size, taps, group, W_proj, base, *, workspace=None, out=None, stream=None):
    """Conv before a sublayer.  Returns (y like x, dyn_out [P, taps, C/group] f32)."""
    dt = _act_dtype(x)
    _need(x, "x", x.dtype, 2)
    _need(W_proj, "W_proj", torch.bfloat16, 2)
    _need(base, "base", torch.float32, 3)
    P, C = x.shape
    taps, group = int(taps), int(group)
    _conv_shapes(C, taps, group, W_proj=(W_proj, P), base=(base, P))
    G = C // group if group >= 1 else 0
    dev = _device(x, W_proj=W_proj, base=base)
    if out is None:
        y = _made(x.shape, x.dtype, dev, stream)
        dyn = _made((P, taps, G), torch.float32, dev, stream)
    else:
        y, dyn = out
        _out(y, "y", x.dtype, P * C, dev)
        _out(dyn, "dyn_out", torch.float32, P * max(taps, 0) * G, dev)
    ws = _workspace(conv_prepare_workspace_size(P, C, taps, group, dt), workspace, dev, stream)
    rc = lib().dflash2_conv_prepare(_p(x), dt, P, C, int(block_size), taps, group,
                                    _p(W_proj), _p(base), _p(y), _p(dyn), _p(ws),
                                    _nbytes(ws), _stream(stream, dev))
    _check("dflash2_conv_prepare", rc)
    return y, dyn


def conv_finish(z, block_size, taps, group, dyn_out, base, *, out=None, stream=None):
    """Conv after the sublayer with prepare's dynamic kernel.  Returns y like z."""
    dt = _act_dtype(z)
    _need(z, "z", z.dtype, 2)
    _need(dyn_out, "dyn_out", torch.float32, 3)
    _need(base, "base", torch.float32, 3)
    P, C = z.shape
    taps, group = int(taps), int(group)
    _conv_shapes(C, taps, group, dyn_out=(dyn_out, P), base=(base, P))
    dev = _device(z, dyn_out=dyn_out, base=base)
    y = _out(out, "y", z.dtype, P * C, dev) if out is not None else _made(z.shape, z.dtype, dev, stream)
    rc = lib().dflash2_conv_finish(_p(z), dt, P, C, int(block_size), taps, group,
                                   _p(dyn_out), _p(base), _p(y), _stream(stream, dev))
    _check("dflash2_conv_finish", rc)
    return y


def conv_finish_prepare(z, block_size, taps, group, dyn_out, base, W_proj, base_next, residual=None, *,
                        workspace=None, out=None, stream=None):
    """A sublayer's conv finish, plus the residual stream when given, then the next
    sublayer's conv prepare.  Returns (h like z, y_next like z, dyn_out_next
    [P, taps, C/group] f32)."""
    dt = _act_dtype(z)
    _need(z, "z", z.dtype, 2)
    _need(dyn_out, "dyn_out", torch.float32, 3)
    _need(base, "base", torch.float32, 3)
    _need(W_proj, "W_proj", torch.bfloat16, 2)
    _need(base_next, "base_next", torch.float32, 3)
    if residual is not None:
        _need(residual, "residual", z.dtype, 2)
        if residual.shape != z.shape:
            raise ValueError("residual must have z's shape")
    P, C = z.shape
    taps, group = int(taps), int(group)
    _conv_shapes(C, taps, group, dyn_out=(dyn_out, P), base=(base, P), W_proj=(W_proj, P),
                 base_next=(base_next, P))
    G = C // group if group >= 1 else 0
    dev = _device(z, dyn_out=dyn_out, base=base, W_proj=W_proj, base_next=base_next, residual=residual)
    if out is None:
        h, y = _made(z.shape, z.dtype, dev, stream), _made(z.shape, z.dtype, dev, stream)
        dyn = _made((P, taps, G), torch.float32, dev, stream)
    else:
        h, y, dyn = out
        _out(h, "h", z.dtype, P * C, dev)
        _out(y, "y_next", z.dtype, P * C, dev)
        _out(dyn, "dyn_out_next", torch.float32, P * max(taps, 0) * G, dev)
    ws = _workspace(int(lib().dflash2_conv_finish_prepare_workspace_size(P, C, taps, group, dt)), workspace, dev, stream)
    rc = lib().dflash2_conv_finish_prepare(_p(z), dt, P, C, int(block_size), taps, group, _p(dyn_out),
                                           _p(base), _p(residual), _p(h), _p(W_proj), _p(base_next), _p(y),
                                           _p(dyn), _p(ws), _nbytes(ws), _stream(stream, dev))
    _check("dflash2_conv_finish_prepare", rc)
    return h, y, dyn


_DTYPES = {torch.bfloat16: DF2_DTYPE_BF16, torch.float32: DF2_DTYPE_F32}


def _rows(t, name, shape=None, dev=None):
    """A bf16 or fp32 matrix whose rows are dense (their distance may exceed their length):
    (its DF2_DTYPE_*, the distance in elements)."""
    if not isinstance(t, torch.Tensor) or not _on_device(t):
        raise TypeError(f"{name} must be a CUDA tensor")
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be {'a matrix' if shape is None else list(shape)}, got {list(t.shape)}")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the call's tensors on {dev}")
    rows, cols = t.shape
    if t.is_contiguous():
        return dt, max(cols, 1)
    ld = t.stride(0) if rows > 1 else max(cols, 1)
    if (cols > 1 and t.stride(1) != 1) or ld < cols:
        raise ValueError(f"{name} must have dense rows")
    return dt, ld


def _scratch(nbytes, workspace, dev, stream):
    """The caller's workspace, or one of this call's own, free for the next call of the
    stream: (tensor, address, bytes)."""
    if workspace is not None:
        ws = _workspace(nbytes, workspace, dev)
        return ws, ws.data_ptr(), _nbytes(ws)
    if nbytes == 0:
        return None, 0, 0
    ws = _empty(nbytes, torch.uint8, dev, stream)
    return ws, ws.data_ptr(), nbytes


def _ptr(t):
    return t.data_ptr() if t is not None else 0


def embedding(table, ids, *, scale=1.0, dtype=None, dev_status=None, out=None, stream=None):
    """scale * table[ids], [*ids.shape, D] in `dtype` (default: the table's).  Rows of negative
    ids are zeros; an id >= V sets the status word and gives NaN.  table and out ([N, D])
    may have rows further apart than their length."""
    dt, ld = _rows(table, "table")
    _need(ids, "ids", torch.int32)
    V, D = table.shape
    N = ids.numel()
    dev = _device(table, ids=ids)
    if out is None:
        dtype = table.dtype if dtype is None else dtype
        odt, old = _DTYPES.get(dtype), D
        if odt is None:
            raise TypeError(f"dtype must be bfloat16 or float32, got {dtype}")
        out = _made((*ids.shape, D), dtype, dev, stream)
    else:
        odt, old = _rows(out, "out", (N, D), dev)
        if dtype is not None and dtype != out.dtype:
            raise TypeError(f"out must be {dtype}, got {out.dtype}")
    if dev_status is not None:
        _status(dev_status, dev)
    rc = lib().dflash2_embedding(table.data_ptr(), dt, V, D, ld, ids.data_ptr(), N, scale, out.data_ptr(), odt, old,
                                 _ptr(dev_status), _stream(stream, dev))
    _check("dflash2_embedding", rc)
    return out


@functools.lru_cache(maxsize=256)
def _size(library, query, *shape):
    """A workspace query's answer for a shape (it depends on nothing else)."""
    return int(getattr(library, query)(*shape))


def embedding_grad_workspace_size(N, V, D) -> int:
    return _size(lib(), "dflash2_embedding_grad_workspace_size", N, V, D)


def embedding_grad(dout, ids, V, *, scale=1.0, dtype=torch.float32, accumulate=False, workspace=None,
                   dev_status=None, out=None, stream=None):
    """The gradient [V, D] of embedding()'s table: scale * the sum of dout's rows of each
    token, in fp32, the same bits every time.  accumulate adds to `out`; otherwise every
    row is written.  dout is [N, D], or [*ids.shape, D] where contiguous."""
    _need(ids, "ids", torch.int32)
    N = ids.numel()
    if isinstance(dout, torch.Tensor) and dout.dim() != 2 and dout.dim() == ids.dim() + 1 and dout.is_contiguous():
        dout = dout.view(N, dout.shape[-1])
    dt, ld = _rows(dout, "dout")
    rows, D = dout.shape
    if rows != N:
        raise ValueError(f"dout must have a row an id ({N}), got {rows}")
    V = int(V)
    dev = _device(dout, ids=ids)
    if out is None:
        if accumulate:
            raise ValueError("accumulate adds to out: out must be given")
        if dtype not in _DTYPES:
            raise TypeError(f"dtype must be bfloat16 or float32, got {dtype}")
        out = _made((V, D), dtype, dev, stream)
        odt, old = _DTYPES[dtype], max(D, 1)
    else:
        odt, old = _rows(out, "out", (V, D), dev)
    if dev_status is not None:
        _status(dev_status, dev)
    _ws, ws, nbytes = _scratch(embedding_grad_workspace_size(N, V, D), workspace, dev, stream)
    rc = lib().dflash2_embedding_grad(dout.data_ptr(), dt, ld, ids.data_ptr(), N, V, D, scale, bool(accumulate),
                                      out.data_ptr(), odt, old, ws, nbytes, _ptr(dev_status), _stream(stream, dev))
    _check("dflash2_embedding_grad", rc)
    return out


def selector_loss_grad_workspace_size(P, V, K, r) -> int:
    return _size(lib(), "dflash2_selector_loss_grad_workspace_size", P, V, K, r)


def selector_loss_grad(pred, targets, topk_ids, topk_vals, G, A, Bc, *, row_weights=None, accumulate=False,
                       dA=True, dBc=True, dtype=torch.float32, workspace=None, dev_status=None, out=None, stream=None):
    """The selector's K-way loss of the teacher-forced scores and the gradients of
    sum(row_weights * loss).  Returns (loss [P], label [P] int32, dscores [P, K], dG [P, r],
    dA [V, r], dBc [V, r]); rows without a candidate target give label -1, NaN loss and
    contribute nothing.

    dA, dBc: a tensor to write (or with accumulate to add to), True for a new one in
    `dtype`, None to leave it out.  out: (loss, label, dscores, dG)."""
    _need(pred, "pred", torch.int32, 1)
    _need(targets, "targets", torch.int32, 1)
    _need(topk_ids, "topk_ids", torch.int32)
    _need(topk_vals, "topk_vals", torch.float32)
    _need(G, "G", torch.float32)
    _need(A, "A", torch.bfloat16, 2)
    _need(Bc, "Bc", torch.bfloat16, 2)
    P = pred.shape[0]
    K = topk_ids.shape[-1]
    V, r = A.shape
    if targets.shape[0] != P or topk_ids.numel() != P * K or topk_vals.numel() != P * K or G.numel() != P * r:
        raise ValueError("shapes do not match [P], [P, K], [P, r]")
    if tuple(Bc.shape) != (V, r):
        raise ValueError("Bc must be [V, r] like A")
    if row_weights is not None:
        _need(row_weights, "row_weights", torch.float32)
        if row_weights.numel() != P:
            raise ValueError("row_weights must be [P]")
    dev = _device(pred, targets=targets, topk_ids=topk_ids, topk_vals=topk_vals, G=G, A=A, Bc=Bc,
                  row_weights=row_weights)
    given = [t for t in (dA, dBc) if isinstance(t, torch.Tensor)]
    if given:
        dtype = given[0].dtype
    if dtype not in _DTYPES:
        raise TypeError(f"dA and dBc must be bfloat16 or float32, got {dtype}")
    if accumulate and (dA is True or dBc is True):
        raise ValueError("accumulate adds to dA and dBc: they must be given (None leaves one out)")
    for name, t in (("dA", dA), ("dBc", dBc)):
        if t is not None and t is not True:
            _out(t, name, dtype, V * r, dev)
    if dA is True:
        dA = _made((V, r), dtype, dev, stream)
    if dBc is True:
        dBc = _made((V, r), dtype, dev, stream)
    if out is None:
        loss, label = _made((P,), torch.float32, dev, stream), _made((P,), torch.int32, dev, stream)
        ds, dG = _made((P, K), torch.float32, dev, stream), _made((P, r), torch.float32, dev, stream)
    else:
        loss, label, ds, dG = out
        _out(loss, "loss", torch.float32, P, dev)
        _out(label, "label", torch.int32, P, dev)
        _out(ds, "dscores", torch.float32, P * K, dev)
        _out(dG, "dG", torch.float32, P * r, dev)
    if dev_status is not None:
        _status(dev_status, dev)
    _ws, ws, nbytes = _scratch(selector_loss_grad_workspace_size(P, V, K, r), workspace, dev, stream)
    rc = lib().dflash2_selector_loss_grad(
        pred.data_ptr(), targets.data_ptr(), P, topk_ids.data_ptr(), topk_vals.data_ptr(), G.data_ptr(), A.data_ptr(),
        Bc.data_ptr(), V, K, r, _ptr(row_weights), bool(accumulate), loss.data_ptr(), label.data_ptr(), ds.data_ptr(),
        dG.data_ptr(), _ptr(dA), _ptr(dBc), _DTYPES[dtype], ws, nbytes, _ptr(dev_status), _stream(stream, dev))
    _check("dflash2_selector_loss_grad", rc)
    return loss, label, ds, dG, dA, dBc


def _loss_inputs(h, W_lm, targets):
    """The unary loss's inputs: (P, D, V, device)."""
    _need(h, "h", torch.bfloat16, 2)
    _need(W_lm, "W_lm", torch.bfloat16, 2)
    _need(targets, "targets", torch.int32)
    (P, D), (V, width) = h.shape, W_lm.shape
    if width != D:
        raise ValueError("W_lm must be [V, D]")
    if targets.numel() != P:
        raise ValueError(f"targets must be [P] ({P}), got {list(targets.shape)}")
    return P, D, V, _device(h, W_lm=W_lm, targets=targets)


def _loss_outputs(out, P, dev, stream):
    if out is None:
        return _made((P,), torch.float32, dev, stream), _made((P,), torch.float32, dev, stream)
    loss, lse = out
    _out(loss, "loss", torch.float32, P, dev)
    if lse is not None:
        _out(lse, "lse", torch.float32, P, dev)
    return loss, lse


def unary_ce_workspace_size(P, D, V) -> int:
    return int(lib().dflash2_unary_ce_workspace_size(P, D, V))


def unary_ce(h, W_lm, targets, *, output_multiplier=1.0, final_logit_softcapping=0.0, workspace=None, dev_status=None,
             out=None, stream=None):
    """The cross-entropy of unary_topk()'s logits over the whole vocabulary, which are never
    stored: (loss [P], lse [P]), fp32, with lse the logarithm of each row's sum of exponentials.
    Rows whose target is negative give NaN in both.  out: (loss, lse or None)."""
    P, D, V, dev = _loss_inputs(h, W_lm, targets)
    loss, lse = _loss_outputs(out, P, dev, stream)
    _status(dev_status, dev)
    _ws, ws, nbytes = _scratch(unary_ce_workspace_size(P, D, V), workspace, dev, stream)
    rc = lib().dflash2_unary_ce(h.data_ptr(), P, D, W_lm.data_ptr(), V, float(output_multiplier),
                                float(final_logit_softcapping), targets.data_ptr(), loss.data_ptr(), _ptr(lse), ws, nbytes,
                                _ptr(dev_status), _stream(stream, dev))
    _check("dflash2_unary_ce", rc)
    return loss, lse


def unary_loss_grad_workspace_size(P, D, V, dh=True, dW=False) -> int:
    return int(lib().dflash2_unary_loss_grad_workspace_size(P, D, V, bool(dh), bool(dW)))


def unary_loss_grad(h, W_lm, targets, *, row_weights=None, output_multiplier=1.0, final_logit_softcapping=0.0,
                    accumulate=False, dh=True, dW=None, dtype=torch.bfloat16, workspace=None, dev_status=None, out=None,
                    stream=None):
    """unary_ce() and the gradients of sum(row_weights * loss): (loss [P], lse [P], dh [P, D],
    dW [V, D]); rows without a target (negative) give NaN, a zero row of dh, and nothing to dW.

    dh, dW: a tensor to write (dW: with accumulate to add to), True for a new one in
    `dtype`, None to leave it out (dW by default: the head is the verifier's).  The factors of
    the products are rounded to bf16 in either type.  out: (loss, lse or None)."""
    P, D, V, dev = _loss_inputs(h, W_lm, targets)
    if row_weights is not None:
        _need(row_weights, "row_weights", torch.float32)
        if row_weights.numel() != P or row_weights.device != dev:
            raise ValueError("row_weights must be [P] on the call's device")
    if accumulate and not isinstance(dW, torch.Tensor):
        raise ValueError("accumulate adds to dW: it must be given")
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be bfloat16 or float32, got {dtype}")
    for name, t, n in (("dh", dh, P * D), ("dW", dW, V * D)):
        if t is not None and t is not True:
            if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES:
                raise TypeError(f"{name} must be a bfloat16 or float32 CUDA tensor, True or None")
            _out(t, name, t.dtype, n, dev)
    if dh is True:
        dh = _made((P, D), dtype, dev, stream)
    if dW is True:
        dW = _made((V, D), dtype, dev, stream)
    loss, lse = _loss_outputs(out, P, dev, stream)
    _status(dev_status, dev)
    _ws, ws, nbytes = _scratch(unary_loss_grad_workspace_size(P, D, V, dh is not None, dW is not None), workspace, dev,
                               stream)
    rc = lib().dflash2_unary_loss_grad(
        h.data_ptr(), P, D, W_lm.data_ptr(), V, float(output_multiplier), float(final_logit_softcapping),
        targets.data_ptr(), _ptr(row_weights), bool(accumulate), loss.data_ptr(), _ptr(lse), _ptr(dh),
        0 if dh is None else _DTYPES[dh.dtype], _ptr(dW), 0 if dW is None else _DTYPES[dW.dtype], ws, nbytes,
        _ptr(dev_status), _stream(stream, dev))
    _check("dflash2_unary_loss_grad", rc)
    return loss, lse, dh, dW


def _random(rate, seed, draw, dev):
    """rate, seed and draw as the library takes them: (rate, seed, draw, its address)."""
    rate = float(rate)
    if not 0.0 <= rate <= 1.0:
        raise ValueError(f"rate must be in [0, 1], got {rate}")
    seed = operator.index(seed)
    if isinstance(draw, torch.Tensor):
        _need(draw, "draw", torch.int64)
        if draw.numel() != 1 or draw.device != dev:
            raise ValueError("draw must be one int64 on the call's device")
        number, at = 0, draw.data_ptr()
    else:
        number, at = operator.index(draw), 0
    if not (0 <= seed < 1 << 64 and 0 <= number < 1 << 64):
        raise ValueError(f"seed and draw must be in [0, 2^64), got {seed} and {number}")
    return rate, seed, number, at


def dropout(x, rate, seed, draw=0, *, residual=None, dtype=None, out=None, stream=None):
    """x with each element dropped with probability `rate` (in steps of 2^-16) and the others
    scaled by 1 / (1 - rate), plus `residual`, in `dtype` (default: out's, or the residual's,
    or x's).  The mask is a function of seed, draw and the element's index in x: nothing is stored,
    dropout_grad makes it again, and another draw gives another mask.

    draw: an integer, or an int64 tensor of one element on the GPU, read when the kernel
    runs; a call that is being captured into a graph needs the tensor.  x, residual and out:
    bf16 or fp32 matrices whose rows may be further apart than their length (residual of
    out's type), or contiguous tensors of any shape.  out may be x or residual."""
    if not isinstance(x, torch.Tensor) or not _on_device(x):
        raise TypeError("x must be a CUDA tensor")
    dev = _device(x)
    rate, seed, number, at = _random(rate, seed, draw, dev)
    for name, t in (("residual", residual), ("out", out)):
        if t is not None:
            if not isinstance(t, torch.Tensor) or t.device != dev:
                raise TypeError(f"{name} must be a tensor on {dev}")
            if t.shape != x.shape:
                raise ValueError(f"{name} must have x's shape {list(x.shape)}, got {list(t.shape)}")
    if out is not None:
        if dtype is not None and dtype != out.dtype:
            raise TypeError(f"out must be {dtype}, got {out.dtype}")
        dtype = out.dtype
    elif dtype is None:
        dtype = (x if residual is None else residual).dtype
    dt, odt = _DTYPES.get(x.dtype), _DTYPES.get(dtype)
    if dt is None or odt is None:
        raise TypeError(f"x and dtype must be bfloat16 or float32, got {x.dtype} and {dtype}")
    if residual is not None and residual.dtype != dtype:
        raise TypeError(f"residual must be {dtype} like the output, got {residual.dtype}")
    dense = x.is_contiguous() and (residual is None or residual.is_contiguous()) and (out is None or out.is_contiguous())
    if not dense and x.dim() != 2:
        raise ValueError("x, residual and out must be matrices or contiguous")
    if out is None:
        out = _made(x.shape, dtype, dev, stream)
    if dense:  # one row
        N, D = 1, x.numel()
        ld = rld = old = D
    else:
        N, D = x.shape
        ld, old = _rows(x, "x")[1], _rows(out, "out")[1]
        rld = 0 if residual is None else _rows(residual, "residual")[1]
    if N * D == 0:
        return out
    rc = lib().dflash2_dropout(x.data_ptr(), dt, N, D, ld, rate, seed, number, at, _ptr(residual), rld, out.data_ptr(),
                               odt, old, _stream(stream, dev))
    if rc == DF2_ERR_UNSUPPORTED and not at and _capturing(stream, dev):
        raise RuntimeError("a captured dropout needs its draw as a tensor on the GPU: with a number every replay "
                           "would drop the same elements")
    _check("dflash2_dropout", rc)
    return out


def dropout_grad(dout, rate, seed, draw=0, *, dtype=None, accumulate=False, out=None, stream=None):
    """The gradient of dropout()'s x: dropout() of dout with the same rate, seed and draw.
    accumulate adds it to `out`.  (The residual's gradient is dout itself.)"""
    if accumulate and out is None:
        raise ValueError("accumulate adds to out: out must be given")
    return dropout(dout, rate, seed, draw, residual=out if accumulate else None, dtype=dtype, out=out, stream=stream)


from .optim import AdamW  # noqa: E402  (needs the checks above)
