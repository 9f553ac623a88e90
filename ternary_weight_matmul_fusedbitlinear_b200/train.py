"""Training calls of libmmf.so: BitLinear and GLU with activations kept in 8 bits, and the LM-head loss.

A forward call returns its output and what the backward needs: the int8 codes
that the forward contraction read anyway (1 byte per element), never a second
copy of the activations and never the logits. As in api.py there is no
arithmetic here, only argument checks and library calls on the current stream
of the input's device.

    pre, k1 = bitlinear_train([f, c, g], x)              # [..., 3, N]: the scan's pre-activations
    y, k2 = glu_train(gate, up, down, x1, residual=x1)
    loss, k3 = head_loss(head, y, labels)
    g3 = head_loss_backward(head, k3, labels)
    g2 = glu_backward(gate, up, down, k2, g3.dx, dres=g3.dx)   # dres: the residual's own gradient
    ...
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional, Sequence, Union

import torch

from . import _lib as L
from .api import DEFAULT_EPS, TLinear, _dtype, _need_cuda, _stream, _workspace

_REDUCTIONS = {"none": 0, "sum": 1, "mean": 2}


class Act8(NamedTuple):
    """A layer's input [M, K] as its forward kept it: int8 codes q [M, K] with x^ = q / scale,
    scale [M], qsum [M] (int32 sums of the codes) and rinv [M] (1 / rms)."""
    q: torch.Tensor
    scale: torch.Tensor
    qsum: torch.Tensor
    rinv: torch.Tensor


class HeadKept(NamedTuple):
    """What head_loss keeps: the codes of its input, lse [M], the number of counted tokens [1], its input's dtype."""
    act: Act8
    lse: torch.Tensor
    count: torch.Tensor
    dtype: torch.dtype


class LinearGrads(NamedTuple):
    """dx [..., K]; dw: one [N, K] per layer; dgain [K] or None; dbias: [N] or None per layer."""
    dx: torch.Tensor
    dw: list
    dgain: Optional[torch.Tensor]
    dbias: list


class GluGrads(NamedTuple):
    """dx [..., d]; dw: of gate, up, down; dgain: of the shared gain and of down's; dbias: of gate, up, down
    (None where the layer has none)."""
    dx: torch.Tensor
    dw: list
    dgain: list
    dbias: list


def _on(device: torch.device):
    """Run on `device`, whichever one is current."""
    return contextlib.nullcontext() if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _same_device(first: torch.Tensor, *ts: Optional[torch.Tensor]) -> None:
    _need_cuda(first, *ts)
    for t in ts:
        if t is not None and t.device != first.device:
            raise ValueError("all tensors must be on one device")


def _layer_tensors(lins: Sequence[TLinear]) -> list:
    return [t for lin in lins for t in (lin.packed, lin.gamma, lin.gain, lin.bias, lin.codes)]


def _c_layers(lins: Sequence[TLinear]):
    return (L.TLinear * len(lins))(*[lin.c() for lin in lins])


def _layers(lins: Union[TLinear, Sequence[TLinear]]) -> list:
    out = [lins] if isinstance(lins, TLinear) else list(lins)
    if not 1 <= len(out) <= 3:
        raise ValueError("1 to 3 layers share one input")
    return out


def _rows(x: torch.Tensor, width: int, what: str) -> int:
    if x.dim() < 1 or x.shape[-1] != width:
        raise ValueError(f"{what} must be [..., {width}], got {tuple(x.shape)}")
    return x.numel() // width


def _new_kept(m: int, k: int, device: torch.device) -> Act8:
    rows = torch.empty(3, max(4, (m + 3) // 4 * 4), dtype=torch.float32, device=device)   # 16-byte aligned rows
    return Act8(torch.empty(m, k, dtype=torch.int8, device=device), rows[0, :m], rows[1, :m].view(torch.int32),
                rows[2, :m])


def _c_kept(kept: Act8, m: int, k: int, like: torch.Tensor) -> L.Act8:
    q, s, qs, r = kept
    if q.shape != (m, k) or s.shape != (m,) or qs.shape != (m,) or r.shape != (m,):
        raise ValueError(f"kept activations must be those of an input of {m} rows of {k}")
    if q.dtype != torch.int8 or qs.dtype != torch.int32 or s.dtype != torch.float32 or r.dtype != torch.float32:
        raise ValueError("kept activations must be int8 codes, float32 scale and rinv, int32 qsum")
    _same_device(like, q, s, qs, r)
    return L.Act8(q.data_ptr(), s.data_ptr(), qs.data_ptr(), r.data_ptr())


def _like(t: Optional[torch.Tensor], ref: torch.Tensor, what: str) -> None:
    if t is not None and (t.numel() != ref.numel() or t.dtype != ref.dtype):
        raise ValueError(f"{what} must have the shape and dtype of the input")


def _bytes(ws: torch.Tensor) -> int:
    return ws.numel() * ws.element_size()


# ---------------------------------------------------------------- BitLinear

def bitlinear_train(lins: Union[TLinear, Sequence[TLinear]], x: torch.Tensor, eps: float = DEFAULT_EPS,
                    ws: Optional[torch.Tensor] = None):
    """Training forward of 1 to 3 layers of one shape and gain on x [..., K] (mmf_bitlinear_train).

    Returns (y, kept): y [..., N] for a layer, [..., n, N] for a sequence of n; kept: Act8."""
    ls = _layers(lins)
    _same_device(x, *_layer_tensors(ls))
    n, N, K = len(ls), ls[0].N, ls[0].K
    m = _rows(x, K, "x")
    dev = x.device
    lead = x.shape[:-1]
    y = torch.empty(*lead, N, dtype=x.dtype, device=dev) if isinstance(lins, TLinear) else \
        torch.empty(*lead, n, N, dtype=x.dtype, device=dev)
    kept = _new_kept(m, K, dev)
    lib = L.load()
    w = _workspace(lib.mmf_bitlinear_train_ws_size(n, N, K), dev, ws)
    ck = _c_kept(kept, m, K, x)
    with _on(dev):
        L.check(lib.mmf_bitlinear_train(_c_layers(ls), n, x.data_ptr(), _dtype(x), m, y.data_ptr(), eps,
                                        ctypes.byref(ck), w.data_ptr(), _bytes(w), _stream(dev)),
                "mmf_bitlinear_train")
    return y, kept


def bitlinear_backward(lins: Union[TLinear, Sequence[TLinear]], kept: Act8, dy: torch.Tensor,
                       x: Optional[torch.Tensor] = None, dres: Optional[torch.Tensor] = None,
                       ws: Optional[torch.Tensor] = None) -> LinearGrads:
    """Gradients of bitlinear_train for dy in y's shape (mmf_bitlinear_backward), all in dy's dtype.

    x: the forward's input, for layers whose gain comes near 0 (otherwise read from the codes);
    dres: added to dx, e.g. the gradient that reaches x along a residual."""
    ls = _layers(lins)
    _same_device(dy, x, dres, *_layer_tensors(ls))
    n, N, K = len(ls), ls[0].N, ls[0].K
    one = isinstance(lins, TLinear)
    m = _rows(dy, N, "dy")
    if not one:
        if dy.dim() < 2 or dy.shape[-2] != n:
            raise ValueError(f"dy must be [..., {n}, {N}], got {tuple(dy.shape)}")
        m //= n
    dev, dt = dy.device, dy.dtype
    code = _dtype(dy)
    dx = torch.empty(*dy.shape[:-1 if one else -2], K, dtype=dt, device=dev)
    _like(x, dx, "x")
    _like(dres, dx, "dres")
    ck = _c_kept(kept, m, K, dy)
    dw = [torch.empty(N, K, dtype=dt, device=dev) for _ in ls]
    dgain = torch.empty(K, dtype=dt, device=dev) if ls[0].gain is not None else None
    dbias = [torch.empty(N, dtype=dt, device=dev) if lin.bias is not None else None for lin in ls]
    fill = [None] * (3 - n)
    cg = L.LinearGrads(dx.data_ptr(), (L.c_vp * 3)(*[t.data_ptr() for t in dw], *fill), _p(dgain),
                       (L.c_vp * 3)(*[_p(t) for t in dbias], *fill))
    lib = L.load()
    w = _workspace(lib.mmf_bitlinear_backward_ws_size(n, N, K, m, code), dev, ws)
    with _on(dev):
        L.check(lib.mmf_bitlinear_backward(_c_layers(ls), n, ctypes.byref(ck), _p(x), dy.data_ptr(), _p(dres), code, m,
                                           ctypes.byref(cg), w.data_ptr(), _bytes(w), _stream(dev)),
                "mmf_bitlinear_backward")
    return LinearGrads(dx, dw, dgain, dbias)


# ---------------------------------------------------------------- GLU

def _glu_layers(gate: TLinear, up: TLinear, down: TLinear):
    ls = [gate, up, down]
    return ls, [ctypes.byref(lin.c()) for lin in ls]


def glu_train(gate: TLinear, up: TLinear, down: TLinear, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
              eps: float = DEFAULT_EPS, ws: Optional[torch.Tensor] = None):
    """glu() that keeps the codes of x and of the product: (y, (kept_x, kept_p)) (mmf_glu_train)."""
    ls, cl = _glu_layers(gate, up, down)
    _same_device(x, residual, *_layer_tensors(ls))
    d, inner = gate.K, gate.N
    m = _rows(x, d, "x")
    _like(residual, x, "residual")
    dev, code = x.device, _dtype(x)
    y = torch.empty_like(x)
    kx, kp = _new_kept(m, d, dev), _new_kept(m, inner, dev)
    lib = L.load()
    w = _workspace(lib.mmf_glu_train_ws_size(m, d, inner, code), dev, ws)
    with _on(dev):
        L.check(lib.mmf_glu_train(*cl, x.data_ptr(), _p(residual), y.data_ptr(), m, code, eps,
                                  ctypes.byref(_c_kept(kx, m, d, x)), ctypes.byref(_c_kept(kp, m, inner, x)),
                                  w.data_ptr(), _bytes(w), _stream(dev)), "mmf_glu_train")
    return y, (kx, kp)


def glu_backward(gate: TLinear, up: TLinear, down: TLinear, kept, dy: torch.Tensor, x: Optional[torch.Tensor] = None,
                 dres: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> GluGrads:
    """Gradients of glu_train for dy [..., d] (mmf_glu_backward); kept, x, dres as in bitlinear_backward.

    With residual=x in the forward, pass dres=dy."""
    ls, cl = _glu_layers(gate, up, down)
    _same_device(dy, x, dres, *_layer_tensors(ls))
    d, inner = gate.K, gate.N
    m = _rows(dy, d, "dy")
    _like(x, dy, "x")
    _like(dres, dy, "dres")
    dev, dt, code = dy.device, dy.dtype, _dtype(dy)
    kx, kp = (_c_kept(k, m, n, dy) for k, n in zip(kept, (d, inner)))
    dx = torch.empty_like(dy)
    dw = [torch.empty(lin.N, lin.K, dtype=dt, device=dev) for lin in ls]
    dgain = [torch.empty(lin.K, dtype=dt, device=dev) if lin.gain is not None else None for lin in (gate, down)]
    dbias = [torch.empty(lin.N, dtype=dt, device=dev) if lin.bias is not None else None for lin in ls]
    cg = L.GluGrads(dx.data_ptr(), *[t.data_ptr() for t in dw], *[_p(t) for t in dgain], *[_p(t) for t in dbias])
    lib = L.load()
    w = _workspace(lib.mmf_glu_backward_ws_size(m, d, inner, code), dev, ws)
    with _on(dev):
        L.check(lib.mmf_glu_backward(*cl, ctypes.byref(kx), ctypes.byref(kp), _p(x), dy.data_ptr(), _p(dres), code, m,
                                     ctypes.byref(cg), w.data_ptr(), _bytes(w), _stream(dev)), "mmf_glu_backward")
    return GluGrads(dx, dw, dgain, dbias)


# ---------------------------------------------------------------- LM head loss

def _head_args(head: TLinear, labels: torch.Tensor, m: int, reduction: str) -> int:
    if reduction not in _REDUCTIONS:
        raise ValueError(f"reduction must be one of {sorted(_REDUCTIONS)}")
    if labels.dtype != torch.int32 or labels.numel() != m:
        raise ValueError(f"labels must be int32, one per token ({m})")
    return _REDUCTIONS[reduction]


def head_loss(head: TLinear, x: torch.Tensor, labels: torch.Tensor, ignore_index: int = -100,
              reduction: str = "mean", eps: float = DEFAULT_EPS, ws: Optional[torch.Tensor] = None):
    """Softmax cross entropy of the logits head(x) against int32 labels, without storing the logits
    (mmf_head_loss): (loss, kept). loss is a float32 scalar ("mean" over the counted tokens, "sum") or the
    per-token losses in labels' shape ("none"); kept: HeadKept for head_loss_backward."""
    _same_device(x, labels, *_layer_tensors([head]))
    m = _rows(x, head.K, "x")
    red = _head_args(head, labels, m, reduction)
    dev = x.device
    loss = torch.empty(labels.shape if red == 0 else (), dtype=torch.float32, device=dev)
    kept = HeadKept(_new_kept(m, head.K, dev), torch.empty(m, dtype=torch.float32, device=dev),
                    torch.empty(1, dtype=torch.float32, device=dev), x.dtype)
    lib = L.load()
    w = _workspace(lib.mmf_head_loss_ws_size(m, head.N, head.K), dev, ws)
    with _on(dev):
        L.check(lib.mmf_head_loss(ctypes.byref(head.c()), x.data_ptr(), _dtype(x), m, labels.data_ptr(), ignore_index,
                                  red, eps, loss.data_ptr(), ctypes.byref(_c_kept(kept.act, m, head.K, x)),
                                  kept.lse.data_ptr(), kept.count.data_ptr(), w.data_ptr(), _bytes(w), _stream(dev)),
                "mmf_head_loss")
    return loss, kept


def head_loss_backward(head: TLinear, kept: HeadKept, labels: torch.Tensor, dloss: Optional[torch.Tensor] = None,
                       ignore_index: int = -100, reduction: str = "mean", x: Optional[torch.Tensor] = None,
                       ws: Optional[torch.Tensor] = None) -> LinearGrads:
    """Gradients of head_loss for dloss (float32: one value, or one per token for "none"; None: 1), in the dtype
    of the forward's input (mmf_head_loss_backward); labels, ignore_index and reduction as there, x as in
    bitlinear_backward."""
    _same_device(labels, dloss, x, kept.lse, kept.count, *_layer_tensors([head]))
    m, N, K = labels.numel(), head.N, head.K
    red = _head_args(head, labels, m, reduction)
    dev, dt = labels.device, kept.dtype
    if dloss is not None and (dloss.dtype != torch.float32 or dloss.numel() != (m if red == 0 else 1)):
        raise ValueError("dloss must be float32, one value (one per token for reduction 'none')")
    if kept.lse.numel() != m:
        raise ValueError("kept must come from head_loss on the same tokens")
    ck = _c_kept(kept.act, m, K, labels)
    dx = torch.empty(*labels.shape, K, dtype=dt, device=dev)
    _like(x, dx, "x")
    code = _dtype(dx)
    dw = torch.empty(N, K, dtype=dt, device=dev)
    dgain = torch.empty(K, dtype=dt, device=dev) if head.gain is not None else None
    dbias = torch.empty(N, dtype=dt, device=dev) if head.bias is not None else None
    cg = L.LinearGrads(dx.data_ptr(), (L.c_vp * 3)(dw.data_ptr()), _p(dgain), (L.c_vp * 3)(_p(dbias)))
    lib = L.load()
    w = _workspace(lib.mmf_head_loss_backward_ws_size(m, N, K, code), dev, ws)
    with _on(dev):
        L.check(lib.mmf_head_loss_backward(ctypes.byref(head.c()), ctypes.byref(ck), _p(x), labels.data_ptr(),
                                           kept.lse.data_ptr(), kept.count.data_ptr(), _p(dloss), ignore_index, red,
                                           code, m, ctypes.byref(cg), w.data_ptr(), _bytes(w), _stream(dev)),
                "mmf_head_loss_backward")
    return LinearGrads(dx, [dw], dgain, [dbias])
