"""Measured cases of the training operators: BitLinear and GLU with activations kept in 8 bits, and the LM-head loss.

Each case is one operator in one direction on seeded inputs. The plain forms below are elementary torch
operations in fp32 (fp64 for sums of squares); with `own` set, `run` makes the library calls instead.

  linear   1..3 ternary BitLinear layers of one input: forward keeping the int8 codes, and the gradients
           of the input, the latent weights (straight through both roundings), the norm's gain and the biases
  glu      the channel mixer down(SiLU(gate(x)) up(x)), trained the same way from the codes of its two inputs
  loss     softmax cross entropy of a ternary head's logits, per token or reduced, and its gradients

Directions: "forward", "backward" (the codes are in hand) and "step" (forward, then backward).
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def _linear(name, way, m, k, n, layers=1, dtype="bf16", gain=False, bias=False, keep_x=False):
    c = {"op": "linear", "way": way, "m": m, "k": k, "n": n, "layers": layers, "dtype": dtype, "gain": gain,
         "bias": bias, "keep_x": keep_x}
    return dict(c, name=name) if name else c


def _glu(name, way, m, d, inner, dtype="bf16", gain=False, bias=False):
    c = {"op": "glu", "way": way, "m": m, "d": d, "inner": inner, "dtype": dtype, "gain": gain, "bias": bias}
    return dict(c, name=name) if name else c


def _loss(name, way, m, k, v, dtype="bf16", reduction="mean", ignored=0.0, gain=False, bias=False):
    c = {"op": "loss", "way": way, "m": m, "k": k, "v": v, "dtype": dtype, "reduction": reduction,
         "ignored": ignored, "gain": gain, "bias": bias}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token through one small projection: launch latency
        _linear("linear step, 1 token f32", "step", 1, 256, 256, dtype="f32"),
        # a small fp32 run (d = 256, inner size 768, 2 x 64 tokens): its down projection, with a gain
        _linear("linear step, small f32", "step", 128, 768, 256, dtype="f32", gain=True),
        # odd token count and output width, gain and bias, the input kept for the norm's gradient
        _linear("linear step, ragged", "step", 1003, 1040, 777, gain=True, bias=True, keep_x=True),
        # the 1.3B shape's f, c, g projections of one input, 4 x 2048 tokens
        _linear("linear step, f|c|g 1.3B", "step", 8192, 2048, 2048, layers=3),
        # the 370M shape's down projection, 8 x 2048 tokens
        _linear("linear backward, 370M down", "backward", 16384, 2816, 1024),
        # the small fp32 run's channel mixer
        _glu("glu backward, small f32", "backward", 128, 256, 768, dtype="f32"),
        # widths that are multiples of 16 only, an odd token count, gains and biases
        _glu("glu step, ragged", "step", 333, 272, 400, gain=True, bias=True),
        # the 370M shape's channel mixer, 8 x 2048 tokens: the largest part of a training step
        _glu("glu step, 370M", "step", 16384, 1024, 2816),
        # the 2.7B shape's channel mixer on 8 x 512 tokens, backward alone
        _glu("glu backward, 2.7B", "backward", 4096, 2560, 6912),
        # evaluation: per-token losses over the 32000-entry vocabulary, 8 x 2048 tokens of the 370M shape
        _loss("loss forward, 370M", "forward", 16384, 1024, 32000, reduction="none"),
        # a training step's head, 4 x 2048 tokens of the 1.3B shape, padded batches
        _loss("loss step, 1.3B", "step", 8192, 2048, 32000, ignored=0.1),
        # an odd small vocabulary in fp32, a tenth of the labels ignored
        _loss("loss step, small f32", "step", 130, 256, 1003, dtype="f32", reduction="sum", ignored=0.1, bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _flops_of(case):
    return work(case)["flops"]


def draw(rng):
    most = 0.9 * max(_flops_of(c) for c in listed())
    while True:
        op = rng.choice(["linear", "linear", "glu", "glu", "loss", "loss"])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        m = _log(rng, 1, 16384)
        k = 16 * _log(rng, 4, 200)
        gain, bias = rng.random() < 0.4, rng.random() < 0.4
        if op == "linear":
            c = _linear(None, rng.choice(["step", "backward"]), m, k, _log(rng, 16, 7000), rng.choice([1, 1, 2, 3]),
                        dtype, gain, bias, rng.random() < 0.3)
        elif op == "glu":   # in fp32 the product's own codes are given: they are decided by its last bits
            way = "backward" if dtype == "f32" else rng.choice(["step", "backward"])
            c = _glu(None, way, m, k, 16 * _log(rng, 4, 440), dtype, gain, bias)
        else:
            c = _loss(None, rng.choice(["forward", "step", "step"]), m, k, _log(rng, 100, 50000), dtype,
                      rng.choice(["mean", "sum", "none"]), rng.choice([0.0, 0.1, 0.5]), gain, bias)
        if _flops_of(c) <= (most if dtype == "bf16" else most / 3):
            return c


def work(case):
    """What one pass reads, writes and computes: packed 2-bit weights, 8-bit codes, each product once."""
    e = 2 if case["dtype"] == "bf16" else 4
    way, m = case["way"], case["m"]
    fwd, bwd = way in ("forward", "step"), way in ("backward", "step")
    if case["op"] == "linear":
        k, n = case["k"], case["n"] * case["layers"]
        b = n * k / 4 + (m * k * e + m * n * e if fwd else 0)
        b += (m * n * e + m * k * (1 + e) + n * k * e) if bwd else 0
        return {"bytes": b, "flops": 2.0 * m * n * k * (fwd + 2 * bwd)}
    if case["op"] == "glu":
        d, i = case["d"], case["inner"]
        b = 3 * d * i / 4 + (2 * m * d * e if fwd else 0)
        b += (m * (d + i) + 2 * m * d * e + 3 * d * i * e) if bwd else 0
        return {"bytes": b, "flops": 2.0 * m * d * i * (3 * fwd + 8 * bwd)}
    k, v = case["k"], case["v"]
    b = v * k / 4 + m * k * e + 4 * m + (m * k * e + v * k * e if bwd else 0)
    return {"bytes": b, "flops": 2.0 * m * k * v * (fwd + 3 * bwd)}


# ---------------------------------------------------------------- inputs

def _pack(w):
    """Codes w in {-1, 0, 1} [N, K] as 2-bit fields of int32 words: column 16j + 4i + b at bits 8b + 2i of word j."""
    n, k = w.shape
    f = (w + 1).to(torch.int64).view(n, k // 16, 4, 4)                 # [n, j, i, b]
    i = torch.arange(4, device=w.device).view(1, 1, 4, 1)
    b = torch.arange(4, device=w.device).view(1, 1, 1, 4)
    return (f << (8 * b + 2 * i)).sum((2, 3)).to(torch.int32)


def _layer(g, n, k, std, gain, bias, dtype):
    """One ternary layer: its codes, their packed words, scale, gain and bias."""
    latent = torch.randn(n, k, generator=g, device="cuda") * std
    gamma = latent.abs().double().mean().float()
    w = torch.clamp(torch.round(latent / (gamma + 1e-5)), -1, 1).to(torch.int8)
    slot = torch.zeros(4, device="cuda")
    slot[0] = gamma
    return {"w": w, "packed": _pack(w), "gamma": slot, "n": n, "k": k, "gain": gain,
            "bias": torch.randn(n, generator=g, device="cuda") * 0.1 if bias else None}


def _gain(g, k, want):
    return 1.0 + 0.2 * torch.randn(k, generator=g, device="cuda") if want else None


def _acts(g, m, k, dtype):
    """Activations N(0, 1) with 0.1 % of them 20 times larger, as residual streams have them."""
    x = torch.randn(m, k, generator=g, device="cuda")
    x = torch.where(torch.rand(m, k, generator=g, device="cuda") < 0.001, 20 * x, x)
    return x.to(DTYPES[dtype])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, m, op = case["dtype"], case["m"], case["op"]
    s = {"case": case, "op": op, "way": case["way"], "m": m}
    if op == "linear":
        k, n = case["k"], case["n"]
        gain = _gain(g, k, case["gain"])
        s["layers"] = [_layer(g, n, k, 0.02, gain, case["bias"], dt) for _ in range(case["layers"])]
        s["x"] = _acts(g, m, k, dt)
        s["dy"] = (torch.randn(m, case["layers"], n, generator=g, device="cuda") * 1e-3).to(DTYPES[dt])
        s["kept"] = _codes(s["x"], gain) if case["way"] == "backward" else None
    elif op == "glu":
        d, i = case["d"], case["inner"]
        gain, gain_p = _gain(g, d, case["gain"]), _gain(g, i, case["gain"])
        s["gate"], s["up"] = (_layer(g, i, d, 0.02, gain, case["bias"], dt) for _ in range(2))
        s["down"] = _layer(g, d, i, 0.02, gain_p, case["bias"], dt)
        s["x"] = _acts(g, m, d, dt)
        s["dy"] = (torch.randn(m, d, generator=g, device="cuda") * 1e-3).to(DTYPES[dt])
        if case["way"] == "backward":
            kx = _codes(s["x"], gain)
            u, v = _product(kx, s["gate"]), _product(kx, s["up"])
            s["kept"] = (kx, _codes((u * torch.sigmoid(u) * v).to(DTYPES[dt]), gain_p))
    else:
        k, v = case["k"], case["v"]
        s["head"] = _layer(g, v, k, 0.1, _gain(g, k, case["gain"]), case["bias"], dt)
        s["x"] = _acts(g, m, k, dt)
        labels = torch.randint(0, v, (m,), generator=g, device="cuda", dtype=torch.int32)
        drop = torch.rand(m, generator=g, device="cuda") < case["ignored"]
        s["labels"] = torch.where(drop, IGNORE, labels)
        none = case["reduction"] == "none"
        s["dloss"] = torch.rand(m if none else 1, generator=g, device="cuda") + 0.5
    return s


# ---------------------------------------------------------------- plain forms

def _codes(x, gain):
    """RMSNorm and absmax int8 codes of each row, every fp32 step rounded once: (q, scale, code sum, 1 / rms)."""
    f = x.float()
    ms = (f.double().square().sum(-1, keepdim=True) / x.shape[-1]).float()
    rinv = torch.ones_like(ms) / torch.sqrt(ms + EPS)
    xh = f * rinv
    xh = xh if gain is None else xh * gain
    top = xh.abs().amax(-1, keepdim=True).clamp_min(1e-5)
    scale = torch.full_like(top, 127.0) / top
    q = torch.clamp(torch.round(xh * scale), -128, 127)
    return (q.to(torch.int8), scale.squeeze(-1), q.sum(-1).to(torch.int32), rinv.squeeze(-1))


def _product(kept, layer):
    """gamma (q . w) / s + bias in fp32; the integer sum is exact."""
    acc = kept[0].float() @ layer["w"].float().t()
    y = acc * layer["gamma"][0] / kept[1][:, None]
    return y if layer["bias"] is None else y + layer["bias"]


def _norm_back(dxh, kept, gain, x):
    """Gradients of the norm's input and gain from that of its output; x is read from the codes when not kept."""
    q, scale, _, rinv = kept
    xt = q.float() / scale[:, None]
    one = torch.ones_like(dxh[0]) if gain is None else gain
    if x is None:
        n = torch.where(one == 0, torch.zeros_like(xt), xt / one)
        c = (dxh * xt).mean(-1, keepdim=True)
    else:
        n = x.float() * rinv[:, None]
        c = (dxh * n * one).mean(-1, keepdim=True)
    return rinv[:, None] * (one * dxh - n * c), (None if gain is None else (dxh * n).sum(0))


def _linear_back(layers, kept, dy, x):
    """dy [M, layers, N] -> input, per-layer weight, gain and per-layer bias gradients in fp32."""
    xt = kept[0].float() / kept[1][:, None]
    dys = [dy[:, i].float() for i in range(len(layers))]
    dxh = sum(g @ (l["w"].float() * l["gamma"][0]) for g, l in zip(dys, layers))
    dx, dgain = _norm_back(dxh, kept, layers[0]["gain"], x)
    return dx, [g.t() @ xt for g in dys], dgain, [None if l["bias"] is None else g.sum(0) for g, l in zip(dys, layers)]


def _cast(v, dt):
    if isinstance(v, (list, tuple)):
        return [_cast(x, dt) for x in v]
    return None if v is None else v.to(dt)


def _plain_linear(s):
    dt, layers = s["x"].dtype, s["layers"]
    out, kept = {}, s["kept"]
    if s["way"] == "step":
        kept = _codes(s["x"], layers[0]["gain"])
        out["y"] = torch.stack([_product(kept, l) for l in layers], 1).to(dt)
    x = s["x"] if s["case"]["keep_x"] else None
    dx, dw, dgain, dbias = _linear_back(layers, kept, s["dy"], x)
    return dict(out, dx=_cast(dx, dt), dw=_cast(dw, dt), dgain=_cast(dgain, dt), dbias=_cast(dbias, dt))


def _plain_glu(s):
    dt, gate, up, down = s["x"].dtype, s["gate"], s["up"], s["down"]
    out = {}
    kx, kp = s["kept"] if s["way"] == "backward" else (_codes(s["x"], gate["gain"]), None)
    u, v = _product(kx, gate), _product(kx, up)
    sig = torch.sigmoid(u)
    if kp is None:
        kp = _codes((u * sig * v).to(dt), down["gain"])     # the product is stored in the run's type
        out["y"] = _product(kp, down).to(dt)
    dp, (ddown,), dgain_down, (dbias_down,) = _linear_back([down], kp, s["dy"][:, None], None)
    du, dv = dp * v * sig * (1 + u * (1 - sig)), dp * u * sig
    dx, (dgate, dup), dgain, dbias = _linear_back([gate, up], kx, torch.stack([du, dv], 1), None)
    return dict(out, dx=_cast(dx, dt), dw=_cast([dgate, dup, ddown], dt), dgain=_cast([dgain, dgain_down], dt),
                dbias=_cast(dbias + [dbias_down], dt))


def _plain_loss(s):
    dt, head, labels = s["x"].dtype, s["head"], s["labels"]
    kept = _codes(s["x"], head["gain"])
    z = _product(kept, head)
    lse = torch.log(torch.exp(z - z.amax(-1, keepdim=True)).sum(-1)) + z.amax(-1)
    rows = torch.arange(s["m"], device=z.device)
    counted = labels != IGNORE
    at = torch.where(counted, labels, 0).long()
    token = torch.where(counted, lse - z[rows, at], 0.0)
    how = s["case"]["reduction"]
    count = counted.sum().clamp_min(1).float() if how == "mean" else torch.ones_like(lse[0])
    out = {"loss": token if how == "none" else token.double().sum().float() / count}
    if s["way"] == "step":
        weight = torch.where(counted, s["dloss"] / count, 0.0)
        dz = torch.exp(z - lse[:, None])
        dz[rows, at] -= 1
        dx, (dw,), dgain, (dbias,) = _linear_back([head], kept, (dz * weight[:, None])[:, None], None)
        out |= dict(dx=_cast(dx, dt), dw=_cast(dw, dt), dgain=_cast(dgain, dt), dbias=_cast(dbias, dt))
    return out


# ---------------------------------------------------------------- the library's calls

def _own_layer(mmf, l):
    return mmf.TLinear(l["packed"], l["gamma"], l["n"], l["k"], l["gain"], l["bias"])


def _own_linear(s):
    import ternary_weight_matmul_fusedbitlinear_b200 as mmf
    lins = [_own_layer(mmf, l) for l in s["layers"]]
    out = {}
    if s["way"] == "step":
        out["y"], kept = mmf.bitlinear_train(lins, s["x"], EPS)
    else:
        kept = mmf.Act8(*s["kept"])
    g = mmf.bitlinear_backward(lins, kept, s["dy"], x=s["x"] if s["case"]["keep_x"] else None)
    return dict(out, dx=g.dx, dw=g.dw, dgain=g.dgain, dbias=g.dbias)


def _own_glu(s):
    import ternary_weight_matmul_fusedbitlinear_b200 as mmf
    gate, up, down = (_own_layer(mmf, s[n]) for n in ("gate", "up", "down"))
    out = {}
    if s["way"] == "step":
        out["y"], kept = mmf.glu_train(gate, up, down, s["x"], eps=EPS)
    else:
        kept = mmf.Act8(*s["kept"][0]), mmf.Act8(*s["kept"][1])
    g = mmf.glu_backward(gate, up, down, kept, s["dy"])
    return dict(out, dx=g.dx, dw=g.dw, dgain=g.dgain, dbias=g.dbias)


def _own_loss(s):
    import ternary_weight_matmul_fusedbitlinear_b200 as mmf
    head, how = _own_layer(mmf, s["head"]), s["case"]["reduction"]
    loss, kept = mmf.head_loss(head, s["x"], s["labels"], ignore_index=IGNORE, reduction=how, eps=EPS)
    if s["way"] == "forward":
        return {"loss": loss}
    g = mmf.head_loss_backward(head, kept, s["labels"], s["dloss"], ignore_index=IGNORE, reduction=how)
    return {"loss": loss, "dx": g.dx, "dw": g.dw[0], "dgain": g.dgain, "dbias": g.dbias[0]}


def run(state):
    if own:
        return {"linear": _own_linear, "glu": _own_glu, "loss": _own_loss}[state["op"]](state)
    return {"linear": _plain_linear, "glu": _plain_glu, "loss": _plain_loss}[state["op"]](state)


# ---------------------------------------------------------------- the definition in 64 bits

class _Row8:
    """Codes of each row, decided by the definition's fp32 steps (numpy), and what stands for them in fp64."""

    def __init__(self, x, gain):
        a = x.float().cpu().numpy()
        ms = ((a.astype(np.float64) ** 2).sum(1, keepdims=True) / a.shape[1]).astype(np.float32)
        self._set(np.float32(1) / np.sqrt(ms + np.float32(EPS)), a, gain)

    def _set(self, rinv, a, gain):
        h = a * rinv
        if gain is not None:
            h = h * gain.cpu().numpy()[None]
        s = np.float32(127) / np.maximum(np.abs(h).max(1, keepdims=True), np.float32(1e-5))
        self.from_arrays(np.rint(h * s), s, rinv)

    def from_arrays(self, q, s, rinv):
        up = lambda v: torch.from_numpy(np.ascontiguousarray(v)).cuda().double()
        self.q, self.s, self.rinv = up(q), up(s), up(rinv)
        self.back = self.q / self.s
        return self

    @classmethod
    def kept(cls, k):
        me = cls.__new__(cls)
        return me.from_arrays(k[0].cpu().numpy().astype(np.float32), k[1].cpu().numpy()[:, None],
                              k[3].cpu().numpy()[:, None])

    def through(self, l):
        y = torch.einsum("mk,nk->mn", self.back, l["w"].double()).mul_(l["gamma"][0].double())
        return y if l["bias"] is None else y.add_(l["bias"].double())

    def gradients(self, pairs, gain, x):
        """pairs: (layer, upstream gradient [M, N] fp64)."""
        up = 0
        for l, g in pairs:
            up = up + torch.einsum("mn,nk->mk", g, l["w"].double()) * l["gamma"][0].double()
        dws = [torch.einsum("mn,mk->nk", g, self.back) for _, g in pairs]
        gd = torch.ones(self.q.shape[1], dtype=torch.float64, device="cuda") if gain is None else gain.double()
        if x is None:
            n = torch.where(gd == 0, torch.zeros_like(self.back), self.back / gd)
            inner = torch.einsum("mk,mk->m", up, self.back)
        else:
            n = x.double() * self.rinv
            inner = torch.einsum("mk,mk,k->m", up, n, gd)
        dx = (up * gd - n * (inner / up.shape[1])[:, None]) * self.rinv
        dgain = None if gain is None else torch.einsum("mk,mk->k", up, n)
        return dx, dws, dgain, [None if l["bias"] is None else g.sum(0) for l, g in pairs]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        ls = s["layers"]
        r = _Row8.kept(s["kept"]) if case["way"] == "backward" else _Row8(s["x"], ls[0]["gain"])
        out = {"y": torch.stack([r.through(l) for l in ls], 1)} if case["way"] == "step" else {}
        dx, dws, dgain, db = r.gradients([(l, s["dy"][:, i].double()) for i, l in enumerate(ls)], ls[0]["gain"],
                                         s["x"] if case["keep_x"] else None)
        return dict(out, dx=dx, dw=dws, dgain=dgain, dbias=db)
    if case["op"] == "glu":
        rx = _Row8.kept(s["kept"][0]) if case["way"] == "backward" else _Row8(s["x"], s["gate"]["gain"])
        u, v = rx.through(s["gate"]), rx.through(s["up"])
        sg = 1 / (1 + torch.exp(-u))
        out = {}
        if case["way"] == "backward":
            rp = _Row8.kept(s["kept"][1])
        else:
            rp = _Row8((u * sg * v).to(DTYPES[case["dtype"]]), s["down"]["gain"])
            out["y"] = rp.through(s["down"])
        dp, dwd, dgp, dbd = rp.gradients([(s["down"], s["dy"].double())], s["down"]["gain"], None)
        dv = dp * u * sg
        du = dp.mul_(v).mul_(sg + u * sg * (1 - sg))
        dx, dws, dg, db = rx.gradients([(s["gate"], du), (s["up"], dv)], s["gate"]["gain"], None)
        return dict(out, dx=dx, dw=dws + dwd, dgain=[dg, dgp], dbias=db + dbd)
    r = _Row8(s["x"], s["head"]["gain"])
    z = r.through(s["head"])
    lab = s["labels"].long()
    on = lab >= 0
    lse = torch.logsumexp(z, 1)
    row = torch.nonzero(on).squeeze(1)
    per = torch.zeros_like(lse)
    per[row] = lse[row] - z[row, lab[row]]
    n = max(1, int(on.sum())) if case["reduction"] == "mean" else 1
    out = {"loss": per if case["reduction"] == "none" else per.sum() / n}
    if case["way"] == "step":
        soft = z.sub_(lse[:, None]).exp_()
        soft[row, lab[row]] -= 1.0
        soft.mul_((on.double() * s["dloss"].double() / n)[:, None])
        dx, dws, dg, db = r.gradients([(s["head"], soft)], s["head"]["gain"], None)
        out |= dict(dx=dx, dw=dws[0], dgain=dg, dbias=db[0])
    return out
