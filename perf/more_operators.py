"""Operators at the edges of a trained MoE layer: what is measured, in plain form and as calls of
the library.

  combine     gradient of the combine: the expert rows' gradients and the slot weights'
  dispatch    gradient of the dispatch: token rows from the permuted rows' gradients
  residual    a block's branch joined to the residual stream -- norm of the branch, gates, residual
              scale -- and the next block's norm of the result, forward and backward
  ortho       momentum and the orthogonalised update of a batch of weight matrices by
              Newton-Schulz products

`run` computes a case in plain torch operations (32-bit), or, where `own` is true, through the
library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32
EPS_POST, EPS_PRE = 1e-6, 1e-5
STEPS, COEFFS = 5, (3.4445, -4.7750, 2.0315)


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the test-sized layer, an unaligned token count: latency
        dict(name="combine_small", op="combine", T=45, H=256, E=16, K=2, dy="f32", drop=0.0, skew=0.0),
        # odd widths, a skewed load, pairs that an expert's capacity rejected (no row)
        dict(name="combine_ragged", op="combine", T=1777, H=2112, E=24, K=3, dy="bf16", drop=0.1, skew=1.0),
        # a training batch at full width: the gradient of the combine's fp32 output
        dict(name="combine_batch", op="combine", T=16384, H=7168, E=256, K=8, dy="f32", drop=0.0, skew=0.5),
        # fine-tuning on a decode-sized batch
        dict(name="dispatch_decode", op="dispatch", T=128, H=7168, E=256, K=8, dx="f32", res=False, drop=0.0, skew=0.0),
        # a training batch, the shared expert's gradient added in
        dict(name="dispatch_batch", op="dispatch", T=16384, H=7168, E=256, K=8, dx="bf16", res=True, drop=0.0, skew=0.5),
        # a decode batch between two blocks: bf16 stream, RMS norm in front of the next one
        dict(name="residual_forward_decode", op="residual", dir="forward", T=128, H=7168, x="bf16", y="f32", post="none",
             pre="rms", alpha=1.0, gate=False, gate_token=False, dr=True),
        # a training batch: norms on both sides, a gate a channel, an fp32 stream
        dict(name="residual_forward_batch", op="residual", dir="forward", T=16384, H=7168, x="f32", y="f32", post="rms",
             pre="layer", alpha=0.9, gate=True, gate_token=False, dr=True),
        # the test-sized block's backward pass, gates of both kinds
        dict(name="residual_backward_small", op="residual", dir="backward", T=45, H=256, x="bf16", y="bf16", post="layer",
             pre="rms", alpha=1.0, gate=True, gate_token=True, dr=True),
        # a training batch's backward pass
        dict(name="residual_backward_batch", op="residual", dir="backward", T=16384, H=7168, x="f32", y="f32", post="rms",
             pre="layer", alpha=0.9, gate=True, gate_token=False, dr=True),
        # the test-sized layer's 16 experts, one projection: latency
        dict(name="ortho_small", op="ortho", B=16, R=256, C=128, g="bf16", momentum=False, nesterov=False),
        # ragged widths, fp32 gradients with momentum
        dict(name="ortho_ragged", op="ortho", B=24, R=2112, C=1088, g="f32", momentum=True, nesterov=True),
        # half of a 32-expert layer's up projections at full width, as a step of the optimiser takes them
        dict(name="ortho_experts", op="ortho", B=16, R=7168, C=2048, g="bf16", momentum=True, nesterov=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["combine", "dispatch", "residual", "ortho"])
    if op in ("combine", "dispatch"):
        H = 64 * _log(rng, 1, 128)
        E = _log(rng, 1, 512)
        K = rng.randint(1, min(16, E))
        c = dict(op=op, T=_log(rng, 1, max(1, min(16384, 16384 * 7168 * 8 // (H * K)))), H=H, E=E, K=K,
                 drop=rng.choice([0.0, 0.0, 0.1]), skew=rng.choice([0.0, 0.5, 1.0]))
        if op == "combine":
            return dict(c, dy=rng.choice(["f32", "bf16"]))
        return dict(c, dx=rng.choice(["f32", "bf16"]), res=rng.random() < 0.5)
    if op == "residual":
        H = 64 * _log(rng, 1, 128)
        post, pre = rng.choice(["none", "layer", "rms"]), rng.choice(["none", "layer", "rms", "rms"])
        return dict(op=op, dir=rng.choice(["forward", "backward"]), T=_log(rng, 1, min(16384, 16384 * 7168 // H)), H=H,
                    x=rng.choice(["f32", "bf16"]), y=rng.choice(["f32", "bf16"]), post=post, pre=pre,
                    alpha=rng.choice([1.0, 0.9]), gate=rng.random() < 0.5, gate_token=rng.random() < 0.4,
                    dr=pre == "none" or rng.random() < 0.7)
    B, R, C = _log(rng, 1, 32), _log(rng, 1, 7168), _log(rng, 1, 7168)
    # no dearer than the largest listed one
    while _products(B, R, C) > _products(16, 7168, 2048):
        B, R, C = (B // 2, R, C) if B > 1 else (B, R * 3 // 4, C * 3 // 4)
    momentum = rng.random() < 0.5
    return dict(op=op, B=B, R=R, C=C, g=rng.choice(["f32", "bf16"]), momentum=momentum,
                nesterov=momentum and rng.random() < 0.5)


def _products(B, R, C):
    """Operations of the products: X X^T and its square are symmetric, half of each is enough."""
    m, n = min(R, C), max(R, C)
    return B * STEPS * (float(m) * m * n + float(m) * m * m + 2.0 * m * m * n)


# ----------------------------------------------------------------------------------- inputs
def _dtype(name):
    return F32 if name == "f32" else BF16


def _tensor(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=F32)


def _slots(g, c):
    """slot_pos [T, K] as the dispatch leaves it: rows ordered by (expert, token); -1 where a pair
    has no row."""
    T, E, K = c["T"], c["E"], c["K"]
    pull = -c["skew"] * torch.log1p(torch.arange(E, device=DEV, dtype=F32))
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=DEV).clamp(1e-9, 1 - 1e-7)))
    expert = (pull + noise).topk(K, dim=1).indices.reshape(-1)
    lost = torch.rand(T * K, generator=g, device=DEV) < c["drop"]
    order = torch.sort(torch.where(lost, torch.full_like(expert, E), expert), stable=True).indices
    slot = torch.empty_like(order)
    slot[order] = torch.arange(T * K, device=DEV)
    return torch.where(lost, torch.full_like(slot, -1), slot).view(T, K).to(I32)


def _gradient(g, B, R, C):
    """Matrices such as a batch's gradients are: a spectrum that falls off, and noise."""
    r = max(1, min(R, C, 1024) // 2)
    fall = torch.arange(1, r + 1, device=DEV, dtype=F32) ** -0.5
    low = (_tensor(g, B, R, r) * fall) @ _tensor(g, B, r, C)
    return 1e-3 * (low + 0.3 * _tensor(g, B, R, C))


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = dict(case)
    s = dict(case=c)
    if c["op"] in ("combine", "dispatch"):
        T, H, K = c["T"], c["H"], c["K"]
        s["slot_pos"] = _slots(g, c)
        if c["op"] == "combine":
            s["Yp"] = torch.empty(T * K, H, device=DEV, dtype=BF16).normal_(0.0, 0.5, generator=g)
            w = torch.rand(T, K, generator=g, device=DEV) + 0.1
            s["topk_w"] = w / w.sum(1, keepdim=True)
            s["dY"] = (1e-2 * _tensor(g, T, H)).to(_dtype(c["dy"]))
        else:
            s["dXp"] = torch.empty(T * K, H, device=DEV, dtype=BF16).normal_(0.0, 1e-2, generator=g)
            s["dres"] = (1e-2 * _tensor(g, T, H)).to(_dtype(c["dx"])) if c["res"] else None
    elif c["op"] == "residual":
        T, H = c["T"], c["H"]
        # a stream whose rows differ in size, with a common offset on some columns, and a branch
        s["x"] = (_tensor(g, T, H) * (0.5 + 2 * torch.rand(T, 1, generator=g, device=DEV)) + 0.3 * _tensor(g, 1, H)).to(_dtype(c["x"]))
        s["y"] = (_tensor(g, T, H) * (0.2 + torch.rand(T, 1, generator=g, device=DEV)) + 0.1 * _tensor(g, 1, H)).to(_dtype(c["y"]))
        s["p"] = dict(post=c["post"], pre=c["pre"], alpha=c["alpha"], eps_post=EPS_POST, eps_pre=EPS_PRE)
        for end in ("post", "pre"):
            if c[end] != "none":
                s["p"]["gamma_" + end] = 1 + 0.1 * _tensor(g, H)
            if c[end] == "layer":
                s["p"]["beta_" + end] = 0.1 * _tensor(g, H)
        if c["gate"]:
            s["p"]["gate"] = 0.5 + 0.2 * _tensor(g, H)
        if c["gate_token"]:
            s["p"]["gate_token"] = torch.rand(T, generator=g, device=DEV)
        if c["dir"] == "backward":
            s["dn"] = (1e-2 * _tensor(g, T, H)).to(BF16) if c["pre"] != "none" else None
            s["dr"] = (1e-2 * _tensor(g, T, H)).to(_dtype(c["x"])) if c["dr"] else None
            s["r"], _, s["stats"] = _join(s["x"], s["y"], s["p"])
            del s["x"]
    else:
        B, R, C = c["B"], c["R"], c["C"]
        s["g"] = _gradient(g, B, R, C).to(_dtype(c["g"]))
        s["m"] = 4 * _gradient(g, B, R, C) if c["momentum"] else None
    return s


# ------------------------------------------------------------------------------ plain forms
def _combine(s):
    slot = s["slot_pos"].long()
    live = (slot >= 0).to(F32)[..., None]
    dY = s["dY"].to(F32)[:, None, :]
    at = slot.clamp(min=0)
    d_topk_w = (s["Yp"][at].to(F32) * live * dY).sum(-1)
    rows = (s["topk_w"][..., None] * dY).to(BF16)
    dYp = torch.zeros_like(s["Yp"])
    # pairs without a row are written behind the last one, which is cut off
    n = dYp.shape[0]
    dYp = torch.cat([dYp, dYp[:1]])
    dYp[torch.where(slot >= 0, slot, torch.full_like(slot, n)).reshape(-1)] = rows.view(-1, rows.shape[-1])
    return dict(dYp=dYp[:n], d_topk_w=d_topk_w)


def _dispatch(s):
    slot = s["slot_pos"].long()
    dX = (s["dXp"][slot.clamp(min=0)].to(F32) * (slot >= 0).to(F32)[..., None]).sum(1)
    if s["dres"] is not None:
        dX = dX + s["dres"].to(F32)
    return dict(dX=dX.to(_dtype(s["case"]["dx"])))


def _statistics(v, kind, eps):
    if kind == "none":
        return torch.zeros_like(v[:, 0]), torch.ones_like(v[:, 0])
    mean = v.mean(1) if kind == "layer" else torch.zeros_like(v[:, 0])
    return mean, 1 / torch.sqrt((v - mean[:, None]).square().mean(1) + eps)


def _affine(v, p, end):
    if p[end] == "none":
        return v
    v = v * p["gamma_" + end]
    return v + p["beta_" + end] if p.get("beta_" + end) is not None else v


def _join(x, y, p):
    """-> r in x's type, the norm of r in bf16 (or None), the statistics [T, 4]"""
    y = y.to(F32)
    mean_y, rstd_y = _statistics(y, p["post"], p["eps_post"])
    b = _affine((y - mean_y[:, None]) * rstd_y[:, None], p, "post")
    if p.get("gate") is not None:
        b = b * p["gate"]
    if p.get("gate_token") is not None:
        b = b * p["gate_token"][:, None]
    r = (p["alpha"] * x.to(F32) + b).to(x.dtype)
    v = r.to(F32)
    mean_r, rstd_r = _statistics(v, p["pre"], p["eps_pre"])
    n = None
    if p["pre"] != "none":
        n = _affine((v - mean_r[:, None]) * rstd_r[:, None], p, "pre").to(BF16)
    return r, n, torch.stack([mean_y, rstd_y, mean_r, rstd_r], 1)


def _through(d, v, rstd, kind):
    """Gradient of a norm's input from that of its normalised rows v."""
    if kind == "none":
        return d
    out = d - v * (d * v).mean(1, keepdim=True)
    if kind == "layer":
        out = out - d.mean(1, keepdim=True)
    return out * rstd[:, None]


def _residual(s):
    p = s["p"]
    if s["case"]["dir"] == "forward":
        r, n, stats = _join(s["x"], s["y"], p)
        return dict(r=r, n=n, stats=stats)
    y, r = s["y"].to(F32), s["r"].to(F32)
    mean_y, rstd_y, mean_r, rstd_r = s["stats"].unbind(1)
    o = {}
    d = torch.zeros_like(r) if s["dr"] is None else s["dr"].to(F32)
    if p["pre"] != "none":
        dn, v = s["dn"].to(F32), (r - mean_r[:, None]) * rstd_r[:, None]
        o["gamma_pre"], o["beta_pre"] = (dn * v).sum(0), dn.sum(0)
        d = d + _through(dn * p["gamma_pre"], v, rstd_r, p["pre"])
    v = (y - mean_y[:, None]) * rstd_y[:, None]
    b = _affine(v, p, "post")
    db = d
    if p.get("gate_token") is not None:
        o["gate_token"] = (d * b * (p["gate"] if p.get("gate") is not None else 1.0)).sum(1)
        db = db * p["gate_token"][:, None]
    if p.get("gate") is not None:
        o["gate"] = (db * b).sum(0)
        db = db * p["gate"]
    if p["post"] != "none":
        o["gamma_post"], o["beta_post"] = (db * v).sum(0), db.sum(0)
        db = _through(db * p["gamma_post"], v, rstd_y, p["post"])
    o = {k: t for k, t in o.items() if p.get(k) is not None}
    return dict(dx=(p["alpha"] * d).to(s["r"].dtype), dy=db.to(BF16), **o)


def _ortho(s):
    c, u = s["case"], s["g"].to(F32)
    o = {}
    if s["m"] is not None:
        mu = 0.95
        s["m"].mul_(mu).add_(u)
        u = u + mu * s["m"] if c["nesterov"] else s["m"]
        o["momentum"] = s["m"]
    x = u.transpose(1, 2) if c["R"] > c["C"] else u
    norm = x.square().sum((1, 2), keepdim=True).sqrt()
    x = x / torch.where(norm > 0, norm, torch.ones_like(norm))
    a, b, k = COEFFS
    for _ in range(STEPS):
        A = x @ x.transpose(1, 2)
        x = a * x + (b * A + k * (A @ A)) @ x
    x = x.transpose(1, 2) if c["R"] > c["C"] else x
    return dict(out=x.to(BF16).contiguous(), **o)


# ------------------------------------------------------------------------- the library's calls
def _buffers(s):
    """Outputs and workspace, which a training loop keeps from step to step."""
    if "out" in s:
        return s["out"], s["ws"]
    from expert_routed_ffn_router_gb300 import binding as B
    c, n = s["case"], 0

    def new(*shape, dtype=F32):
        return torch.empty(*shape, dtype=dtype, device=DEV)
    if c["op"] == "combine":
        o = dict(dYp=torch.zeros_like(s["Yp"]), d_topk_w=new(c["T"], c["K"]))
    elif c["op"] == "dispatch":
        o = dict(dX=new(c["T"], c["H"], dtype=_dtype(c["dx"])))
    elif c["op"] == "residual" and c["dir"] == "forward":
        o = dict(r=torch.empty_like(s["x"]), n=new(c["T"], c["H"], dtype=BF16) if c["pre"] != "none" else None,
                 stats=new(c["T"], 4))
    elif c["op"] == "residual":
        s["grads"] = {k: torch.empty_like(v) for k, v in s["p"].items() if torch.is_tensor(v)}
        o = dict(dx=torch.empty_like(s["r"]), dy=new(c["T"], c["H"], dtype=BF16), **s["grads"])
        n = B.moe_residual_norm_backward_workspace_bytes(c["T"], c["H"])
    else:
        o = dict(out=new(c["B"], c["R"], c["C"], dtype=BF16))
        if c["momentum"]:
            o["momentum"] = s["m"]
        n = B.moe_orthogonalize_workspace_bytes(c["B"], c["R"], c["C"])
    s["out"], s["ws"] = o, torch.zeros(max(n, 256), dtype=torch.uint8, device=DEV)
    return s["out"], s["ws"]


def _own(s):
    from expert_routed_ffn_router_gb300 import binding as B
    c = s["case"]
    o, ws = _buffers(s)
    if c["op"] == "combine":
        B.moe_combine_backward(s["dY"], s["Yp"], s["slot_pos"], s["topk_w"], o["dYp"], o["d_topk_w"])
    elif c["op"] == "dispatch":
        B.moe_dispatch_backward(s["dXp"], s["slot_pos"], s["dres"], o["dX"])
    elif c["op"] == "residual" and c["dir"] == "forward":
        B.moe_residual_norm(s["x"], s["y"], s["p"], o["r"], o["n"], o["stats"])
    elif c["op"] == "residual":
        B.moe_residual_norm_backward(s["dn"], s["dr"], s["y"], s["r"], s["stats"], s["p"], o["dx"], o["dy"], s["grads"], ws)
    else:
        B.moe_orthogonalize(s["g"], o["out"], ws, momentum=s["m"], mu=0.95, nesterov=c["nesterov"], steps=STEPS)
    return o


def run(state):
    if own:
        return _own(state)
    return {"combine": _combine, "dispatch": _dispatch, "residual": _residual, "ortho": _ortho}[state["case"]["op"]](state)


# ------------------------------------------------------------------------- bytes and products
def work(case):
    c = case
    size = {"f32": 4, "bf16": 2}
    if c["op"] in ("combine", "dispatch"):
        T, H, K = c["T"], c["H"], c["K"]
        rows = T * K * (1 - c["drop"]) * H
        if c["op"] == "combine":
            return dict(bytes=4 * rows + T * H * size[c["dy"]] + 12 * T * K, flops=3 * rows)
        return dict(bytes=2 * rows + T * H * size[c["dx"]] * (2 if c["res"] else 1) + 4 * T * K, flops=rows)
    if c["op"] == "residual":
        T, H, x, y = c["T"], c["H"], size[c["x"]], size[c["y"]]
        pre = c["pre"] != "none"
        small = sum((c["post"] != "none", c["post"] == "layer", pre, c["pre"] == "layer", c["gate"])) * 4 * H
        token = 16 * T + (4 * T if c["gate_token"] else 0)
        if c["dir"] == "forward":
            return dict(bytes=T * H * (2 * x + y + (2 if pre else 0)) + small + token, flops=16 * T * H)
        # the branch is not read where nothing depends on it
        branch = y if c["post"] != "none" or c["gate"] or c["gate_token"] else 0
        read = branch + ((2 + x) if pre else 0) + (x if c["dr"] else 0)
        return dict(bytes=T * H * (read + x + 2) + 2 * small + 2 * token, flops=30 * T * H)
    n = c["B"] * c["R"] * c["C"]
    return dict(bytes=n * (size[c["g"]] + 2 + (8 if c["momentum"] else 0)), flops=_products(c["B"], c["R"], c["C"]))


# ------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    F64 = torch.float64
    if c["op"] == "combine":
        # slot by slot: a pair's row and its weight's gradient
        dY = s["dY"].to(F64)
        dYp = torch.zeros(s["Yp"].shape, dtype=F64, device=DEV)
        dw = torch.zeros(c["T"], c["K"], dtype=F64, device=DEV)
        for j in range(c["K"]):
            t = (s["slot_pos"][:, j] >= 0).nonzero().squeeze(1)
            at = s["slot_pos"][t, j].long()
            dYp[at] = dY[t] * s["topk_w"][t, j].to(F64)[:, None]
            dw[t, j] = torch.einsum("th,th->t", dY[t], s["Yp"][at].to(F64))
        return dict(dYp=dYp, d_topk_w=dw)
    if c["op"] == "dispatch":
        dX = torch.zeros(c["T"], c["H"], dtype=F64, device=DEV) if s["dres"] is None else s["dres"].to(F64)
        for j in range(c["K"]):
            t = (s["slot_pos"][:, j] >= 0).nonzero().squeeze(1)
            dX.index_add_(0, t, s["dXp"][s["slot_pos"][t, j].long()].to(F64))
        return dict(dX=dX)
    if c["op"] == "residual":
        p = {k: v.to(F64) if torch.is_tensor(v) else v for k, v in s["p"].items()}

        def norm(v, end):
            kind = c[end]
            if kind == "none":
                return v, torch.zeros(c["T"], dtype=F64, device=DEV), torch.ones(c["T"], dtype=F64, device=DEV)
            mean = v.sum(1) / c["H"] if kind == "layer" else torch.zeros(c["T"], dtype=F64, device=DEV)
            rstd = (((v - mean[:, None]) ** 2).sum(1) / c["H"] + p["eps_" + end]) ** -0.5
            out = torch.einsum("th,t,h->th", v - mean[:, None], rstd, p["gamma_" + end])
            return (out + p["beta_" + end] if kind == "layer" else out), mean, rstd
        if c["dir"] == "forward":
            b, mean_y, rstd_y = norm(s["y"].to(F64), "post")
            scale = torch.ones(c["H"], dtype=F64, device=DEV) if p.get("gate") is None else p["gate"]
            token = torch.ones(c["T"], dtype=F64, device=DEV) if p.get("gate_token") is None else p["gate_token"]
            r = p["alpha"] * s["x"].to(F64) + torch.einsum("th,t,h->th", b, token, scale)
            # the next norm is that of the stream as it is stored
            n, mean_r, rstd_r = norm(r.to(s["x"].dtype).to(F64), "pre")
            return dict(r=r, n=None if c["pre"] == "none" else n, stats=torch.stack([mean_y, rstd_y, mean_r, rstd_r], 1))
        # the gradients, for the statistics that the caller hands over
        with torch.no_grad():
            T, H = c["T"], c["H"]
            mean_y, rstd_y, mean_r, rstd_r = (t[:, None] for t in s["stats"].to(F64).unbind(1))
            o = {}
            d = torch.zeros(T, H, dtype=F64, device=DEV)
            if s["dr"] is not None:
                d += s["dr"].to(F64)
            if c["pre"] != "none":
                dn, v = s["dn"].to(F64), s["r"].to(F64).sub(mean_r).mul_(rstd_r)
                o["gamma_pre"], o["beta_pre"] = torch.einsum("th,th->h", dn, v), torch.einsum("th->h", dn)
                e = torch.einsum("th,h->th", dn, p["gamma_pre"])
                t = e - torch.einsum("th,th->t", e, v)[:, None] / H * v
                if c["pre"] == "layer":
                    t -= e.sum(1, keepdim=True) / H
                d.addcmul_(t, rstd_r)
            v = s["y"].to(F64).sub(mean_y).mul_(rstd_y)
            b = v
            if c["post"] != "none":
                b = v * p["gamma_post"] + (p["beta_post"] if c["post"] == "layer" else 0.0)
            ones = torch.ones(H, dtype=F64, device=DEV)
            gh = p.get("gate") if p.get("gate") is not None else ones
            gt = p.get("gate_token") if p.get("gate_token") is not None else torch.ones(T, dtype=F64, device=DEV)
            o["gate"] = torch.einsum("th,th,t->h", d, b, gt)
            o["gate_token"] = torch.einsum("th,th,h->t", d, b, gh)
            db = torch.einsum("th,t,h->th", d, gt, gh)
            dy = db
            if c["post"] != "none":
                o["gamma_post"], o["beta_post"] = torch.einsum("th,th->h", db, v), torch.einsum("th->h", db)
                e = torch.einsum("th,h->th", db, p["gamma_post"])
                dy = e - torch.einsum("th,th->t", e, v)[:, None] / H * v
                if c["post"] == "layer":
                    dy -= e.sum(1, keepdim=True) / H
                dy *= rstd_y
            return dict(dx=p["alpha"] * d, dy=dy, **{k: t for k, t in o.items() if p.get(k) is not None})
    # matrix by matrix, on the side of the smaller dimension
    outs, moms = [], []
    for i in range(c["B"]):
        u = s["g"][i].to(F64)
        if c["momentum"]:
            m = 0.95 * s["m"][i].to(F64) + u
            u = u + 0.95 * m if c["nesterov"] else m
            moms.append(m)
        x = u / torch.linalg.vector_norm(u) if bool(u.any()) else u
        for _ in range(STEPS):
            A = x @ x.mT if c["R"] <= c["C"] else x.mT @ x
            P = COEFFS[1] * A + COEFFS[2] * (A @ A)
            P.diagonal().add_(COEFFS[0])
            x = P @ x if c["R"] <= c["C"] else x @ P
        outs.append(x)
    o = dict(out=torch.stack(outs))
    if c["momentum"]:
        o["momentum"] = torch.stack(moms)
    return o
