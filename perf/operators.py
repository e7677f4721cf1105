"""Training operators around the MoE layer: what is measured, in plain form and as calls of
the library.

Four operators of a pre-norm MoE block's training step:

  norm        layer norm of the token rows and its backward pass
  route       top-k routing from given gate logits and its backward pass
  checkpoint  token rows kept as E4M3 bytes with one power-of-two scale per 128 columns, and
              taken back
  experts     the expert FFN's backward pass from the (8-bit or bf16) token rows

`run` computes a case in plain torch operations (32-bit, the selection in 64-bit), or, where
`own` is true, through the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
BLOCK = 128                                     # columns that share a scale
MASKED = torch.finfo(BF16).min                  # a logit at or below it is masked out
EPS = 1e-5


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # latency of a decode batch's norm: 64 requests of 2 query tokens, bf16 stream
        dict(name="norm_forward_decode", op="norm", dir="forward", T=128, H=7168, x="bf16", res=False),
        # the smallest backward call: an unaligned token count on the test-sized layer
        dict(name="norm_backward_small", op="norm", dir="backward", T=45, H=256, x="f32", res=False),
        # a training batch with an fp32 residual stream, the residual's gradient added in
        dict(name="norm_backward_batch", op="norm", dir="backward", T=16384, H=7168, x="f32", res=True),
        # routing of two tokens (one request with one draft token), group-limited sigmoid
        dict(name="route_forward_two", op="route", dir="forward", T=2, E=256, K=8, l="f32", scoring="sigmoid",
             n_group=8, topk_group=4, group_top=2, renorm=True, bias=True),
        # a prefill or training batch through the same router
        dict(name="route_forward_batch", op="route", dir="forward", T=16384, E=256, K=8, l="f32", scoring="sigmoid",
             n_group=8, topk_group=4, group_top=2, renorm=True, bias=True),
        # a dense gradient: softmax over an odd number of experts, weights not renormalised
        dict(name="route_backward_softmax", op="route", dir="backward", T=8191, E=160, K=6, l="bf16", scoring="softmax",
             n_group=1, topk_group=1, group_top=1, renorm=False, bias=False),
        # the rows of a decode batch packed and taken back
        dict(name="checkpoint_decode", op="checkpoint", T=128, n=7168),
        # a training batch's rows
        dict(name="checkpoint_batch", op="checkpoint", T=16384, n=7168),
        # the test-sized layer's experts, rows kept in bf16: latency
        dict(name="experts_small", op="experts", T=16, H=256, E=16, K=2, I=128, packed=False, skew=0.0),
        # few rows per expert at full width: the weights' and gradients' bytes bound it
        dict(name="experts_few_rows", op="experts", T=32, H=7168, E=32, K=8, I=2048, packed=True, skew=0.0),
        # ragged groups, odd widths, a skewed expert load
        dict(name="experts_ragged", op="experts", T=1777, H=2112, E=24, K=3, I=1088, packed=True, skew=1.0),
        # a training batch at full width: bound by the tensor cores
        dict(name="experts_batch", op="experts", T=4096, H=7168, E=32, K=8, I=2048, packed=True, skew=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "checkpoint", "experts"])
    if op == "norm":
        H = 64 * _log(rng, 1, 128)
        T = _log(rng, 1, min(16384, 16384 * 7168 // H))
        d = rng.choice(["forward", "backward"])
        return dict(op=op, dir=d, T=T, H=H, x=rng.choice(["bf16", "f32"]), res=d == "backward" and rng.random() < 0.5)
    if op == "route":
        n_group = rng.choice([1, 1, 2, 4, 8])
        E = n_group * _log(rng, 4, 512 // n_group)
        topk_group = rng.randint(1, n_group)
        K = rng.randint(1, min(16, topk_group * (E // n_group)))
        return dict(op=op, dir=rng.choice(["forward", "backward"]), T=_log(rng, 1, min(16384, 16384 * 256 // E)), E=E, K=K,
                    l=rng.choice(["f32", "bf16"]), scoring=rng.choice(["sigmoid", "softmax"]), n_group=n_group,
                    topk_group=topk_group, group_top=rng.choice([1, 2]), renorm=rng.random() < 0.5,
                    bias=rng.random() < 0.5)
    if op == "checkpoint":
        n = 64 * _log(rng, 1, 128)
        return dict(op=op, T=_log(rng, 1, min(16384, 16384 * 7168 // n)), n=n)
    E = _log(rng, 1, 64)
    K = rng.randint(1, min(8, E))
    H, I = 64 * _log(rng, 1, 112), 64 * _log(rng, 1, 32)
    # no dearer than the batch listed above, in products and in the weights' bytes
    while E * H * I > 32 * 7168 * 2048:
        H, I = max(64, H // 128 * 64), max(64, I // 128 * 64)
    top = min(4096, 4096 * 8 * 7168 * 2048 // (K * H * I))
    return dict(op=op, T=_log(rng, 1, top), H=H, E=E, K=K, I=I, packed=rng.random() < 0.6,
                skew=rng.choice([0.0, 0.5, 1.0]))


# ----------------------------------------------------------------------------------- inputs
def _pack(x):
    """E4M3 values and power-of-two exponents of rows in blocks of 128 columns."""
    T, n = x.shape
    nb = -(-n // BLOCK)
    v = torch.nn.functional.pad(x.to(F32), (0, nb * BLOCK - n)).view(T, nb, BLOCK)
    amax = v.abs().amax(-1)
    m, e = torch.frexp(amax)                    # amax = m 2^e, and 448 = 0.875 * 2^9
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(-124, 127)
    k = torch.where(amax > 0, k, torch.zeros_like(k))
    q = torch.ldexp(v, -k.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.view(T, nb * BLOCK)[:, :n].contiguous(), k.to(torch.int8)


def _unpack(q, s):
    """The values that packed rows stand for (32-bit; exact in bf16)."""
    T, n = q.shape
    return torch.ldexp(q.to(F32), s.repeat_interleave(BLOCK, 1)[:, :n].to(torch.int32))


def _tensor(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=F32)


def _assign(g, T, E, K, skew):
    """K distinct experts a token; with skew > 0 some experts draw more tokens."""
    pull = -skew * torch.log1p(torch.arange(E, device=DEV, dtype=F32))
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=DEV).clamp(1e-9, 1 - 1e-7)))
    return (pull + noise).topk(K, dim=1).indices


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=dict(case))
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        dt = F32 if case["x"] == "f32" else BF16
        # a residual stream: rows of differing size, a common offset on some columns
        s["x"] = (_tensor(g, T, H) * (0.5 + 2 * torch.rand(T, 1, generator=g, device=DEV)) + 0.3 * _tensor(g, 1, H)).to(dt)
        s["gamma"] = 1 + 0.1 * _tensor(g, H)
        s["beta"] = 0.1 * _tensor(g, H)
        if case["dir"] == "backward":
            s["dy"] = (1e-2 * _tensor(g, T, H)).to(BF16)
            s["res"] = (1e-2 * _tensor(g, T, H)).to(dt) if case["res"] else None
            x = s["x"].to(F32)
            s["mean"] = x.mean(1)
            s["rstd"] = (x - s["mean"][:, None]).square().mean(1).add(EPS).rsqrt()
    elif case["op"] == "route":
        T, E, K = case["T"], case["E"], case["K"]
        dt = F32 if case["l"] == "f32" else BF16
        s["logits"] = (1.7 * _tensor(g, T, E)).to(dt)
        s["bias"] = 0.2 * torch.rand(E, generator=g, device=DEV) - 0.1 if case["bias"] else None
        if case["dir"] == "backward":
            s["idx"] = _choose(s["logits"], s["bias"], case).to(torch.int32)
            s["dw"] = 1e-2 * _tensor(g, T, K)
    elif case["op"] == "checkpoint":
        # the norm's output, as the layer reads it
        s["x"] = (_tensor(g, case["T"], case["n"]) * (0.5 + torch.rand(case["T"], 1, generator=g, device=DEV))).to(BF16)
    else:
        T, H, E, K, I = (case[k] for k in ("T", "H", "E", "K", "I"))
        x = _tensor(g, T, H).to(BF16)
        s["x"], s["x_scale"] = _pack(x) if case["packed"] else (x, None)
        if case["packed"]:
            s["x"] = s["x"].view(torch.uint8)
        s["dY"] = (1e-2 * _tensor(g, T, H)).to(BF16)
        for name, shape in (("W1", (E, H, I)), ("W3", (E, H, I)), ("W2", (E, I, H))):
            s[name] = torch.empty(shape, device=DEV, dtype=BF16).normal_(0.0, 0.02, generator=g)
        idx = _assign(g, T, E, K, case["skew"])
        w = torch.rand(T, K, generator=g, device=DEV) + 0.1
        s["topk_w"] = w / w.sum(1, keepdim=True)
        # the dispatch's bookkeeping: rows ordered by (expert, token)
        flat = idx.reshape(-1)
        order = torch.sort(flat, stable=True).indices
        slot = torch.empty_like(order)
        slot[order] = torch.arange(T * K, device=DEV)
        counts = torch.bincount(flat, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["slot_pos"] = slot.view(T, K).to(torch.int32)
        s["idx"] = idx.to(torch.int32)
        s["most"] = int(counts.max())           # rows of the busiest expert
    return s


# ------------------------------------------------------------------------------ plain forms
def _choose(logits, bias, c):
    """The selected experts, descending, equal values by index; in 64 bits."""
    l = logits.double()
    off = logits <= MASKED
    sc = torch.sigmoid(l) if c["scoring"] == "sigmoid" else torch.softmax(l, 1)
    sel = sc if bias is None else sc + bias.double()
    sel = torch.where(off, torch.full_like(sel, -1e300), sel)
    T, E = l.shape
    if c["n_group"] > 1:
        G = E // c["n_group"]
        per = sel.view(T, c["n_group"], G)
        score = per.sort(dim=-1, descending=True).values[..., :min(c["group_top"], G)].sum(-1)
        keep = score.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        kept = torch.zeros(T, c["n_group"], dtype=torch.bool, device=l.device).scatter_(1, keep, True)
        sel = torch.where(kept[:, :, None], per, torch.full_like(per, -math.inf)).view(T, E)
    return sel.sort(dim=1, descending=True, stable=True).indices[:, :c["K"]]


def _scores(logits, c):
    l = logits.to(F32)
    l = torch.where(logits <= MASKED, torch.full_like(l, -math.inf), l)
    if c["scoring"] == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _norm(s):
    c, x = s["case"], s["x"].to(F32)
    if c["dir"] == "forward":
        mean = x.mean(1)
        d = x - mean[:, None]
        rstd = 1 / torch.sqrt(d.square().mean(1) + EPS)
        return dict(y=(d * rstd[:, None] * s["gamma"] + s["beta"]).to(BF16), mean=mean, rstd=rstd)
    dy, r = s["dy"].to(F32), s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * r
    a = dy * s["gamma"]
    dx = r * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
    if s["res"] is not None:
        dx = dx + s["res"].to(F32)
    return dict(dx=dx.to(s["x"].dtype), dgamma=(dy * xh).sum(0), dbeta=dy.sum(0))


def _route(s):
    c, logits = s["case"], s["logits"]
    if c["dir"] == "forward":
        idx = _choose(logits, s["bias"], c)
        w = _scores(logits, c).gather(1, idx)
        if c["renorm"]:
            total = w.sum(1, keepdim=True)
            w = torch.where(total > 0, w / total, torch.zeros_like(w))
        return dict(topk_idx=idx.to(torch.int32), topk_w=w)
    idx, dw, sc = s["idx"].long(), s["dw"], _scores(logits, c)
    v = sc.gather(1, idx)
    if c["renorm"]:
        w = v / v.sum(1, keepdim=True)
        d = w * (dw - (w * dw).sum(1, keepdim=True))
        d = d * (1 - v) if c["scoring"] == "sigmoid" else d
        out = torch.zeros_like(sc).scatter_(1, idx, d)
    elif c["scoring"] == "sigmoid":
        out = torch.zeros_like(sc).scatter_(1, idx, v * (1 - v) * dw)
    else:
        out = sc * (torch.zeros_like(sc).scatter_(1, idx, dw) - (v * dw).sum(1, keepdim=True))
    return dict(d_logits=out.to(logits.dtype))


def _checkpoint(s):
    q, k = _pack(s["x"])
    return dict(values=_unpack(q, k).to(BF16), exponents=k)


def _experts(s):
    c = s["case"]
    T, H, E, K = c["T"], c["H"], c["E"], c["K"]
    x = s["x"].to(F32) if s["x_scale"] is None else _unpack(s["x"].view(torch.float8_e4m3fn), s["x_scale"])
    dev, M = x.device, s["most"]
    off = s["offsets"].long()
    slot = s["slot_pos"].long().reshape(-1)
    # rows of every expert side by side, padded to the busiest one's: pair (t, j) of each
    pair_of = torch.empty(T * K, dtype=torch.long, device=dev)
    pair_of[slot] = torch.arange(T * K, device=dev)
    pos = off[:-1, None] + torch.arange(M, device=dev)
    live = (pos < off[1:, None]).to(F32)[..., None]
    pair = pair_of[pos.clamp(max=T * K - 1)]
    X, D = x[pair // K] * live, s["dY"].to(F32)[pair // K] * live
    w = s["topk_w"].reshape(-1)[pair][..., None] * live
    W1, W3, W2 = s["W1"].to(F32), s["W3"].to(F32), s["W2"].to(F32)
    g, u, p = X @ W1, X @ W3, D @ W2.transpose(1, 2)
    sg = 1 / (1 + torch.exp(-g))
    h = g * sg * u
    dw = (p * h).sum(-1)
    pw = p * w
    dg, du = pw * u * sg * (1 + g * (1 - sg)), pw * g * sg
    dXp = dg @ W1.transpose(1, 2) + du @ W3.transpose(1, 2)
    place = s["idx"].long().reshape(-1)
    place = place * M + slot - off[place]
    return dict(dX=dXp.view(E * M, H)[place].view(T, K, H).sum(1).to(BF16), d_topk_w=dw.reshape(-1)[place].view(T, K),
                dW1=(X.transpose(1, 2) @ dg).to(BF16), dW3=(X.transpose(1, 2) @ du).to(BF16),
                dW2=((h * w).transpose(1, 2) @ D).to(BF16))


# ------------------------------------------------------------------------- the library's calls
def _buffers(s):
    """Outputs and workspace, which a training loop keeps from step to step."""
    if "out" in s:
        return s["out"], s["ws"]
    from expert_routed_ffn_router_gb300 import binding as B
    c, o, n = s["case"], {}, 0

    def new(*shape, dtype=F32):
        return torch.empty(*shape, dtype=dtype, device=DEV)
    if c["op"] == "norm" and c["dir"] == "forward":
        o = dict(y=new(c["T"], c["H"], dtype=BF16), mean=new(c["T"]), rstd=new(c["T"]))
    elif c["op"] == "norm":
        o = dict(dx=torch.empty_like(s["x"]), dgamma=new(c["H"]), dbeta=new(c["H"]))
        n = B.moe_layer_norm_backward_workspace_bytes(c["T"], c["H"])
    elif c["op"] == "route" and c["dir"] == "forward":
        o = dict(topk_idx=new(c["T"], c["K"], dtype=torch.int32), topk_w=new(c["T"], c["K"]))
    elif c["op"] == "route":
        o = dict(d_logits=torch.empty_like(s["logits"]))
    elif c["op"] == "checkpoint":
        nb = -(-c["n"] // BLOCK)
        o = dict(values=torch.empty_like(s["x"]), exponents=new(c["T"], nb, dtype=torch.int8))
        s["q"] = new(c["T"], c["n"], dtype=torch.uint8)
    else:
        o = dict(dX=new(c["T"], c["H"], dtype=BF16), d_topk_w=new(c["T"], c["K"]), dW1=torch.empty_like(s["W1"]),
                 dW3=torch.empty_like(s["W3"]), dW2=torch.empty_like(s["W2"]))
        n = B.moe_expert_ffn_backward_workspace_bytes(c["T"], c["H"], c["E"], c["K"], c["I"])
    if c["op"] == "route":
        s["routing"] = B.MoeRouting.make(c["scoring"], c["n_group"], c["topk_group"], c["group_top"], c["renorm"])
    s["out"], s["ws"] = o, torch.zeros(max(n, 256), dtype=torch.uint8, device=DEV)
    return s["out"], s["ws"]


def _own(s):
    from expert_routed_ffn_router_gb300 import binding as B
    c = s["case"]
    o, ws = _buffers(s)
    if c["op"] == "norm" and c["dir"] == "forward":
        B.moe_layer_norm(s["x"], s["gamma"], s["beta"], EPS, o["y"], o["mean"], o["rstd"])
    elif c["op"] == "norm":
        B.moe_layer_norm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["res"], o["dx"], o["dgamma"],
                                  o["dbeta"], ws)
    elif c["op"] == "route" and c["dir"] == "forward":
        B.moe_route_logits(s["logits"], s["bias"], c["K"], s["routing"], o["topk_idx"], o["topk_w"])
    elif c["op"] == "route":
        B.moe_route_logits_backward(s["logits"], s["routing"], s["idx"], s["dw"], o["d_logits"])
    elif c["op"] == "checkpoint":
        B.moe_checkpoint_pack(s["x"], s["q"], o["exponents"])
        B.moe_checkpoint_unpack(s["q"], o["exponents"], o["values"])
    else:
        B.moe_expert_ffn_backward(s["x"], s["x_scale"], s["dY"], s["offsets"], s["slot_pos"], s["topk_w"], s["W1"],
                                  s["W3"], s["W2"], o["dX"], o["d_topk_w"], o["dW1"], o["dW3"], o["dW2"], ws)
    return o


def run(state):
    if own:
        return _own(state)
    return {"norm": _norm, "route": _route, "checkpoint": _checkpoint, "experts": _experts}[state["case"]["op"]](state)


# ------------------------------------------------------------------------- bytes and products
def work(case):
    c = case
    if c["op"] == "norm":
        n, b = c["T"] * c["H"], 4 if c["x"] == "f32" else 2
        if c["dir"] == "forward":
            return dict(bytes=n * (b + 2) + 8 * c["T"] + 8 * c["H"], flops=8 * n)
        return dict(bytes=n * (2 + 2 * b + (b if c["res"] else 0)) + 8 * c["T"] + 12 * c["H"], flops=14 * n)
    if c["op"] == "route":
        b, pairs = 4 if c["l"] == "f32" else 2, c["T"] * c["K"]
        if c["dir"] == "forward":
            return dict(bytes=c["T"] * c["E"] * b + 8 * pairs + (4 * c["E"] if c["bias"] else 0), flops=4 * c["T"] * c["E"])
        dense = c["scoring"] == "softmax" and not c["renorm"]
        read = c["T"] * c["E"] if dense else pairs
        return dict(bytes=(c["T"] * c["E"] + read) * b + 8 * pairs, flops=4 * read + 4 * pairs)
    if c["op"] == "checkpoint":
        # packed and taken back: bf16 read, bytes written, bytes read, bf16 written
        n = c["T"] * c["n"]
        return dict(bytes=6 * n + 2 * c["T"] * (-(-c["n"] // BLOCK)), flops=4 * n)
    T, H, E, K, I = (c[k] for k in ("T", "H", "E", "K", "I"))
    used = E * (1 - (1 - K / E) ** T)           # experts that have rows
    matrix = 3 * H * I * 2
    return dict(bytes=matrix * (used + E) + T * H * ((1 if c["packed"] else 2) + 4) + 12 * T * K, flops=16.0 * T * K * H * I)


# ------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    F64 = torch.float64
    if c["op"] == "norm":
        x = s["x"].to(F64).requires_grad_(c["dir"] == "backward")
        gamma = s["gamma"].to(F64).requires_grad_(c["dir"] == "backward")
        beta = s["beta"].to(F64).requires_grad_(c["dir"] == "backward")
        if c["dir"] == "forward":
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rstd = (var + EPS) ** -0.5
            return dict(y=gamma * ((x - mean[:, None]) * rstd[:, None]) + beta, mean=mean, rstd=rstd)
        # the gradient for the statistics that the caller hands over
        mean, rstd = s["mean"].to(F64)[:, None], s["rstd"].to(F64)[:, None]
        dy = s["dy"].to(F64)
        with torch.no_grad():
            xh = x.sub(mean).mul_(rstd)
            t = torch.einsum("th,h->th", dy, gamma)
            dx = torch.einsum("th,th->t", t, xh)[:, None] / c["H"] * xh
            dx = (t - t.sum(1, keepdim=True) / c["H"] - dx) * rstd
            if s["res"] is not None:
                dx += s["res"].to(F64)
            return dict(dx=dx, dgamma=torch.einsum("th,th->h", dy, xh), dbeta=torch.einsum("th->h", dy))
    if c["op"] == "route":
        import numpy as np
        l = s["logits"].to(F64).cpu().numpy()
        z = np.exp(l - l.max(1, keepdims=True)) if c["scoring"] == "softmax" else 1.0 / (1.0 + np.exp(-l))
        sc = z / z.sum(1, keepdims=True) if c["scoring"] == "softmax" else z
        rows = np.arange(c["T"])[:, None]
        if c["dir"] == "forward":
            sel = sc + (0.0 if s["bias"] is None else s["bias"].to(F64).cpu().numpy())
            G = c["E"] // c["n_group"]
            best = -np.sort(-sel.reshape(c["T"], c["n_group"], G), axis=2)[:, :, :c["group_top"]].sum(2)
            out = np.argsort(-best, axis=1, kind="stable")[:, c["topk_group"]:]
            lost = np.zeros((c["T"], c["n_group"]), bool)
            lost[rows, out] = True
            sel = np.where(np.repeat(lost, G, axis=1), -np.inf, sel)
            idx = np.argsort(-sel, axis=1, kind="stable")[:, :c["K"]]
            w = sc[rows, idx]
            return dict(topk_idx=idx.astype(np.int32), topk_w=w / w.sum(1, keepdims=True) if c["renorm"] else w)
        # through the definition, by automatic differentiation
        t = torch.from_numpy(l).requires_grad_(True)
        v = (torch.softmax(t, 1) if c["scoring"] == "softmax" else torch.sigmoid(t)).gather(1, s["idx"].long().cpu())
        v = v / v.sum(1, keepdim=True) if c["renorm"] else v
        v.backward(s["dw"].to(F64).cpu())
        return dict(d_logits=t.grad)
    if c["op"] == "checkpoint":
        # by the spacing of E4M3 numbers: 2^-3 of the leading power, 2^-9 at the least
        v = s["x"].to(F64)
        nb = -(-c["n"] // BLOCK)
        v = torch.nn.functional.pad(v, (0, nb * BLOCK - c["n"])).view(c["T"], nb, BLOCK)
        amax = v.abs().amax(-1, keepdim=True)
        k = torch.ceil(torch.log2(torch.where(amax > 0, amax, torch.full_like(amax, 448.0)) / 448.0)).clamp(-124, 127)
        lead = torch.floor(torch.log2(torch.where(v == 0, torch.ones_like(v), v.abs())))
        step = torch.exp2(torch.maximum(lead - k, torch.full_like(k, -6.0)) - 3 + k)
        v = torch.round(v / step) * step
        return dict(values=v.view(c["T"], nb * BLOCK)[:, :c["n"]], exponents=k.squeeze(-1))
    # sum of the outputs times dY, differentiated expert by expert
    x = s["x"].to(F64) if s["x_scale"] is None else _unpack(s["x"].view(torch.float8_e4m3fn), s["x_scale"]).to(F64)
    dY, w = s["dY"].to(F64), s["topk_w"].to(F64)
    dX, dw = torch.zeros_like(x), torch.zeros_like(w)
    grads = {n: torch.zeros(s[n].shape, dtype=F64, device=x.device) for n in ("W1", "W3", "W2")}
    for e in range(c["E"]):
        t, j = (s["idx"] == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        xe, we = x[t].requires_grad_(True), w[t, j].requires_grad_(True)
        W = [s[n][e].to(F64).requires_grad_(True) for n in ("W1", "W3", "W2")]
        y = (torch.nn.functional.silu(xe @ W[0]) * (xe @ W[1])) @ W[2]
        got = torch.autograd.grad((we[:, None] * y * dY[t]).sum(), [xe, we] + W)
        dX.index_add_(0, t, got[0])
        dw[t, j] = got[1]
        for n, v in zip(("W1", "W3", "W2"), got[2:]):
            grads[n][e] = v
    return dict(dX=dX, d_topk_w=dw, dW1=grads["W1"], dW3=grads["W3"], dW2=grads["W2"])
