"""One training step of a pre-norm MoE block on the library's entry points.

    out = x + sum_j w_j FFN_e(j)(n) + FFN_shared(n),   n = layer_norm(x)

or, with a norm behind the experts, a gate for each channel or another scale of the stream,

    out = alpha x + gate post_norm(sum_j w_j FFN_e(j)(n) + FFN_shared(n))

with the routing weights w of a gate that is trained: logits = n W_gate^T in fp32.  Between the
forward and the backward pass the block keeps x, the norm's statistics, the logits, the routing
and its dispatch, and n in bf16, or with ``packed=True`` as an 8-bit checkpoint (E4M3 bytes and
exponents, half the memory; the gradients are then those of rows with a 3-bit mantissa); the
experts' activations are computed again.

    block = MoETrainBlock(weights, T=4096, K=8)
    out = block.forward(x)                  # x fp32 or bf16 [T, H]
    dx, grads = block.backward(dout)        # dout of x's type

Outputs, what is kept and the workspace are allocated once; the gate's products, in fp32, and the
sum of the branches' gradients take temporaries of torch's allocator in each pass (fp32 copies of
n and dn, T x H each).  Both passes only enqueue work on the current stream and can be captured in
a CUDA graph.  The three products with the gate are plain library products (torch.mm); the
additions and casts around them are torch's, everything else runs in the library's kernels.

Roundings of the gradient that reaches the norm: the experts' dX and the shared expert's are bf16
as the kernels leave them; they are added to the gate's part in fp32, and the sum is rounded to
bf16 once, the type moe_layer_norm_backward takes.

    python -m expert_routed_ffn_router_gb300.train --steps 30

fits a small block to random targets and prints the loss; with ``--muon`` the experts' matrices take
orthogonalised updates with momentum (Muon, below) in place of plain gradient descent.
"""
from __future__ import annotations

import argparse
import math

import torch

from . import binding as B

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
EXPERTS = ("W1", "W3", "W2")


class MoETrainBlock:
    """weights: gamma, beta fp32 [H]; W_gate fp32 [E, H]; bias fp32 [E] or None (selection
    only); W1, W3 bf16 [E, H, I], W2 bf16 [E, I, H]; optionally the shared expert's W1s, W3s
    [H, Is], W2s [Is, H], and gate fp32 [H], gamma_post and beta_post fp32 [H] (with post).  routing:
    as for moe_route_logits; post, alpha: as for moe_residual_norm."""

    def __init__(self, weights: dict, T: int, K: int, routing=None, eps: float = 1e-5,
                 packed: bool = False, x_dtype=F32, post: str = "none", alpha: float = 1.0):
        self.w, self.T, self.K, self.eps, self.packed = weights, T, K, eps, packed
        self.routing = B.MoeRouting.make(**routing) if isinstance(routing, dict) else routing
        self.E, self.H, self.I = weights["W1"].shape
        self.shared = weights.get("W1s") is not None
        Is = weights["W1s"].shape[-1] if self.shared else 0
        E, H, I = self.E, self.H, self.I
        dev = weights["W1"].device

        def new(*shape, dtype=F32):
            return torch.empty(*shape, dtype=dtype, device=dev)

        # kept from the forward pass
        self.x = None
        self.n = new(T, H, dtype=BF16)
        self.mean, self.rstd = new(T), new(T)
        self.logits = new(T, E)
        self.topk_idx, self.topk_w = new(T, K, dtype=I32), new(T, K)
        self.counts, self.offsets = new(E, dtype=I32), new(E + 1, dtype=I32)
        self.slot_pos = new(T, K, dtype=I32)
        self.q = new(T, H, dtype=torch.uint8) if packed else None
        self.scale = new(T, (H + 127) // 128, dtype=torch.int8) if packed else None
        # forward
        self.perm, self.Xp = new(T * K, dtype=I32), new(T * K, H, dtype=BF16)
        self.Yp, self.Y = new(T * K, H, dtype=BF16), new(T, H)
        self.Ysh = new(T, H) if self.shared else None
        self.out = new(T, H, dtype=x_dtype)
        # backward
        self.d_topk_w, self.d_logits = new(T, K), new(T, E)
        self.dn, self.dY, self.dx = new(T, H, dtype=BF16), new(T, H, dtype=BF16), new(T, H, dtype=x_dtype)
        self.dn_shared = new(T, H, dtype=BF16) if self.shared else None
        # the branch's own norm, gate and scale: the stream is joined by one kernel each way then
        ends = tuple(n for n in (("gamma_post", "beta_post") if post != "none" else ()) + ("gate",)
                     if weights.get(n) is not None)
        self.join = dict(post=post, alpha=alpha, eps_post=eps, **{n: weights[n] for n in ends})
        self.joined = post != "none" or alpha != 1.0 or bool(ends)
        self.stats = new(T, 4) if self.joined else None
        names = EXPERTS + (tuple(n + "s" for n in EXPERTS) if self.shared else ())
        self.grads = {n: torch.empty_like(weights[n]) for n in ("gamma", "beta", "W_gate") + names + ends}
        self.join_grads = {n: self.grads[n] for n in ends}
        # the shared expert: one group that holds every token once, weight 1
        self.all_rows = torch.tensor([0, T], dtype=I32, device=dev)
        self.each_row = torch.arange(T, dtype=I32, device=dev).view(T, 1)
        nbytes = max(B.moe_workspace_bytes(T, H, E, K, I, Is), B.moe_expert_ffn_workspace_bytes(T * K, E, I),
                     B.moe_expert_ffn_backward_workspace_bytes(T, H, E, K, I),
                     B.moe_layer_norm_backward_workspace_bytes(T, H),
                     B.moe_residual_norm_backward_workspace_bytes(T, H) if self.joined else 0,
                     B.moe_expert_ffn_workspace_bytes(T, 1, Is) if self.shared else 0,
                     B.moe_expert_ffn_backward_workspace_bytes(T, H, 1, 1, Is) if self.shared else 0)
        if nbytes == 0 or B.moe_expert_ffn_backward_workspace_bytes(T, H, E, K, I) == 0:
            raise B.MoeError("moe_expert_ffn_backward_workspace_bytes", -2)
        self.ws = torch.zeros(nbytes, dtype=torch.uint8, device=dev)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        w, K, E = self.w, self.K, self.E
        self.x = x
        B.moe_layer_norm(x, w["gamma"], w["beta"], self.eps, self.n, self.mean, self.rstd)
        if self.packed:
            B.moe_checkpoint_pack(self.n, self.q, self.scale)
        torch.mm(self.n.float(), w["W_gate"].t(), out=self.logits)
        B.moe_route_logits(self.logits, w.get("bias"), K, self.routing, self.topk_idx, self.topk_w)
        B.moe_dispatch(self.n, self.topk_idx, E, self.counts, self.offsets, self.perm, self.slot_pos,
                       self.Xp, None, self.ws)
        B.moe_expert_ffn(self.Xp, self.offsets, E, w["W1"], w["W3"], w["W2"], self.Yp, self.ws)
        if self.shared:
            B.moe_expert_ffn(self.n, self.all_rows, 1, w["W1s"], w["W3s"], w["W2s"], self.Ysh, self.ws)
        B.moe_combine(self.Yp, self.slot_pos, self.topk_w, self.Ysh, self.Y)
        if self.joined:
            B.moe_residual_norm(x, self.Y, self.join, self.out, None, self.stats)
        else:
            torch.add(x, self.Y, out=self.out)
        return self.out

    def backward(self, dout: torch.Tensor):
        """Gradient of the last forward call's output -> (dx, gradients by weight name): the
        block's own buffers, which the next call overwrites."""
        if self.x is None:
            raise RuntimeError("backward() before forward()")
        w, g = self.w, self.grads
        rows, scale = (self.q, self.scale) if self.packed else (self.n, None)
        dres = dout
        if self.joined:
            dres = self.dx
            B.moe_residual_norm_backward(None, dout, self.Y, None, self.stats, self.join, self.dx, self.dY,
                                         self.join_grads, self.ws)
        else:
            self.dY.copy_(dout)
        B.moe_expert_ffn_backward(rows, scale, self.dY, self.offsets, self.slot_pos, self.topk_w, w["W1"],
                                  w["W3"], w["W2"], self.dn, self.d_topk_w, g["W1"], g["W3"], g["W2"], self.ws)
        B.moe_route_logits_backward(self.logits, self.routing, self.topk_idx, self.d_topk_w, self.d_logits)
        n = (B.moe_checkpoint_unpack(self.q, self.scale) if self.packed else self.n).float()
        torch.mm(self.d_logits.t(), n, out=g["W_gate"])
        dn = torch.addmm(self.dn.float(), self.d_logits, w["W_gate"])
        if self.shared:
            B.moe_expert_ffn_backward(rows, scale, self.dY, self.all_rows, self.each_row, None,
                                      w["W1s"][None], w["W3s"][None], w["W2s"][None], self.dn_shared, None,
                                      g["W1s"][None], g["W3s"][None], g["W2s"][None], self.ws)
            dn += self.dn_shared
        B.moe_layer_norm_backward(dn.to(BF16), self.x, w["gamma"], self.mean, self.rstd, dres, self.dx,
                                  g["gamma"], g["beta"], self.ws)
        return self.dx, g

    def status(self) -> int:
        """Conditions the kernels recorded (moe_read_status; synchronises)."""
        return B.moe_read_status(self.ws)


class Muon:
    """Orthogonalised updates with momentum for a block's matrices.

        m <- mu m + g,  W <- (1 - lr decay) W - lr 0.2 sqrt(max(R, C)) orthogonalised(g + mu m)

    The factor gives every entry of the update a mean square of about 0.2^2, whatever the matrix's
    sides.  weights: the bf16 tensors by name, [R, C] or [E, R, C]; master copies in fp32 and the
    momentum are kept here.  experts: matrices that one call orthogonalises, at most (the workspace
    grows with them; None: all of a tensor); a call starts on a boundary of 16 bytes, which takes up
    to eight matrices where R C is no multiple of 8."""

    def __init__(self, weights: dict, lr: float = 0.02, mu: float = 0.95, decay: float = 0.0, experts=None):
        if experts is not None and (int(experts) != experts or experts < 1):
            raise ValueError(f"experts: {experts!r}, expected a number of matrices from 1 on, or None")
        experts = None if experts is None else int(experts)
        self.weights, self.lr, self.mu, self.decay, self.experts = weights, lr, mu, decay, experts
        self.master = {n: w.float() for n, w in weights.items()}
        self.momentum = {n: torch.zeros_like(m) for n, m in self.master.items()}
        self.update = {n: torch.empty_like(w, dtype=BF16) for n, w in weights.items()}
        need = 256
        for w in weights.values():
            b, R, C = self._shape(w)
            k = self._chunk(b, R, C)
            # (of the last call too, which has the rest: fewer matrices may need more)
            need = max(need, *(B.moe_orthogonalize_workspace_bytes(n, R, C) for n in (k, b % k) if n))
        device = next(iter(weights.values())).device if weights else "cuda"
        self.ws = torch.zeros(need, dtype=torch.uint8, device=device)

    @staticmethod
    def _shape(w):
        return ((1,) + tuple(w.shape))[-3:]

    def _chunk(self, b, R, C):
        """Matrices of a call: b, or as many up to `experts` as end on a boundary of 16 bytes."""
        if self.experts is None or self.experts >= b:
            return max(1, b)
        each = 8 // math.gcd(R * C, 8)
        if self.experts < each:
            raise ValueError(f"experts: {self.experts}, matrices of {R} x {C} take a multiple of {each}")
        return self.experts // each * each

    def step(self, grads: dict) -> None:
        """grads: the gradients by name (bf16 or fp32), of all or some of the weights."""
        for n, g in grads.items():
            b, R, C = self._shape(g)
            k = self._chunk(b, R, C)
            v = [t.view(b, R, C) for t in (g, self.update[n], self.momentum[n])]
            for i in range(0, b, k):
                gi, ui, mi = (t[i:i + k] for t in v)
                B.moe_orthogonalize(gi, ui, self.ws, momentum=mi, mu=self.mu, nesterov=True,
                                    scale=0.2 * max(R, C) ** 0.5)
            self.master[n].mul_(1 - self.lr * self.decay).sub_(self.update[n], alpha=self.lr)
            self.weights[n].copy_(self.master[n])

    def status(self) -> int:
        """Conditions the kernels recorded (moe_read_status; synchronises)."""
        return B.moe_read_status(self.ws)


def random_weights(H, E, I, Is, device, seed=0) -> dict:
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, std, dtype):
        return (std * torch.randn(*shape, generator=g, device=device)).to(dtype)
    w = dict(gamma=torch.ones(H, device=device), beta=torch.zeros(H, device=device),
             W_gate=normal(E, H, std=H ** -0.5, dtype=F32), bias=torch.zeros(E, device=device))
    shapes = [("W1", (E, H, I)), ("W3", (E, H, I)), ("W2", (E, I, H))]
    if Is:
        shapes += [("W1s", (H, Is)), ("W3s", (H, Is)), ("W2s", (Is, H))]
    for name, shape in shapes:
        w[name] = normal(*shape, std=shape[-2] ** -0.5, dtype=BF16)
    return w


def fit(steps=30, T=512, H=256, E=16, K=2, I=128, Is=128, lr=2.0, seed=0, device="cuda", packed=False,
        muon=False):
    """Plain gradient descent (muon: orthogonalised updates for the experts' matrices) on mean
    (out - target)^2 over one fixed batch; the losses."""
    g = torch.Generator(device=device).manual_seed(seed + 1)
    x = torch.randn(T, H, generator=g, device=device)
    target = x + 0.5 * torch.randn(T, H, generator=g, device=device)
    weights = random_weights(H, E, I, Is, device, seed)
    block = MoETrainBlock(weights, T, K, packed=packed)
    matrices = [n for n in block.grads if n.rstrip("s") in EXPERTS] if muon else []
    optimizer = Muon({n: weights[n] for n in matrices}, lr=0.01 * lr) if muon else None
    master = {n: weights[n].float() for n in block.grads if n not in matrices}
    losses = []
    for _ in range(steps):
        diff = block.forward(x) - target
        losses.append(float(diff.square().mean()))
        _, grads = block.backward(2.0 / diff.numel() * diff)
        for n in master:
            master[n] -= lr * grads[n].float()
            weights[n].copy_(master[n])
        if muon:
            optimizer.step({n: grads[n] for n in matrices})
    status = block.status() or (optimizer.status() if muon else 0)       # (reading it resets it)
    if status != 0:
        raise B.MoeError("training step", status)
    return losses


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--T", type=int, default=512)
    ap.add_argument("--lr", type=float, default=2.0)
    rows = ap.add_mutually_exclusive_group()
    rows.add_argument("--packed", action="store_true", help="keep the token rows in 8 bits for the backward pass")
    rows.add_argument("--bf16-rows", action="store_true", help="keep them in bf16 (the default)")
    ap.add_argument("--muon", action="store_true", help="orthogonalised updates for the experts' matrices")
    a = ap.parse_args(argv)
    for i, v in enumerate(fit(steps=a.steps, T=a.T, lr=a.lr, packed=a.packed, muon=a.muon)):
        print(f"step {i:3d}  loss {v:.6f}")


if __name__ == "__main__":
    main()
