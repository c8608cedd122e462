"""Node-wise blocks between aggregation layers, with their training steps.

NodeBlock, one block:

    H' = H + (act(Y Wg) * (Y Wu)) Wd,   Y = act_norm(group_norm(H))

group norm over the segments of nodes (partitions, or the graphs of a batch),
the gated projections, the dense transform back to the layer's width and the
residual; the backward; and one clipped AdamW step over all five weights.

NodeStack, several on one residual stream, with norms by rows before and after:

    H_l+1 = H_l + s_l norm((act(Y_l Wg) * (Y_l Wu)) Wd) w_post,   Y_l = norm(H_l) w_pre

where one call between two blocks takes the norm after the first, its scale, the
sum and the norm before the second; Muon steps for the matrices, AdamW for the
vectors.  Every step is a call of the library; torch holds the memory, adds
NodeBlock's residual and widens the gated projections' gradients, which the
library rounds to the weights' 2-byte type, to the optimisers' fp32 (so 8 of their
bits count, with Muon as with AdamW)."""
from __future__ import annotations

import torch

from . import (AdamwTensors, MuonTensors, adamw_state, gnn_adamw_step, gnn_dense_bwd, gnn_dense_fwd, gnn_gated_bwd,
               gnn_gated_fwd, gnn_group_norm_bwd, gnn_group_norm_fwd, gnn_muon_step, gnn_residual_norm_bwd,
               gnn_residual_norm_fwd, ldb_for)


class NodeBlock:
    """F: the layer's width (a multiple of 16, at most 256, as the dense
    transform takes it); F_mid: a multiple of 16, at most 1024.  seg_start:
    int64 borders of the segments (``Boundary.part_start``; None: all nodes are
    one).  state_bits: 32 or 8 for AdamW's states."""

    def __init__(self, F: int, F_mid: int, groups: int, seg_start=None, act: str = "silu", act_norm: str = "none",
                 state_bits: int = 32, seed: int = 0, device="cuda"):
        if F % 16 or F > 256 or F_mid % 16 or F_mid > 1024:
            raise ValueError(f"NodeBlock: F={F} has to be a multiple of 16 up to 256, F_mid={F_mid} one up to 1024")
        self.F, self.F_mid, self.groups, self.seg, self.act, self.act_norm = F, F_mid, groups, seg_start, act, act_norm
        gen = torch.Generator(device=device).manual_seed(seed)

        def glorot(r, c):
            lim = (6.0 / (r + c)) ** 0.5
            return (torch.rand(r, c, generator=gen, device=device) * 2 - 1) * lim

        # fp32 weights that AdamW updates, and the bf16 copies the tensor cores read
        self.weights = dict(gamma=torch.ones(F, device=device), beta=torch.zeros(F, device=device),
                            Wg=glorot(F, F_mid), Wu=glorot(F, F_mid), Wd=glorot(F_mid, F))
        self.bf16 = {k: w.to(torch.bfloat16) for k, w in self.weights.items() if k.startswith("W")}
        self.grads = {k: torch.zeros_like(w) for k, w in self.weights.items()}
        self.grad_norm = torch.zeros(1, device=device)
        self.state = adamw_state(device)
        eight = state_bits == 8
        kind = torch.float8_e4m3fn if eight else torch.float32
        ws = list(self.weights.values())
        scale = lambda: [torch.zeros(-(-w.numel() // 256), device=device) for w in ws] if eight else None  # noqa: E731
        self._tensors = AdamwTensors([w.view(-1) for w in ws], [g.view(-1) for g in self.grads.values()],
                                     [torch.zeros(w.numel(), device=device).to(kind) for w in ws],
                                     [torch.zeros(w.numel(), device=device).to(kind) for w in ws], scale(), scale(),
                                     [self.bf16[k].view(-1) if k in self.bf16 else None for k in self.weights])
        self._kept = None

    def forward(self, H, out=None, stream=None):
        """H: fp32 [n, F]; returns H' (fp32 [n, F], `out` if given; with out = H in
        place, which costs a copy: the backward needs H as it was)."""
        n, F, Fm, dev = H.shape[0], self.F, self.F_mid, H.device
        segs = 1 if self.seg is None else self.seg.numel() - 1
        with torch.cuda.stream(stream):
            Y = torch.empty(n, ldb_for(F), dtype=torch.bfloat16, device=dev)
            M = torch.empty(n, ldb_for(Fm), dtype=torch.bfloat16, device=dev)
            mean, rstd = torch.empty(segs, self.groups, device=dev), torch.empty(segs, self.groups, device=dev)
            Z = torch.empty(n, F, device=dev)
            w = self.weights
            gnn_group_norm_fwd(H, n, F, self.groups, Y, mean, rstd, seg_start=self.seg, gamma=w["gamma"],
                               beta=w["beta"], act=self.act_norm, stream=stream)
            gnn_gated_fwd(Y, n, F, self.bf16["Wg"], self.bf16["Wu"], Fm, M, act=self.act, stream=stream)
            gnn_dense_fwd(M, n, Fm, self.bf16["Wd"], F, False, Z, stream=stream)
            shared = out is not None and out.untyped_storage().data_ptr() == H.untyped_storage().data_ptr()
            self._kept = (H.clone() if shared else H, Y, M, mean, rstd)
            return torch.add(H, Z, out=out)

    def backward(self, dH_out, stream=None):
        """dH_out: fp32 [n, F]; fills self.grads and returns dH (fp32 [n, F])."""
        H, Y, M, mean, rstd = self._kept
        n, F, Fm, dev = H.shape[0], self.F, self.F_mid, H.device
        with torch.cuda.stream(stream):
            dM = torch.empty(n, Fm, device=dev)
            gnn_dense_bwd(M, n, Fm, self.bf16["Wd"], F, dH_out, None, False, dM, self.grads["Wd"], stream=stream)
            dY = torch.empty_like(Y)
            dWg, dWu = torch.empty_like(self.bf16["Wg"]), torch.empty_like(self.bf16["Wu"])
            gnn_gated_bwd(dM, Y, n, F, self.bf16["Wg"], self.bf16["Wu"], Fm, dX=dY, dWg=dWg, dWu=dWu, act=self.act,
                          stream=stream)
            self.grads["Wg"].copy_(dWg)
            self.grads["Wu"].copy_(dWu)
            dH = torch.empty(n, F, device=dev)
            gnn_group_norm_bwd(dY, H, n, F, self.groups, mean, rstd, dH, dgamma=self.grads["gamma"],
                               dbeta=self.grads["beta"], seg_start=self.seg, gamma=self.weights["gamma"],
                               beta=self.weights["beta"], act=self.act_norm, stream=stream)
            return dH.add_(dH_out)

    def step(self, lr: float, max_norm: float = 1.0, stream=None, **hyper):
        """One AdamW step from self.grads (fp32 weights and bf16 copies)."""
        gnn_adamw_step(self._tensors, self.state, lr, max_norm=max_norm, grad_norm=self.grad_norm, stream=stream, **hyper)


class NodeStack:
    """depth blocks of width F (a multiple of 16, at most 256) and F_mid (a multiple
    of 16, at most 1024).  norm: "rms" or "layer"; scale: what every block's learned
    scale s starts at.  The passes of one step go to one stream."""

    def __init__(self, depth: int, F: int, F_mid: int, act: str = "silu", norm: str = "rms", scale: float = 1.0,
                 seed: int = 0, device="cuda"):
        if F % 16 or F > 256 or F_mid % 16 or F_mid > 1024 or depth < 1:
            raise ValueError(f"NodeStack: depth={depth} >= 1, F={F} a multiple of 16 up to 256, F_mid={F_mid} one up to 1024")
        self.depth, self.F, self.F_mid, self.act, self.norm = depth, F, F_mid, act, norm
        gen = torch.Generator(device=device).manual_seed(seed)

        def glorot(r, c):
            lim = (6.0 / (r + c)) ** 0.5
            return (torch.rand(r, c, generator=gen, device=device) * 2 - 1) * lim

        ones = lambda: torch.ones(F, device=device)  # noqa: E731
        # fp32 weights that the steps update, and the bf16 copies the tensor cores read
        self.weights = [dict(w_pre=ones(), Wg=glorot(F, F_mid), Wu=glorot(F, F_mid), Wd=glorot(F_mid, F), w_post=ones(),
                             scale=ones() * scale) for _ in range(depth)]
        self.bf16 = [{k: w[k].to(torch.bfloat16) for k in ("Wg", "Wu", "Wd")} for w in self.weights]
        self.grads = [{k: torch.zeros_like(v) for k, v in w.items()} for w in self.weights]
        mats = [(w[k], g[k], b[k]) for w, g, b in zip(self.weights, self.grads, self.bf16) for k in ("Wg", "Wu", "Wd")]
        vecs = [(w[k], g[k]) for w, g in zip(self.weights, self.grads) for k in ("w_pre", "w_post", "scale")]
        self.momenta = [torch.zeros_like(w) for w, _, _ in mats]
        self.norms = torch.zeros(len(mats), device=device)
        self._muon = MuonTensors([w for w, _, _ in mats], [g for _, g, _ in mats], self.momenta, [b for _, _, b in mats])
        self.state = adamw_state(device)
        self._adamw = AdamwTensors([w for w, _ in vecs], [g for _, g in vecs], [torch.zeros(F, device=device) for _ in vecs],
                                   [torch.zeros(F, device=device) for _ in vecs])
        self._kept = None

    def forward(self, H, stream=None):
        """H: fp32 [n, F], n >= 1; returns the stream behind the last block (fp32 [n, F]).
        H is kept, not copied: it stays as it is until the backward has run."""
        if H.dim() != 2 or H.shape[0] < 1 or H.shape[1] != self.F or H.dtype is not torch.float32:
            raise ValueError(f"H: needs fp32 [n, {self.F}] with n >= 1, got {H.dtype} {tuple(H.shape)}")
        n, F, Fm, dev, norm = H.shape[0], self.F, self.F_mid, H.device, self.norm
        with torch.cuda.stream(stream):
            operand = lambda c: torch.empty(n, ldb_for(c), dtype=torch.bfloat16, device=dev)  # noqa: E731
            stats = lambda: torch.empty(n, 4, device=dev)  # noqa: E731
            Y, st = operand(F), stats()
            gnn_residual_norm_fwd(None, H, n, F, None, Y, st, pre=norm, w_pre=self.weights[0]["w_pre"], stream=stream)
            kept = [(H, Y, st)]
            for i, (w, b) in enumerate(zip(self.weights, self.bf16)):
                last = i + 1 == self.depth
                M, Z, out, st = operand(Fm), torch.empty(n, F, device=dev), torch.empty(n, F, device=dev), stats()
                gnn_gated_fwd(Y, n, F, b["Wg"], b["Wu"], Fm, M, act=self.act, stream=stream)
                gnn_dense_fwd(M, n, Fm, b["Wd"], F, False, Z, stream=stream)
                Y = None if last else operand(F)
                gnn_residual_norm_fwd(Z, H, n, F, out, Y, st, post=norm, w_post=w["w_post"], scale=w["scale"],
                                      pre="none" if last else norm, w_pre=None if last else self.weights[i + 1]["w_pre"],
                                      stream=stream)
                kept.append((M, Z, out, Y, st))
                H = out
            self._kept = kept
            return H

    def backward(self, dH, stream=None):
        """dH: fp32 [n, F]; fills self.grads and returns the gradient of forward's H."""
        (H0, Y0, st0), *blocks = self._kept
        n, F, Fm, dev, norm = H0.shape[0], self.F, self.F_mid, H0.device, self.norm
        with torch.cuda.stream(stream):
            dY = None
            for i in reversed(range(self.depth)):
                w, b, g = self.weights[i], self.bf16[i], self.grads[i]
                M, Z, out, _, st = blocks[i]
                Y = Y0 if i == 0 else blocks[i - 1][3]
                last = i + 1 == self.depth
                dR, dZ, dM = torch.empty(n, F, device=dev), torch.empty(n, F, device=dev), torch.empty(n, Fm, device=dev)
                gnn_residual_norm_bwd(dH, dY, Z, out, n, F, st, dR, dZ, post=norm, w_post=w["w_post"], scale=w["scale"],
                                      pre="none" if last else norm, w_pre=None if last else self.weights[i + 1]["w_pre"],
                                      dw_post=g["w_post"], dscale=g["scale"],
                                      dw_pre=None if last else self.grads[i + 1]["w_pre"], stream=stream)
                gnn_dense_bwd(M, n, Fm, b["Wd"], F, dZ, None, False, dM, g["Wd"], stream=stream)
                dY, dWg, dWu = torch.empty_like(Y), torch.empty_like(b["Wg"]), torch.empty_like(b["Wu"])
                gnn_gated_bwd(dM, Y, n, F, b["Wg"], b["Wu"], Fm, dX=dY, dWg=dWg, dWu=dWu, act=self.act, stream=stream)
                g["Wg"].copy_(dWg)
                g["Wu"].copy_(dWu)
                dH = dR
            dR = torch.empty(n, F, device=dev)
            gnn_residual_norm_bwd(dH, dY, None, H0, n, F, st0, dR, pre=norm, w_pre=self.weights[0]["w_pre"],
                                  dw_pre=self.grads[0]["w_pre"], stream=stream)
            return dR

    def step(self, lr: float, momentum: float = 0.95, nesterov: bool = True, weight_decay: float = 0.0, stream=None,
             **vectors):
        """One step from self.grads: Muon for the matrices (fp32 weights and bf16
        copies), AdamW for the vectors (`vectors`: its other arguments)."""
        gnn_muon_step(self._muon, lr, momentum=momentum, nesterov=nesterov, weight_decay=weight_decay, norms=self.norms,
                      stream=stream)
        gnn_adamw_step(self._adamw, self.state, lr, weight_decay=vectors.pop("vector_decay", 0.0), stream=stream, **vectors)
