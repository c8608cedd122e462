"""A node-wise block between two aggregation layers, with its training step:

    H' = H + (act(Y Wg) * (Y Wu)) Wd,   Y = act_norm(group_norm(H))

group norm over the segments of nodes (partitions, or the graphs of a batch),
the gated projections, the dense transform back to the layer's width and the
residual; the backward; and one clipped AdamW step over all five weights.
Every step is a call of the library; torch holds the memory and adds the
residual."""
from __future__ import annotations

import torch

from . import (AdamwTensors, adamw_state, gnn_adamw_step, gnn_dense_bwd, gnn_dense_fwd, gnn_gated_bwd,
               gnn_gated_fwd, gnn_group_norm_bwd, gnn_group_norm_fwd, ldb_for)


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
