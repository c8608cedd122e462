"""Python binding of libgnnagg.so (boundary-quantised GCN aggregation on
GB300).  Functions carry the C entry points' names and only marshal torch
tensors (device memory) and the current CUDA stream into the C ABI; every
step of the computation runs in the library's CUDA kernels.  There is no CPU
path: without the library or a CUDA device the calls raise."""
from __future__ import annotations

import ctypes
import functools
import math
import threading
from dataclasses import dataclass, field
from typing import Optional, Sequence

from . import _abi
from ._abi import (CSR_DEDUP, CSR_GCN, CSR_MEAN, CSR_SELF_LOOPS, CSR_SYMMETRIZE,  # noqa: F401
                   GnnAdamwTensor, GnnBitRule, GnnBlocked, GnnMuonTensor,
                   GnnBoundary, GnnCsr, GnnError, GnnLdrState, call, load)

LdrState = GnnLdrState

__all__ = [
    "Csr", "Boundary", "BitRule", "GnnError", "load", "build",
    "gnn_csr_build", "gnn_csr_split", "gnn_spmm_workspace", "spmm_ws", "gnn_spmm_fwd_noalloc", "gnn_boundary_index", "gnn_boundary_long_slots", "gnn_boundary_set_bits", "gnn_slot_offsets",
    "gnn_quant_pack", "gnn_quant_pack_owned", "gnn_dequant_unpack", "gnn_spmm_fwd", "gnn_spmm_bwd", "gnn_sync_check", "gnn_kernel_launches",
    "rowbytes", "ld_for", "ldb_for", "gnn_dense_workspace", "gnn_dense_fwd", "gnn_dense_bwd",
    "gnn_layer_workspace", "gnn_layer_fwd", "gnn_layer_bwd",
    "gnn_halo_quant_pack", "gnn_spmm_bwd_local", "gnn_quant_pack_slots", "gnn_halo_quant_pack_slots", "gnn_layer_fwd_async", "gnn_layer_bwd_async",
    "LdrState", "gnn_ldr_init", "gnn_ldr_update", "gnn_quant_divide",
    "gnn_layer_tf_workspace", "gnn_layer_fwd_tf", "gnn_layer_bwd_tf",
    "gnn_gat_index", "gnn_gat_workspace", "gnn_gat_layer_fwd", "gnn_gat_layer_bwd",
    "gnn_spmm_bwd_masked", "gnn_spmm_bwd_local_masked", "gnn_dense_bwd_z", "ldz_for",
    "gnn_group_norm_workspace", "gnn_group_norm_fwd", "gnn_group_norm_bwd",
    "gnn_gated_workspace", "gnn_gated_fwd", "gnn_gated_bwd",
    "gnn_residual_norm_workspace", "gnn_residual_norm_fwd", "gnn_residual_norm_bwd",
    "NS_COEFFS", "gnn_orthogonalise_workspace", "gnn_orthogonalise", "MuonTensors", "gnn_muon_workspace", "gnn_muon_step",
    "AdamwTensors", "adamw_state", "gnn_adamw_workspace", "gnn_adamw_step",
    "Blocked", "gnn_blocked_build", "gnn_spmm_fwd_blocked", "gnn_spmm_bwd_blocked",
]


def build(force: bool = False) -> str:
    from . import builder as _b
    return _b.build(force=force)


def _torch():
    import torch
    if not torch.cuda.is_available():
        raise RuntimeError("sparse_aggregation_message_gb300 needs a CUDA device")
    return torch


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream=None) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def ld_for(F: int) -> int:
    """fp32 row stride: F rounded up to a multiple of 4."""
    return (F + 3) // 4 * 4


def ldb_for(F: int) -> int:
    """bf16 row stride for dense-transform inputs: F rounded up to 16."""
    return (F + 15) // 16 * 16


def ldz_for(F: int) -> int:
    """bf16 row stride of a pre-activation gradient dZ: F rounded up to 64."""
    return (F + 63) // 64 * 64


def rowbytes(b: int, F: int) -> int:
    return 16 * ((4 * F + 15) // 16) if b == 32 else 16 * ((F * b + 127) // 128)


@dataclass
class BitRule:
    """Boundary-pool width rule: level = #{i : 100*c > pct[i]*n}, mask =
    bits[level], width = min(8, mask * base)."""
    pct: Sequence[int]
    bits: Sequence[int]

    def to_c(self) -> GnnBitRule:
        r = GnnBitRule()
        r.n_levels = len(self.bits)
        assert len(self.pct) == len(self.bits) - 1
        for i, p in enumerate(self.pct):
            r.pct[i] = int(p)
        for i, b in enumerate(self.bits):
            r.bits[i] = int(b)
        return r


@dataclass
class Csr:
    n: int
    nnz: int
    symmetric: bool
    rowptr: object
    col: object
    val: object
    split_len: int = 0
    n_long: int = 0
    n_pieces: int = 0
    split: dict = field(default_factory=dict)
    val_t: object = None  # A^T weights (mean aggregation); None when A is symmetric

    def c(self) -> GnnCsr:
        s = self.split
        return GnnCsr(self.n, int(self.symmetric), self.nnz, _ptr(self.rowptr), _ptr(self.col),
                      _ptr(self.val), self.split_len, self.n_long, self.n_pieces,
                      _ptr(s.get("long_rows")), _ptr(s.get("piece_ptr")), _ptr(s.get("piece_row")),
                      _ptr(s.get("piece_beg")), _ptr(self.val_t))


@dataclass
class Boundary:
    P: int
    n: int
    n_slots: int
    nnz_cut: int
    F: int
    arrays: dict = field(default_factory=dict)
    long_slot_len: int = 0
    n_long_slots: int = 0

    def __getattr__(self, k):
        arrays = self.__dict__.get("arrays", {})
        if k in arrays:
            return arrays[k]
        raise AttributeError(k)

    def c(self, slot_off=None, F=None) -> GnnBoundary:
        a = self.arrays
        b = GnnBoundary()
        b.P, b.n, b.n_slots, b.nnz_cut = self.P, self.n, self.n_slots, self.nnz_cut
        b.F = self.F if F is None else F
        for k in ("part_start", "send_start", "slot_node", "col_remap", "val_remap", "local_cnt",
                  "slot_rowptr", "slot_col", "slot_val", "own_ptr", "own_slot", "node_bits",
                  "slot_bits"):
            setattr(b, k, _ptr(a[k]))
        b.slot_off = _ptr(a["slot_off"] if slot_off is None else slot_off)
        b.long_slot_len, b.n_long_slots = self.long_slot_len, self.n_long_slots
        b.long_slots = _ptr(a.get("long_slots"))
        b.val_remap_t = _ptr(a.get("val_remap_t"))
        b.halo_order = _ptr(a.get("halo_order"))
        return b


def _workspace(nbytes: int, device):
    torch = _torch()
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


_scratch_of = threading.local()
_SCRATCH_MOST = 32 << 20


class _Torch:
    """What the node-wise calls use of torch, looked up once: a small call takes
    a few microseconds, of which an import statement was a noticeable part."""

    def __init__(self):
        import torch
        self.types = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
        self.f32, self.f64, self.i64, self.u8 = torch.float32, torch.float64, torch.int64, torch.uint8
        self.empty, self.on_stream = torch.empty, torch.cuda.stream
        self.device = torch._C._cuda_getDevice
        self.raw_stream, self.capturing = torch._C._cuda_getCurrentRawStream, torch._C._cuda_isCurrentStreamCapturing


_bits = None


def _torch_bits() -> _Torch:
    global _bits
    if _bits is None:
        _bits = _Torch()
    return _bits


def _scratch(nbytes: int, t, stream):
    """(pointer, bytes, owner) of a workspace for a call on t that brings none.
    A thread keeps one small buffer for each device and stream it calls on (what
    runs there is ordered; an allocation a call cost as much time as three
    launches).  Large ones, calls on a stream of their own and calls that are
    captured into a graph allocate: on the call's stream, so that the allocator
    hands the memory out again only behind the call's work, and in the graph's own
    pool."""
    b = _bits or _torch_bits()
    if stream is not None:
        with b.on_stream(stream):
            buf = b.empty(nbytes, dtype=b.u8, device=t.device)
    elif nbytes > _SCRATCH_MOST or b.capturing():
        buf = b.empty(nbytes, dtype=b.u8, device=t.device)
    else:
        kept = _scratch_of.__dict__
        dev = t.get_device()
        key = (dev, b.raw_stream(dev))
        mine = kept.get(key)
        if mine is None or mine[1] < nbytes:
            buf = b.empty(max(nbytes, 1 << 20), dtype=b.u8, device=t.device)
            mine = kept[key] = (buf.data_ptr(), buf.numel(), buf)
        return mine
    return buf.data_ptr(), buf.numel(), buf


def gnn_csr_build(n: int, src, dst, flags: int = CSR_GCN, stream=None) -> Csr:
    """Edge list (int32 device tensors) -> Csr with GCN weights (or mean
    weights with CSR_MEAN, plus the A^T weights when symmetrised)."""
    torch = _torch()
    dev = src.device
    m = int(src.numel())
    ws_bytes = ctypes.c_size_t()
    call("gnn_csr_build_workspace", n, m, flags, ctypes.byref(ws_bytes))
    ws = _workspace(ws_bytes.value, dev)
    cap = (2 * m if flags & CSR_SYMMETRIZE else m) + (n if flags & CSR_SELF_LOOPS else 0)
    rowptr = torch.empty(n + 1, dtype=torch.int64, device=dev)
    col = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
    val = torch.empty(max(cap, 1), dtype=torch.float32, device=dev)
    want_t = bool(flags & CSR_MEAN) and bool(flags & CSR_SYMMETRIZE)
    val_t = torch.empty(max(cap, 1), dtype=torch.float32, device=dev) if want_t else None
    out = GnnCsr(n, 0, 0, rowptr.data_ptr(), col.data_ptr(), val.data_ptr())
    out.val_t = _ptr(val_t)
    call("gnn_csr_build", n, m, _ptr(src), _ptr(dst), flags, cap, ctypes.byref(out), _ptr(ws),
         ws.numel(), _stream(stream))
    nnz = int(out.nnz)
    return Csr(n=n, nnz=nnz, symmetric=bool(out.symmetric), rowptr=rowptr, col=col[:nnz],
               val=val[:nnz], val_t=val_t[:nnz] if (val_t is not None and out.val_t) else None)


def gnn_csr_split(csr: Csr, split_len: int = 512, stream=None) -> Csr:
    """Attach a row-split plan: rows longer than split_len are cut into pieces
    of split_len entries (load balance for high-degree rows)."""
    torch = _torch()
    dev = csr.rowptr.device
    c = csr.c()
    ws_bytes = ctypes.c_size_t()
    call("gnn_csr_split_workspace", ctypes.byref(c), ctypes.byref(ws_bytes))
    ws = _workspace(ws_bytes.value, dev)
    nl, npc = ctypes.c_int32(), ctypes.c_int64()
    st = _stream(stream)
    call("gnn_csr_split_count", ctypes.byref(c), split_len, ctypes.byref(nl), ctypes.byref(npc),
         _ptr(ws), ws.numel(), st)
    nl, npc = nl.value, npc.value
    split = dict(long_rows=torch.empty(max(nl, 1), dtype=torch.int32, device=dev),
                 piece_ptr=torch.empty(nl + 1, dtype=torch.int64, device=dev),
                 piece_row=torch.empty(max(npc, 1), dtype=torch.int32, device=dev),
                 piece_beg=torch.empty(max(npc, 1), dtype=torch.int64, device=dev))
    out = Csr(csr.n, csr.nnz, csr.symmetric, csr.rowptr, csr.col, csr.val, split_len, nl, npc, split,
              csr.val_t)
    c2 = out.c()
    call("gnn_csr_split", ctypes.byref(c2), _ptr(ws), ws.numel(), st)
    return out


def gnn_spmm_workspace(csr: Csr, F: int) -> int:
    nb = ctypes.c_size_t()
    c = csr.c()
    call("gnn_spmm_workspace", ctypes.byref(c), F, ctypes.byref(nb))
    return nb.value


def spmm_ws(csr: Csr, F: int, device="cuda"):
    """A workspace tensor sized for the aggregation calls (or None)."""
    nb = gnn_spmm_workspace(csr, F)
    return _workspace(nb, device) if nb else None


def gnn_boundary_index(csr: Csr, P: int, rule: BitRule, base_bits: int, F: int,
                       stream=None) -> Boundary:
    torch = _torch()
    dev = csr.rowptr.device
    c = csr.c()
    ws_bytes = ctypes.c_size_t()
    call("gnn_boundary_workspace", ctypes.byref(c), P, ctypes.byref(ws_bytes))
    ws = _workspace(ws_bytes.value, dev)
    S, nc = ctypes.c_int64(), ctypes.c_int64()
    st = _stream(stream)
    call("gnn_boundary_count", ctypes.byref(c), P, ctypes.byref(S), ctypes.byref(nc), _ptr(ws),
         ws.numel(), st)
    S, nc, n = S.value, nc.value, csr.n
    i32, i64, u8, f32 = torch.int32, torch.int64, torch.uint8, torch.float32

    def e(k, dt):
        return torch.empty(max(k, 1), dtype=dt, device=dev)

    a = dict(part_start=e(P + 1, i64), send_start=e(P + 1, i64), slot_node=e(S, i32),
             col_remap=e(csr.nnz, i32), val_remap=e(csr.nnz, f32), local_cnt=e(n, i32),
             slot_rowptr=e(S + 1, i64), slot_col=e(nc, i32),
             slot_val=e(nc, f32), own_ptr=e(n + 1, i64), own_slot=e(S, i32), node_bits=e(n, u8),
             slot_bits=e(S, u8), slot_off=e(S + 1, i64))
    if csr.val_t is not None:
        a["val_remap_t"] = e(csr.nnz, f32)
    b = Boundary(P=P, n=n, n_slots=S, nnz_cut=nc, F=F, arrays=a)
    cb = b.c()
    call("gnn_boundary_index", ctypes.byref(c), ctypes.byref(rule.to_c()), base_bits, F,
         ctypes.byref(cb), _ptr(ws), ws.numel(), st)
    sizes = dict(part_start=P + 1, send_start=P + 1, slot_node=S, col_remap=csr.nnz,
                 val_remap=csr.nnz, local_cnt=n, slot_rowptr=S + 1, slot_col=nc, slot_val=nc, own_ptr=n + 1, own_slot=S,
                 node_bits=n, slot_bits=S, slot_off=S + 1, val_remap_t=csr.nnz)
    b.arrays = {k: v[:sizes[k]] for k, v in a.items()}
    return b


def gnn_boundary_long_slots(csr: Csr, bnd: Boundary, long_slot_len: int = 128, stream=None,
                            halo_order: bool = True) -> None:
    """Attach the list of slots with more than long_slot_len backward entries
    (their halo partials are then summed by a whole thread block each) and,
    with halo_order, the halo kernel's visiting order (slots by first
    backward entry)."""
    torch = _torch()
    dev = csr.rowptr.device
    c = csr.c()
    ws_bytes = ctypes.c_size_t()
    call("gnn_boundary_workspace", ctypes.byref(c), bnd.P, ctypes.byref(ws_bytes))
    ws = _workspace(ws_bytes.value, dev)
    cb = bnd.c()
    nl = ctypes.c_int32()
    st = _stream(stream)
    call("gnn_boundary_long_slots_count", ctypes.byref(cb), long_slot_len, ctypes.byref(nl), _ptr(ws),
         ws.numel(), st)
    bnd.arrays["long_slots"] = torch.empty(max(nl.value, 1), dtype=torch.int32, device=dev)
    bnd.long_slot_len, bnd.n_long_slots = long_slot_len, nl.value
    if halo_order:
        bnd.arrays["halo_order"] = torch.empty(max(bnd.n_slots, 1), dtype=torch.int32, device=dev)
    else:
        bnd.arrays.pop("halo_order", None)
    cb = bnd.c()
    call("gnn_boundary_long_slots", ctypes.byref(cb), _ptr(ws), ws.numel(), st)


def gnn_boundary_set_bits(csr: Csr, bnd: Boundary, rule: BitRule, base_bits: int, F: int,
                          stream=None) -> None:
    dev = csr.rowptr.device
    c = csr.c()
    ws_bytes = ctypes.c_size_t()
    call("gnn_boundary_workspace", ctypes.byref(c), bnd.P, ctypes.byref(ws_bytes))
    ws = _workspace(ws_bytes.value, dev)
    cb = bnd.c()
    call("gnn_boundary_set_bits", ctypes.byref(c), ctypes.byref(rule.to_c()), base_bits, F,
         ctypes.byref(cb), _ptr(ws), ws.numel(), _stream(stream))
    bnd.F = F


def gnn_slot_offsets(slot_bits, n_slots: int, F: int, stream=None):
    """Byte offsets [S+1] of each slot's packed row for feature width F."""
    torch = _torch()
    dev = slot_bits.device
    ws_bytes = ctypes.c_size_t()
    call("gnn_slot_offsets_workspace", n_slots, ctypes.byref(ws_bytes))
    ws = _workspace(ws_bytes.value, dev)
    off = torch.empty(n_slots + 1, dtype=torch.int64, device=dev)
    call("gnn_slot_offsets", _ptr(slot_bits), n_slots, F, _ptr(off), _ptr(ws), ws.numel(),
         _stream(stream))
    return off


def gnn_quant_pack(X, F: int, row_idx, n_rows: int, row_bits, row_off, seed: int, packed, meta,
                   stream=None) -> None:
    call("gnn_quant_pack", _ptr(X), X.stride(0), F, _ptr(row_idx), n_rows, _ptr(row_bits),
         _ptr(row_off), seed & 0xFFFFFFFF, _ptr(packed), _ptr(meta), _stream(stream))


def gnn_quant_pack_owned(bnd: Boundary, X, F: int, seed: int, packed, meta, slot_off=None,
                         stream=None) -> None:
    """Every slot's forward message (the bytes gnn_quant_pack writes for the
    slot rows), formed node by node: each boundary node's row is prepared once
    for all the partitions it is sent to."""
    cb = bnd.c(slot_off, F if slot_off is not None else None)
    call("gnn_quant_pack_owned", ctypes.byref(cb), _ptr(X), X.stride(0), F, seed & 0xFFFFFFFF,
         _ptr(packed), _ptr(meta), _stream(stream))


def gnn_quant_divide(a, b, q, stream=None) -> None:
    """q = a / b as the quantiser divides (fp32 tensors of equal size)."""
    call("gnn_quant_divide", _ptr(a), _ptr(b), _ptr(q), a.numel(), _stream(stream))


def gnn_dequant_unpack(packed, meta, row_off, row_bits, n_rows: int, F: int, out,
                       stream=None) -> None:
    call("gnn_dequant_unpack", _ptr(packed), _ptr(meta), _ptr(row_off), _ptr(row_bits), n_rows, F,
         _ptr(out), out.stride(0), _stream(stream))


def gnn_spmm_fwd_noalloc(csr: Csr, bnd: Optional[Boundary], H, F: int, packed=None, meta=None,
                         M=None, Mb=None, slot_off=None, stream=None) -> None:
    """gnn_spmm_fwd for callers that cannot allocate: scratch comes from a
    fixed device array inside the library (see the C header)."""
    c = csr.c()
    cb = bnd.c(slot_off, F if slot_off is not None else None) if bnd is not None else None
    call("gnn_spmm_fwd_noalloc", ctypes.byref(c), ctypes.byref(cb) if cb is not None else None,
         _ptr(H), H.stride(0), F, _ptr(packed), _ptr(meta), _ptr(M),
         M.stride(0) if M is not None else 0, _ptr(Mb), Mb.stride(0) if Mb is not None else 0,
         _stream(stream))


def _ws_args(csr: Csr, F: int, ws, device):
    if ws is None and csr.split_len:
        ws = spmm_ws(csr, F, device)
    return _ptr(ws), (ws.numel() * ws.element_size() if ws is not None else 0)


def gnn_spmm_fwd(csr: Csr, bnd: Optional[Boundary], H, F: int, packed=None, meta=None, M=None,
                 Mb=None, slot_off=None, ws=None, stream=None) -> None:
    c = csr.c()
    cb = bnd.c(slot_off, F if slot_off is not None else None) if bnd is not None else None
    wp, wn = _ws_args(csr, F, ws, H.device)
    call("gnn_spmm_fwd", ctypes.byref(c), ctypes.byref(cb) if cb is not None else None, _ptr(H),
         H.stride(0), F, _ptr(packed), _ptr(meta), _ptr(M), M.stride(0) if M is not None else 0,
         _ptr(Mb), Mb.stride(0) if Mb is not None else 0, wp, wn, _stream(stream))


def gnn_spmm_bwd(csr: Csr, bnd: Optional[Boundary], G, F: int, seed: int, packed_ws, meta_ws, dH,
                 slot_off=None, ws=None, stream=None) -> None:
    c = csr.c()
    cb = bnd.c(slot_off, F if slot_off is not None else None) if bnd is not None else None
    wp, wn = _ws_args(csr, F, ws, G.device)
    call("gnn_spmm_bwd", ctypes.byref(c), ctypes.byref(cb) if cb is not None else None, _ptr(G),
         G.stride(0), F, seed & 0xFFFFFFFF, _ptr(packed_ws), _ptr(meta_ws), _ptr(dH), dH.stride(0),
         wp, wn, _stream(stream))


def gnn_halo_quant_pack(bnd: Boundary, G, F: int, seed: int, packed, meta, slot_off=None,
                        stream=None) -> None:
    """Backward messages only: each slot's halo partial of G, quantised and
    packed."""
    cb = bnd.c(slot_off, F if slot_off is not None else None)
    call("gnn_halo_quant_pack", ctypes.byref(cb), _ptr(G), G.stride(0), F, seed & 0xFFFFFFFF,
         _ptr(packed), _ptr(meta), _stream(stream))


def gnn_quant_pack_slots(X, F: int, slot_node, s0: int, s1: int, slot_bits, slot_off, seed: int,
                         packed, meta, stream=None) -> None:
    """Forward messages of slots s0..s1-1 only (row key s), at their places in
    the slot-ordered buffer."""
    call("gnn_quant_pack_slots", _ptr(X), X.stride(0), F, _ptr(slot_node), int(s0), int(s1),
         _ptr(slot_bits), _ptr(slot_off), seed & 0xFFFFFFFF, _ptr(packed), _ptr(meta),
         _stream(stream))


def gnn_halo_quant_pack_slots(bnd: Boundary, G, F: int, s0: int, s1: int, seed: int, packed, meta,
                              slot_off=None, stream=None) -> None:
    """Backward messages of slots s0..s1-1 only."""
    cb = bnd.c(slot_off, F if slot_off is not None else None)
    call("gnn_halo_quant_pack_slots", ctypes.byref(cb), _ptr(G), G.stride(0), F, int(s0), int(s1),
         seed & 0xFFFFFFFF, _ptr(packed), _ptr(meta), _stream(stream))


def gnn_spmm_bwd_local(csr: Csr, bnd: Boundary, G, F: int, packed, meta, dH, slot_off=None,
                       ws=None, stream=None) -> None:
    """Owner-side backward aggregation: local transpose entries plus the
    dequantised backward messages in packed/meta."""
    c = csr.c()
    cb = bnd.c(slot_off, F if slot_off is not None else None)
    wp, wn = _ws_args(csr, F, ws, G.device)
    call("gnn_spmm_bwd_local", ctypes.byref(c), ctypes.byref(cb), _ptr(G), G.stride(0), F,
         _ptr(packed), _ptr(meta), _ptr(dH), dH.stride(0), wp, wn, _stream(stream))


def gnn_spmm_bwd_masked(csr: Csr, bnd: Optional[Boundary], G, F: int, seed: int, packed_ws, meta_ws,
                        H_mask, dZ, slot_off=None, ws=None, stream=None) -> None:
    """dZ (bf16, row stride >= ldz_for(F)) = bf16((A^T G) * 1[H_mask > 0])."""
    c = csr.c()
    cb = bnd.c(slot_off, F if slot_off is not None else None) if bnd is not None else None
    wp, wn = _ws_args(csr, F, ws, G.device)
    call("gnn_spmm_bwd_masked", ctypes.byref(c), ctypes.byref(cb) if cb is not None else None,
         _ptr(G), G.stride(0), F, seed & 0xFFFFFFFF, _ptr(packed_ws), _ptr(meta_ws), _ptr(H_mask),
         H_mask.stride(0) if H_mask is not None else 0, _ptr(dZ), dZ.stride(0), wp, wn,
         _stream(stream))


def gnn_spmm_bwd_local_masked(csr: Csr, bnd: Boundary, G, F: int, packed, meta, H_mask, dZ,
                              slot_off=None, ws=None, stream=None) -> None:
    """The owner-side half of gnn_spmm_bwd_masked: dZ = bf16((local A^T G +
    the dequantised messages in packed/meta) * 1[H_mask > 0])."""
    c = csr.c()
    cb = bnd.c(slot_off, F if slot_off is not None else None)
    wp, wn = _ws_args(csr, F, ws, G.device)
    call("gnn_spmm_bwd_local_masked", ctypes.byref(c), ctypes.byref(cb), _ptr(G), G.stride(0), F,
         _ptr(packed), _ptr(meta), _ptr(H_mask), H_mask.stride(0) if H_mask is not None else 0,
         _ptr(dZ), dZ.stride(0), wp, wn, _stream(stream))


def gnn_kernel_launches() -> int:
    """Kernels launched through the library by this process so far."""
    return int(load().gnn_kernel_launches())


def gnn_sync_check(stream=None) -> None:
    call("gnn_sync_check", _stream(stream))


# ---------------------------------------------------------------- dense transform and layers
def gnn_dense_workspace(n: int, F_in: int, F_out: int) -> int:
    nb = ctypes.c_size_t()
    call("gnn_dense_workspace", n, F_in, F_out, ctypes.byref(nb))
    return nb.value


def gnn_dense_fwd(Mb, n: int, F_in: int, W, F_out: int, relu: bool, H_out, ws=None,
                  stream=None) -> None:
    """H_out = act(Mb W) on tcgen05 (Mb, W bf16 tensors; H_out fp32)."""
    if ws is None:
        ws = _workspace(gnn_dense_workspace(n, F_in, F_out), Mb.device)
    call("gnn_dense_fwd", _ptr(Mb), Mb.stride(0), n, F_in, _ptr(W), F_out, int(relu), _ptr(H_out),
         H_out.stride(0), _ptr(ws), ws.numel(), _stream(stream))


def gnn_dense_bwd(Mb, n: int, F_in: int, W, F_out: int, dH_out, H_out, relu: bool, dM, dW,
                  ws=None, stream=None) -> None:
    if ws is None:
        ws = _workspace(gnn_dense_workspace(n, F_in, F_out), Mb.device)
    call("gnn_dense_bwd", _ptr(Mb), Mb.stride(0), n, F_in, _ptr(W), F_out, _ptr(dH_out),
         dH_out.stride(0), _ptr(H_out), H_out.stride(0) if H_out is not None else 0, int(relu),
         _ptr(dM), dM.stride(0) if dM is not None else 0, _ptr(dW), _ptr(ws), ws.numel(),
         _stream(stream))


def gnn_dense_bwd_z(Mb, n: int, F_in: int, W, F_out: int, dZ, dM, dW, ws=None, stream=None) -> None:
    if ws is None:
        ws = _workspace(gnn_dense_workspace(n, F_in, F_out), Mb.device)
    call("gnn_dense_bwd_z", _ptr(Mb), Mb.stride(0), n, F_in, _ptr(W), F_out, _ptr(dZ), dZ.stride(0),
         _ptr(dM), dM.stride(0) if dM is not None else 0, _ptr(dW), _ptr(ws), ws.numel(),
         _stream(stream))


def gnn_layer_workspace(csr: Csr, F_in: int, F_out: int) -> int:
    nb = ctypes.c_size_t()
    c = csr.c()
    call("gnn_layer_workspace", ctypes.byref(c), F_in, F_out, ctypes.byref(nb))
    return nb.value


def gnn_layer_fwd(csr: Csr, bnd: Optional[Boundary], H_in, F_in: int, W, F_out: int, relu: bool,
                  seed: int, packed_ws, meta_ws, Mb, H_out, slot_off=None, ws=None,
                  stream=None) -> None:
    c = csr.c()
    cb = bnd.c(slot_off, F_in if slot_off is not None else None) if bnd is not None else None
    if ws is None:
        ws = _workspace(gnn_layer_workspace(csr, F_in, F_out), H_in.device)
    call("gnn_layer_fwd", ctypes.byref(c), ctypes.byref(cb) if cb is not None else None, _ptr(H_in),
         H_in.stride(0), F_in, _ptr(W), F_out, int(relu), seed & 0xFFFFFFFF, _ptr(packed_ws),
         _ptr(meta_ws), _ptr(Mb), Mb.stride(0), _ptr(H_out), H_out.stride(0), _ptr(ws), ws.numel(),
         _stream(stream))


def gnn_layer_bwd(csr: Csr, bnd: Optional[Boundary], dH_out, H_out, relu: bool, Mb, W, F_in: int,
                  F_out: int, seed: int, packed_ws, meta_ws, dW, dH_in=None, slot_off=None,
                  ws=None, stream=None) -> None:
    c = csr.c()
    cb = bnd.c(slot_off, F_in if slot_off is not None else None) if bnd is not None else None
    if ws is None:
        ws = _workspace(gnn_layer_workspace(csr, F_in, F_out), dH_out.device)
    call("gnn_layer_bwd", ctypes.byref(c), ctypes.byref(cb) if cb is not None else None,
         _ptr(dH_out), dH_out.stride(0), _ptr(H_out), H_out.stride(0) if H_out is not None else 0,
         int(relu), _ptr(Mb), Mb.stride(0), _ptr(W), F_in, F_out, seed & 0xFFFFFFFF, _ptr(packed_ws),
         _ptr(meta_ws), _ptr(dW), _ptr(dH_in), dH_in.stride(0) if dH_in is not None else 0,
         _ptr(ws), ws.numel(), _stream(stream))


def gnn_layer_fwd_async(csr: Csr, bnd: Boundary, H_in, F_in: int, W, F_out: int, relu: bool,
                        seed: int, packed_prev, meta_prev, packed_next, meta_next, Mb, H_out,
                        aux, slot_off=None, ws=None, stream=None) -> None:
    """Forward layer of an asynchronous epoch: remote sources read the
    previous epoch's messages; this epoch's are packed on ``aux`` meanwhile."""
    c = csr.c()
    cb = bnd.c(slot_off, F_in if slot_off is not None else None)
    if ws is None:
        ws = _workspace(gnn_layer_workspace(csr, F_in, F_out), H_in.device)
    call("gnn_layer_fwd_async", ctypes.byref(c), ctypes.byref(cb), _ptr(H_in), H_in.stride(0), F_in,
         _ptr(W), F_out, int(relu), seed & 0xFFFFFFFF, _ptr(packed_prev), _ptr(meta_prev),
         _ptr(packed_next), _ptr(meta_next), _ptr(Mb), Mb.stride(0), _ptr(H_out), H_out.stride(0),
         _ptr(ws), ws.numel(), _stream(stream), aux.cuda_stream)


def gnn_layer_bwd_async(csr: Csr, bnd: Boundary, dH_out, H_out, relu: bool, Mb, W, F_in: int,
                        F_out: int, seed: int, packed_prev, meta_prev, packed_next, meta_next, dW,
                        dH_in, aux, slot_off=None, ws=None, stream=None) -> None:
    c = csr.c()
    cb = bnd.c(slot_off, F_in if slot_off is not None else None)
    if ws is None:
        ws = _workspace(gnn_layer_workspace(csr, F_in, F_out), dH_out.device)
    call("gnn_layer_bwd_async", ctypes.byref(c), ctypes.byref(cb), _ptr(dH_out), dH_out.stride(0),
         _ptr(H_out), H_out.stride(0) if H_out is not None else 0, int(relu), _ptr(Mb), Mb.stride(0),
         _ptr(W), F_in, F_out, seed & 0xFFFFFFFF, _ptr(packed_prev), _ptr(meta_prev),
         _ptr(packed_next), _ptr(meta_next), _ptr(dW), _ptr(dH_in),
         dH_in.stride(0) if dH_in is not None else 0, _ptr(ws), ws.numel(), _stream(stream),
         aux.cuda_stream)


# ---------------------------------------------------------------- transform-first layers
def gnn_layer_tf_workspace(csr: Csr, F_in: int, F_out: int) -> int:
    nb = ctypes.c_size_t()
    c = csr.c()
    call("gnn_layer_tf_workspace", ctypes.byref(c), F_in, F_out, ctypes.byref(nb))
    return nb.value


def gnn_layer_fwd_tf(csr: Csr, bnd: Optional[Boundary], H_in, F_in: int, W, F_out: int,
                     relu: bool, seed: int, packed_ws, meta_ws, Hb, Y, H_out, slot_off=None,
                     ws=None, stream=None) -> None:
    """Y = bf16(H_in) W, messages from Y, H_out = act(A Y) (aggregation at
    width F_out; bnd offsets for F_out)."""
    c = csr.c()
    cb = bnd.c(slot_off, F_out if slot_off is not None else None) if bnd is not None else None
    if ws is None:
        ws = _workspace(gnn_layer_tf_workspace(csr, F_in, F_out), H_in.device)
    call("gnn_layer_fwd_tf", ctypes.byref(c), ctypes.byref(cb) if cb is not None else None,
         _ptr(H_in), H_in.stride(0), F_in, _ptr(W), F_out, int(relu), seed & 0xFFFFFFFF,
         _ptr(packed_ws), _ptr(meta_ws), _ptr(Hb), Hb.stride(0), _ptr(Y), Y.stride(0), _ptr(H_out),
         H_out.stride(0), _ptr(ws), ws.numel(), _stream(stream))


def gnn_layer_bwd_tf(csr: Csr, bnd: Optional[Boundary], dH_out, H_out, relu: bool, Hb, W,
                     F_in: int, F_out: int, seed: int, packed_ws, meta_ws, dW, dH_in=None,
                     slot_off=None, ws=None, stream=None) -> None:
    c = csr.c()
    cb = bnd.c(slot_off, F_out if slot_off is not None else None) if bnd is not None else None
    if ws is None:
        ws = _workspace(gnn_layer_tf_workspace(csr, F_in, F_out), dH_out.device)
    call("gnn_layer_bwd_tf", ctypes.byref(c), ctypes.byref(cb) if cb is not None else None,
         _ptr(dH_out), dH_out.stride(0), _ptr(H_out), H_out.stride(0) if H_out is not None else 0,
         int(relu), _ptr(Hb), Hb.stride(0), _ptr(W), F_in, F_out, seed & 0xFFFFFFFF,
         _ptr(packed_ws), _ptr(meta_ws), _ptr(dW), _ptr(dH_in),
         dH_in.stride(0) if dH_in is not None else 0, _ptr(ws), ws.numel(), _stream(stream))


# ---------------------------------------------------------------- cluster-blocked aggregation
@dataclass
class Blocked:
    T: int
    n_rb: int
    n_tiles: int
    n_entries: int
    arrays: dict
    residual: Csr

    def c(self) -> GnnBlocked:
        a = self.arrays
        b = GnnBlocked()
        b.T, b.n_rb, b.n_tiles, b.n_entries = self.T, self.n_rb, self.n_tiles, self.n_entries
        for k in ("rb_tile_ptr", "tile_cb", "tile_ptr", "tile_rowptr", "ent_col", "ent_val",
                  "res_local_cnt"):
            setattr(b, k, _ptr(a.get(k)))
        b.residual = self.residual.c()
        return b


def gnn_blocked_build(csr: Csr, bnd: Optional[Boundary], min_entries: int = 1024, T: int = 128,
                      split_len: int = 128, stream=None) -> Blocked:
    """Dense T x T tiles (at least min_entries entries) and the residual CSR,
    with a split plan of split_len entries for the residual (0: none)."""
    torch = _torch()
    dev = csr.rowptr.device
    c = csr.c()
    cb = bnd.c() if bnd is not None else None
    pb = ctypes.byref(cb) if cb is not None else None
    nb = ctypes.c_size_t()
    call("gnn_blocked_workspace", ctypes.byref(c), pb, T, min_entries, ctypes.byref(nb))
    ws = _workspace(nb.value, dev)
    nt, ne, nr = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    st = _stream(stream)
    call("gnn_blocked_count", ctypes.byref(c), pb, T, min_entries, ctypes.byref(nt), ctypes.byref(ne),
         ctypes.byref(nr), _ptr(ws), ws.numel(), st)
    nt, ne, nr, n = nt.value, ne.value, nr.value, csr.n
    n_rb = (n + T - 1) // T

    def e(k, dt):
        return torch.empty(max(k, 1), dtype=dt, device=dev)

    a = dict(rb_tile_ptr=e(n_rb + 1, torch.int64), tile_cb=e(nt, torch.int32),
             tile_ptr=e(nt + 1, torch.int64), tile_rowptr=e(nt * (T + 1), torch.int32),
             ent_col=e(ne + 16, torch.uint8), ent_val=e(ne, torch.float32))
    if bnd is not None:
        a["res_local_cnt"] = e(n, torch.int32)
    res = Csr(n=n, nnz=nr, symmetric=False, rowptr=e(n + 1, torch.int64), col=e(nr, torch.int32),
              val=e(nr, torch.float32))
    bl = Blocked(T=T, n_rb=n_rb, n_tiles=nt, n_entries=ne, arrays=a, residual=res)
    out = bl.c()
    call("gnn_blocked_build", ctypes.byref(c), pb, T, min_entries, ctypes.byref(out), _ptr(ws), ws.numel(), st)
    res.col, res.val = res.col[:nr], res.val[:nr]
    if split_len and nr > 0:
        bl.residual = gnn_csr_split(res, split_len, stream)
    return bl


def _blocked_ws(bl: Blocked, F: int, device, ws):
    if ws is not None:
        return ws
    nb = ctypes.c_size_t()
    b = bl.c()
    call("gnn_blocked_spmm_workspace", ctypes.byref(b), F, ctypes.byref(nb))
    return _workspace(nb.value, device)


def gnn_spmm_fwd_blocked(csr: Csr, bnd: Optional[Boundary], bl: Blocked, H, F: int, packed=None,
                         meta=None, M=None, Mb=None, slot_off=None, ws=None, stream=None) -> None:
    c = csr.c()
    cb = bnd.c(slot_off, F if slot_off is not None else None) if bnd is not None else None
    b = bl.c()
    ws = _blocked_ws(bl, F, H.device, ws)
    call("gnn_spmm_fwd_blocked", ctypes.byref(c), ctypes.byref(cb) if cb is not None else None,
         ctypes.byref(b), _ptr(H), H.stride(0), F, _ptr(packed), _ptr(meta), _ptr(M),
         M.stride(0) if M is not None else 0, _ptr(Mb), Mb.stride(0) if Mb is not None else 0,
         _ptr(ws), ws.numel(), _stream(stream))


def gnn_spmm_bwd_blocked(csr: Csr, bnd: Optional[Boundary], bl: Blocked, G, F: int, seed: int,
                         packed_ws=None, meta_ws=None, H_mask=None, dH=None, dZ=None, slot_off=None,
                         ws=None, stream=None) -> None:
    c = csr.c()
    cb = bnd.c(slot_off, F if slot_off is not None else None) if bnd is not None else None
    b = bl.c()
    ws = _blocked_ws(bl, F, G.device, ws)
    call("gnn_spmm_bwd_blocked", ctypes.byref(c), ctypes.byref(cb) if cb is not None else None,
         ctypes.byref(b), _ptr(G), G.stride(0), F, seed & 0xFFFFFFFF, _ptr(packed_ws), _ptr(meta_ws),
         _ptr(H_mask), H_mask.stride(0) if H_mask is not None else 0, _ptr(dH),
         dH.stride(0) if dH is not None else 0, _ptr(dZ), dZ.stride(0) if dZ is not None else 0,
         _ptr(ws), ws.numel(), _stream(stream))


# ---------------------------------------------------------------- attention aggregator
def gnn_gat_index(csr: Csr, bnd: Optional[Boundary], stream=None):
    """Position maps (tpos [nnz], spos [nnz_cut] or None) for the backward."""
    torch = _torch()
    dev = csr.rowptr.device
    tpos = torch.empty(max(csr.nnz, 1), dtype=torch.int64, device=dev)
    spos = torch.empty(max(bnd.nnz_cut, 1), dtype=torch.int64, device=dev) if bnd is not None else None
    c = csr.c()
    cb = bnd.c() if bnd is not None else None
    call("gnn_gat_index", ctypes.byref(c), ctypes.byref(cb) if cb is not None else None, _ptr(tpos),
         _ptr(spos), _stream(stream))
    return tpos, spos


def gnn_gat_workspace(csr: Csr, bnd: Optional[Boundary], F_in: int, F_out: int) -> int:
    nb = ctypes.c_size_t()
    c = csr.c()
    cb = bnd.c() if bnd is not None else None
    call("gnn_gat_workspace", ctypes.byref(c), ctypes.byref(cb) if cb is not None else None, F_in,
         F_out, ctypes.byref(nb))
    return nb.value


def _gat_bnd(bnd, slot_off, F_out):
    return bnd.c(slot_off, F_out if slot_off is not None else None) if bnd is not None else None


def gnn_gat_layer_fwd(csr: Csr, bnd: Optional[Boundary], H_in, F_in: int, W, F_out: int, a_l, a_r,
                      relu: bool, seed: int, packed, meta, Hb, Y, alpha, H_out, slot_off=None,
                      ws=None, stream=None) -> None:
    c = csr.c()
    cb = _gat_bnd(bnd, slot_off, F_out)
    if ws is None:
        ws = _workspace(gnn_gat_workspace(csr, bnd, F_in, F_out), H_in.device)
    call("gnn_gat_layer_fwd", ctypes.byref(c), ctypes.byref(cb) if cb is not None else None,
         _ptr(H_in), H_in.stride(0), F_in, _ptr(W), F_out, _ptr(a_l), _ptr(a_r), int(relu),
         seed & 0xFFFFFFFF, _ptr(packed), _ptr(meta), _ptr(Hb), Hb.stride(0), _ptr(Y), Y.stride(0),
         _ptr(alpha), _ptr(H_out), H_out.stride(0), _ptr(ws), ws.numel(), _stream(stream))


def gnn_gat_layer_bwd(csr: Csr, bnd: Optional[Boundary], tpos, spos, dH_out, H_out, relu: bool, Hb,
                      Y, alpha, packed_fwd, meta_fwd, W, a_l, a_r, F_in: int, F_out: int, seed: int,
                      packed_ws, meta_ws, dW, da_l, da_r, dH_in=None, g_out=None, slot_off=None,
                      ws=None, stream=None) -> None:
    c = csr.c()
    cb = _gat_bnd(bnd, slot_off, F_out)
    if ws is None:
        ws = _workspace(gnn_gat_workspace(csr, bnd, F_in, F_out), dH_out.device)
    call("gnn_gat_layer_bwd", ctypes.byref(c), ctypes.byref(cb) if cb is not None else None,
         _ptr(tpos), _ptr(spos), _ptr(dH_out), dH_out.stride(0), _ptr(H_out),
         H_out.stride(0) if H_out is not None else 0, int(relu), _ptr(Hb), Hb.stride(0), _ptr(Y),
         Y.stride(0), _ptr(alpha), _ptr(packed_fwd), _ptr(meta_fwd), _ptr(W), _ptr(a_l), _ptr(a_r),
         F_in, F_out, seed & 0xFFFFFFFF, _ptr(packed_ws), _ptr(meta_ws), _ptr(dW), _ptr(da_l),
         _ptr(da_r), _ptr(dH_in), dH_in.stride(0) if dH_in is not None else 0, _ptr(g_out),
         _ptr(ws), ws.numel(), _stream(stream))


# ---------------------------------------------------------------- node-wise block
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "sigmoid": 4}


def _type(t) -> int:
    """The library's number of a tensor's type (-1, which it refuses, for one it does not have)."""
    return (_bits or _torch_bits()).types.get(t.dtype, -1)


def _rows(t, n: int, F: int, what: str) -> int:
    """Row stride of a matrix that holds n rows of F columns, each contiguous."""
    shape = t.shape
    if len(shape) == 2:
        ld, step = t.stride()
        if shape[0] >= n and shape[1] >= F and (step == 1 or shape[1] == 1):
            if t.is_cuda:
                return ld
            raise ValueError(f"{what}: needs a CUDA tensor")
    raise ValueError(f"{what}: needs a [>={n}, >={F}] matrix with contiguous rows, got "
                     f"{tuple(shape)} with strides {t.stride()}")


def _f32(t, count: int, what: str):
    """Pointer of a contiguous fp32 vector (None for None)."""
    if t is None:
        return None
    if t.dtype is (_bits or _torch_bits()).f32 and t.is_cuda and t.numel() >= count and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{what}: needs a contiguous fp32 CUDA tensor of {count} elements")


def _current(t, stream) -> int:
    """The raw stream of a call on t: `stream`, or the current one.  The launch
    goes to the current device, so t has to be there."""
    b = _bits or _torch_bits()
    dev = t.get_device()
    if dev != b.device():
        raise ValueError(f"tensors on cuda:{dev}, but the current device is cuda:{b.device()}: set it with torch.cuda.device")
    return b.raw_stream(dev) if stream is None else stream.cuda_stream


def _act(act: str) -> int:
    k = ACTS.get(act)
    if k is None:
        raise ValueError(f"act: one of {sorted(ACTS)}, got {act!r}")
    return k


def _seg(seg_start):
    if seg_start is None:
        return None, 1
    k = seg_start.numel()
    if seg_start.dtype is (_bits or _torch_bits()).i64 and seg_start.is_cuda and seg_start.dim() == 1 and k >= 2 and \
            seg_start.is_contiguous():
        return seg_start.data_ptr(), k - 1
    raise ValueError("seg_start: needs a contiguous int64 CUDA tensor of n_seg + 1 elements")


def _ws(ws, nbytes: int, t, stream):
    """(pointer, bytes, owner) of the caller's workspace, or of one of the binding's."""
    if ws is None:
        return _scratch(nbytes, t, stream)
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("ws: needs a contiguous CUDA tensor")
    return ws.data_ptr(), ws.numel(), ws


@functools.lru_cache(maxsize=1024)
def gnn_group_norm_workspace(n: int, C: int, groups: int, n_seg: int = 1) -> int:
    nb = ctypes.c_size_t()
    call("gnn_group_norm_workspace", n, C, groups, n_seg, ctypes.byref(nb))
    return nb.value


def gnn_group_norm_fwd(X, n: int, C: int, groups: int, Y, mean, rstd, seg_start=None, gamma=None, beta=None,
                       eps: float = 1e-5, act: str = "none", ws=None, stream=None) -> None:
    """Y = act(gamma (x - mean) rstd + beta) over the segments of rows that
    seg_start cuts (``Boundary.part_start`` fits; None: all rows are one);
    mean and rstd [n_seg, groups] are kept for the backward."""
    seg, n_seg = _seg(seg_start)
    ldx, ldy = _rows(X, n, C, "X"), _rows(Y, n, C, "Y")
    at, size, ws = _ws(ws, gnn_group_norm_workspace(n, C, groups, n_seg), X, stream)
    call("gnn_group_norm_fwd", X.data_ptr(), ldx, _type(X), n, C, groups, seg, n_seg, _f32(gamma, C, "gamma"),
         _f32(beta, C, "beta"), eps, _act(act), Y.data_ptr(), ldy, _type(Y),
         _f32(mean, n_seg * groups, "mean"), _f32(rstd, n_seg * groups, "rstd"), at, size, _current(X, stream))


def gnn_group_norm_bwd(dY, X, n: int, C: int, groups: int, mean, rstd, dX, dgamma=None, dbeta=None,
                       seg_start=None, gamma=None, beta=None, act: str = "none", ws=None,
                       stream=None) -> None:
    """dX, dgamma and dbeta of gnn_group_norm_fwd from dY, X and the kept
    mean and rstd (dY has Y's type, dX has X's)."""
    seg, n_seg = _seg(seg_start)
    ldx, ldy, lddx = _rows(X, n, C, "X"), _rows(dY, n, C, "dY"), _rows(dX, n, C, "dX")
    if dX.dtype is not X.dtype:
        raise ValueError("dX: needs X's type")
    at, size, ws = _ws(ws, gnn_group_norm_workspace(n, C, groups, n_seg), X, stream)
    call("gnn_group_norm_bwd", dY.data_ptr(), ldy, _type(dY), X.data_ptr(), ldx, _type(X), n, C, groups, seg, n_seg,
         _f32(gamma, C, "gamma"), _f32(beta, C, "beta"), _act(act), _f32(mean, n_seg * groups, "mean"),
         _f32(rstd, n_seg * groups, "rstd"), dX.data_ptr(), lddx, _f32(dgamma, C, "dgamma"),
         _f32(dbeta, C, "dbeta"), at, size, _current(X, stream))


@functools.lru_cache(maxsize=1024)
def gnn_gated_workspace(n: int, F_in: int, F_mid: int):
    """Workspace bytes of gnn_gated_fwd and gnn_gated_bwd."""
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    call("gnn_gated_workspace", n, F_in, F_mid, ctypes.byref(f), ctypes.byref(b))
    return f.value, b.value


def _one_type(X, *others) -> int:
    d = X.dtype
    for t in others:
        if t is not None and t.dtype is not d:
            raise ValueError(f"operands of one type are needed: X has {d}, another {t.dtype}")
    return _type(X)


def gnn_gated_fwd(X, n: int, F_in: int, Wg, Wu, F_mid: int, H, act: str = "silu", ws=None,
                  stream=None) -> None:
    """H = act(X Wg) * (X Wu) on tcgen05 (X, Wg, Wu, H of one type, bf16 or
    fp16; Wg, Wu [F_in, F_mid]).  It needs no workspace."""
    t = _one_type(X, Wg, Wu, H)
    call("gnn_gated_fwd", X.data_ptr(), _rows(X, n, F_in, "X"), t, n, F_in, Wg.data_ptr(), _rows(Wg, F_in, F_mid, "Wg"),
         Wu.data_ptr(), _rows(Wu, F_in, F_mid, "Wu"), F_mid, _act(act), H.data_ptr(), _rows(H, n, F_mid, "H"),
         _ptr(ws), ws.numel() if ws is not None else 0, _current(X, stream))


def gnn_gated_bwd(dH, X, n: int, F_in: int, Wg, Wu, F_mid: int, dX=None, dWg=None, dWu=None,
                  act: str = "silu", ws=None, stream=None) -> None:
    """dX, dWg and dWu of gnn_gated_fwd (X's type; the projections are
    recomputed).  dH has X's type or fp32."""
    t = _one_type(X, Wg, Wu, dX, dWg, dWu)
    at, size, ws = _ws(ws, gnn_gated_workspace(n, F_in, F_mid)[1], X, stream)
    call("gnn_gated_bwd", _ptr(dH), _rows(dH, n, F_mid, "dH"), _type(dH), _ptr(X), _rows(X, n, F_in, "X"), t, n,
         F_in, _ptr(Wg), _rows(Wg, F_in, F_mid, "Wg"), _ptr(Wu), _rows(Wu, F_in, F_mid, "Wu"), F_mid, _act(act),
         _ptr(dX), _rows(dX, n, F_in, "dX") if dX is not None else 0,
         _ptr(dWg), _rows(dWg, F_in, F_mid, "dWg") if dWg is not None else 0,
         _ptr(dWu), _rows(dWu, F_in, F_mid, "dWu") if dWu is not None else 0,
         at, size, _current(X, stream))


NORMS = {"none": 0, "rms": 1, "layer": 2}
# the calls' arguments as a struct's bytes, in which None is a zero
_RESIDUAL_FWD, _RESIDUAL_BWD = _abi.RESIDUAL_FWD.pack, _abi.RESIDUAL_BWD.pack


def _norm(kind: str, what: str) -> int:
    k = NORMS.get(kind)
    if k is None:
        raise ValueError(f"{what}: one of {sorted(NORMS)}, got {kind!r}")
    return k


def _gate(gate, n: int, C: int, what: str):
    """(pointer, stride, columns) of a gate: a matrix, or one value a row."""
    if gate is None:
        return 0, 0, 0
    if gate.dim() == 1:
        if gate.numel() < n or not gate.is_cuda:
            raise ValueError(f"{what}: needs a CUDA tensor of {n} values or a matrix")
        return gate.data_ptr(), gate.stride()[0], 1
    return gate.data_ptr(), _rows(gate, n, C, what), C


def _scale(scale, C: int):
    if scale is None:
        return 0, 0
    k = scale.numel()
    if k != 1 and k != C:
        raise ValueError(f"scale: needs 1 or {C} values, got {k}")
    return _f32(scale, k, "scale"), k


def _types(what, t, *others):
    for name, o in others:
        if o is not None and o.dtype is not t.dtype:
            raise ValueError(f"{name}: needs {what}'s type {t.dtype}, got {o.dtype}")


def _place(t, n: int, C: int, what: str):
    return (0, 0) if t is None else (t.data_ptr(), _rows(t, n, C, what))


@functools.lru_cache(maxsize=1024)
def gnn_residual_norm_workspace(n: int, C: int) -> int:
    """Workspace bytes of gnn_residual_norm_bwd."""
    nb = ctypes.c_size_t()
    call("gnn_residual_norm_workspace", n, C, ctypes.byref(nb))
    return nb.value


def gnn_residual_norm_fwd(B, R, n: int, C: int, H, Y=None, stats=None, gate=None, gate_act: str = "sigmoid",
                          post: str = "rms", w_post=None, b_post=None, scale=None, pre: str = "rms", w_pre=None,
                          b_pre=None, eps: float = 1e-6, stream=None) -> None:
    """H = R + scale act(gate) (w_post norm(B) + b_post) and Y = w_pre norm(H) +
    b_pre by rows (norms "none", "rms", "layer").  gate: [n, C] or one value a
    row [n], of B's type; scale: fp32, C values or one; stats (fp32 [n, 4]) is
    kept for the backward.  B None: H = R (H may be None), Y is R's norm."""
    b = _bits or _torch_bits()
    rt = R.dtype
    if H is not None and H.dtype is not rt:
        raise ValueError(f"H: needs R's type {rt}, got {H.dtype}")
    if gate is not None:
        _types("B", R if B is None else B, ("gate", gate))
    at_b, ldb = _place(B, n, C, "B")
    at_g, ldg, gate_cols = _gate(gate, n, C, "gate")
    at_s, scale_cols = _scale(scale, C)
    at_h, ldh = _place(H, n, C, "H")
    at_y, ldy = _place(Y, n, C, "Y")
    types = b.types
    rt = types.get(rt, -1)
    yt = rt if Y is None else types.get(Y.dtype, -1)
    bt = types.get(B.dtype, -1) if B is not None else rt if rt == yt else 0
    if Y is None:
        yt = bt
    call("gnn_residual_norm_fwd_struct", _RESIDUAL_FWD(
        at_b, ldb, bt, R.data_ptr(), _rows(R, n, C, "R"), rt, at_g, ldg, gate_cols, _act(gate_act), n, C,
        _norm(post, "post") if B is not None else 0, w_post is not None and _f32(w_post, C, "w_post"),
        b_post is not None and _f32(b_post, C, "b_post"), at_s, scale_cols, _norm(pre, "pre"),
        w_pre is not None and _f32(w_pre, C, "w_pre"), b_pre is not None and _f32(b_pre, C, "b_pre"), eps, at_h, ldh, at_y, ldy,
        yt, stats is not None and _f32(stats, 4 * n, "stats"), _current(R, stream)))


def gnn_residual_norm_bwd(dH, dY, B, H, n: int, C: int, stats, dR=None, dB=None, gate=None, dgate=None,
                          gate_act: str = "sigmoid", post: str = "rms", w_post=None, b_post=None, scale=None,
                          pre: str = "rms", w_pre=None, dw_post=None, db_post=None, dscale=None, dw_pre=None,
                          db_pre=None, ws=None, stream=None) -> None:
    """Gradients of gnn_residual_norm_fwd from dH and dY (one may be None), with
    B, H, gate, weights and stats as they were there; each output may be None."""
    S = H if H is not None else dH
    if S is None:
        raise ValueError("H: needed where there is no dH")
    _types("B", S if B is None else B, ("gate", gate), ("dgate", dgate), ("dB", dB))
    _types("H", S, ("dH", dH), ("dR", dR))
    at_dh, lddh = _place(dH, n, C, "dH")
    at_dy, lddy = _place(dY, n, C, "dY")
    at_b, ldb = _place(B, n, C, "B")
    at_h, ldh = _place(H, n, C, "H")
    at_dr, lddr = _place(dR, n, C, "dR")
    at_db, lddb = _place(dB, n, C, "dB")
    at_g, ldg, gate_cols = _gate(gate, n, C, "gate")
    at_dg, lddg, dgate_cols = _gate(dgate, n, C, "dgate")
    if dgate is not None and dgate_cols != gate_cols:
        raise ValueError("dgate: needs the gate's shape")
    at_s, scale_cols = _scale(scale, C)
    bt = _type(B) if B is not None else _type(S) if dY is None or S.dtype is dY.dtype else 0
    at, size, ws = _ws(ws, gnn_residual_norm_workspace(n, C), S, stream)
    vec = lambda t, k, what: t is not None and _f32(t, k, what)  # noqa: E731
    call("gnn_residual_norm_bwd_struct", _RESIDUAL_BWD(
        at_dh, lddh, at_dy, lddy, bt if dY is None else _type(dY), at_b, ldb, bt, at_h, ldh, _type(S), at_g, ldg, gate_cols,
        _act(gate_act), n, C, _norm(post, "post") if B is not None else 0, vec(w_post, C, "w_post"), vec(b_post, C, "b_post"),
        at_s, scale_cols, _norm(pre, "pre"), vec(w_pre, C, "w_pre"), vec(stats, 4 * n, "stats"), at_dr, lddr, at_db, lddb,
        at_dg, lddg, vec(dw_post, C, "dw_post"), vec(db_post, C, "db_post"), vec(dscale, scale_cols, "dscale"),
        vec(dw_pre, C, "dw_pre"), vec(db_pre, C, "db_pre"), at, size, _current(S, stream)))


class AdamwTensors:
    """The tensors of an optimiser, checked once: lists of parameters (fp32 or
    bf16, updated in place), their gradients, m, v and, with 8-bit states
    (torch.float8_e4m3fn m and v), the scales m_scale and v_scale (fp32, one
    per 256 elements of a tensor); copies (bf16, optional, None for a tensor
    without one) receive the updated parameters.  All are contiguous CUDA tensors and stay the caller's."""

    def __init__(self, params, grads, m, v, m_scale=None, v_scale=None, copies=None):
        import torch
        k = len(params)
        self.count = k
        lists = dict(params=params, grads=grads, m=m, v=v, m_scale=m_scale, v_scale=v_scale, copies=copies)
        for name, ts in lists.items():
            if ts is not None and len(ts) != k:
                raise ValueError(f"{name}: {len(ts)} tensors for {k} parameters")
        self.state_bits = 8 if k and m[0].dtype == torch.float8_e4m3fn else 32
        if self.state_bits == 8 and (m_scale is None or v_scale is None):
            raise ValueError("8-bit states need m_scale and v_scale")
        state = torch.float8_e4m3fn if self.state_bits == 8 else torch.float32
        want = dict(params=params[0].dtype if k else torch.float32, grads=grads[0].dtype if k else torch.float32,
                    m=state, v=state, m_scale=torch.float32, v_scale=torch.float32, copies=torch.bfloat16)
        for name, ts in lists.items():
            for i, t in enumerate(ts or ()):
                if t is None and name == "copies":
                    continue
                n = params[i].numel()
                size = -(-n // 256) if name.endswith("scale") else n
                if t.device != params[0].device:
                    raise ValueError(f"{name}[{i}]: on {t.device}, params[0] on {params[0].device}")
                if t.dtype != want[name] or t.numel() != size or not t.is_contiguous() or t.device.type != "cuda":
                    raise ValueError(f"{name}[{i}]: needs a contiguous {want[name]} CUDA tensor of {size} elements")
        places = [p.data_ptr() for p in params if p.numel()]
        if len(set(places)) < len(places):
            raise ValueError("params: a tensor is listed twice")
        self.param_type = _type(params[0]) if k else 0
        self.grad_type = _type(grads[0]) if k else 0
        self.device = params[0].device if k else None
        self._keep = {name: list(ts) for name, ts in lists.items() if ts is not None}
        at = lambda ts, i: None if ts is None or ts[i] is None else ts[i].data_ptr()  # noqa: E731
        self.c = (GnnAdamwTensor * max(k, 1))(*[
            GnnAdamwTensor(at(params, i), at(grads, i), at(m, i), at(v, i),
                           at(m_scale, i) if self.state_bits == 8 else None,
                           at(v_scale, i) if self.state_bits == 8 else None, at(copies, i), params[i].numel())
            for i in range(k)])


def adamw_state(device="cuda"):
    """A new optimiser's step state: {steps, beta1^steps, beta2^steps, steps
    skipped} as a device fp64 tensor (save and load it with the weights)."""
    import torch
    return torch.tensor([0.0, 1.0, 1.0, 0.0], dtype=torch.float64, device=device)


@functools.lru_cache(maxsize=1)
def gnn_adamw_workspace() -> int:
    nb = ctypes.c_size_t()
    call("gnn_adamw_workspace", ctypes.byref(nb))
    return nb.value


def gnn_adamw_step(tensors: AdamwTensors, state, lr: float, beta1: float = 0.9, beta2: float = 0.999,
                   eps: float = 1e-8, weight_decay: float = 0.01, grad_scale: float = 1.0,
                   max_norm: float = 0.0, grad_norm=None, ws=None, stream=None) -> None:
    """One AdamW step over every tensor; with max_norm > 0 the gradients are
    clipped by their global norm (written to grad_norm, fp32 [1]) and a step
    whose norm is not finite is skipped."""
    if state.dtype is not (_bits or _torch_bits()).f64 or state.numel() != 4 or not state.is_contiguous() or \
            not state.is_cuda:
        raise ValueError("state: needs the fp64 CUDA tensor that adamw_state makes")
    if tensors.device is not None and state.device != tensors.device:
        raise ValueError(f"state: on {state.device}, the tensors on {tensors.device}")
    at, size, ws = _ws(ws, gnn_adamw_workspace(), state, stream)
    call("gnn_adamw_step", tensors.c, tensors.count, tensors.param_type, tensors.grad_type, tensors.state_bits,
         state.data_ptr(), lr, beta1, beta2, eps, weight_decay, grad_scale, max_norm, _f32(grad_norm, 1, "grad_norm"), at,
         size, _current(state, stream))


# Muon's quintic: its singular values end between 0.7 and 1.2.
NS_COEFFS = (3.4445, -4.7750, 2.0315)


def _coeffs(coeffs, steps: int):
    """One triple for every step, or a triple each, as a C array."""
    if not isinstance(coeffs, tuple) or any(isinstance(c, list) for c in coeffs):
        coeffs = tuple(tuple(c) if hasattr(c, "__len__") else c for c in coeffs)
    return _coeff_array(coeffs, steps)


@functools.lru_cache(maxsize=64)
def _coeff_array(coeffs, steps: int):
    each = coeffs if coeffs and hasattr(coeffs[0], "__len__") else (coeffs,) * steps
    flat = [float(c) for triple in each for c in triple]
    if len(each) != steps or any(len(triple) != 3 for triple in each):
        raise ValueError(f"coeffs: needs three numbers, or three for each of {steps} steps")
    return (ctypes.c_float * max(len(flat), 1))(*flat)


@functools.lru_cache(maxsize=1024)
def gnn_orthogonalise_workspace(count: int, rows: int, cols: int) -> int:
    nb = ctypes.c_size_t()
    call("gnn_orthogonalise_workspace", count, rows, cols, ctypes.byref(nb))
    return nb.value


def _matrices(t, what: str):
    """(row stride, stride between matrices) of [rows, cols] or [count, rows, cols]."""
    if t.dim() not in (2, 3) or not t.is_cuda or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{what}: needs a CUDA matrix, or a batch of them, with contiguous rows, got {tuple(t.shape)} "
                         f"with strides {t.stride()}")
    cols = t.shape[-1]
    ld = t.stride(-2) if t.shape[-2] > 1 else cols
    return ld, t.stride(0) if t.dim() == 3 else 0


def gnn_orthogonalise(X, O, steps: int = 5, coeffs=NS_COEFFS, eps: float = 1e-7, norms=None, ws=None,  # noqa: E741
                      stream=None) -> None:
    """O = X / (|X| + eps) after `steps` of Newton-Schulz with coefficients
    (a, b, c), or a triple for each step; X [rows, cols] or [count, rows, cols], O
    of X's shape, any of fp32, bf16 and fp16 each; norms (fp32 [count]) receives
    every |X|.  Operands are held to 22 bits in fp16's range, which the steps must not
    leave: every singular value v stays below 7 and a + b v^2 + c v^4 within 60 of
    zero (NS_COEFFS: 1.3 and 3.5).  A matrix whose norm is not finite gives NaN."""
    ldx, sx = _matrices(X, "X")
    ldo, so = _matrices(O, "O")
    if O.shape != X.shape:
        raise ValueError(f"O: needs X's shape {tuple(X.shape)}, got {tuple(O.shape)}")
    rows, cols = X.shape[-2:]
    count = X.shape[0] if X.dim() == 3 else 1
    at, size, ws = _ws(ws, gnn_orthogonalise_workspace(count, rows, cols), X, stream)
    call("gnn_orthogonalise", X.data_ptr(), ldx, sx, _type(X), count, rows, cols,
         _coeffs(coeffs, steps), steps, eps, O.data_ptr(), ldo,
         so, _type(O), _f32(norms, count, "norms"), at, size, _current(X, stream))


def _share(a, b) -> bool:
    """Whether (start, rows, stride, width) in bytes of two matrices may share one; rows
    that lie apart in a common period of the strides (columns of one buffer) do not."""
    (pa, ra, sa, wa), (pb, rb, sb, wb) = a, b
    if pa + (ra - 1) * sa + wa <= pb or pb + (rb - 1) * sb + wb <= pa:
        return False
    period = math.gcd(sa if ra > 1 else 0, sb if rb > 1 else 0)
    d = (pb - pa) % period if period else 0
    return period == 0 or d < wa or d + wb > period


class MuonTensors:
    """The matrices of a Muon optimiser, checked once: lists of parameters (fp32
    or bf16 [rows, cols], updated in place), their gradients (fp32, bf16 or fp16),
    momenta (fp32 or bf16) and, optionally, copies (bf16, None for a matrix without
    one; bf16 parameters may be their own), with contiguous rows, and the factors on
    the updates; scales None: 0.2 sqrt(max(rows, cols)), which makes an update's mean
    square that of AdamW's, so that both take one learning rate.  Matrices lie apart
    from one another (columns of one buffer do; gradients may be shared).  All stay the
    caller's."""

    def __init__(self, params, grads, momenta, copies=None, scales=None):
        import torch
        k = len(params)
        self.count = k
        lists = dict(params=params, grads=grads, momenta=momenta, copies=copies)
        for name, ts in dict(lists, scales=scales).items():
            if ts is not None and len(ts) != k:
                raise ValueError(f"{name}: {len(ts)} for {k} parameters")
        want = dict(params=params[0].dtype if k else torch.float32, grads=grads[0].dtype if k else torch.float32,
                    momenta=momenta[0].dtype if k else torch.float32, copies=torch.bfloat16)
        for name, ts in lists.items():
            for i, t in enumerate(ts or ()):
                if t is None and name == "copies":
                    continue
                if t.device != params[0].device:
                    raise ValueError(f"{name}[{i}]: on {t.device}, params[0] on {params[0].device}")
                if t.dim() != 2 or t.shape != params[i].shape or t.dtype != want[name] or t.device.type != "cuda" or \
                        (t.shape[1] > 1 and t.stride(1) != 1):
                    raise ValueError(f"{name}[{i}]: needs a {want[name]} CUDA matrix of {tuple(params[i].shape)} with "
                                     "contiguous rows")
        for name in ("params", "momenta", "copies"):
            places = [t.data_ptr() for t in lists[name] or () if t is not None and t.numel()]
            if len(set(places)) < len(places):
                raise ValueError(f"{name}: a matrix is listed twice")
        spans = sorted(((t.data_ptr(), t.shape[0], _matrices(t, name)[0] * t.dtype.itemsize, t.shape[1] * t.dtype.itemsize), name, i)
                       for name, ts in lists.items() for i, t in enumerate(ts or ()) if t is not None and t.numel())
        open_ = []  # those whose end lies ahead
        for span, name, i in spans:
            open_ = [o for o in open_ if o[0][0] + (o[0][1] - 1) * o[0][2] + o[0][3] > span[0]]
            for other, its, j in open_:
                own = i == j and {name, its} == {"params", "copies"} and span == other
                if not (name == its == "grads") and not own and _share(span, other):
                    raise ValueError(f"{name}[{i}]: overlaps {its}[{j}]")
            open_.append((span, name, i))
        self.param_type, self.grad_type, self.m_type = (_type(t[0]) if k else 0 for t in (params, grads, momenta))
        self.device = params[0].device if k else None
        self._keep = {name: list(ts) for name, ts in lists.items() if ts is not None}
        at = lambda ts, i: None if ts is None or ts[i] is None else ts[i].data_ptr()  # noqa: E731
        ld = lambda ts, i: 0 if ts is None or ts[i] is None else _matrices(ts[i], "matrix")[0]  # noqa: E731
        four = (params, grads, momenta, copies)
        self.c = (GnnMuonTensor * max(k, 1))(*[
            GnnMuonTensor(*(at(ts, i) for ts in four), *(ld(ts, i) for ts in four), *params[i].shape,
                          0.2 * max(params[i].shape) ** 0.5 if scales is None else float(scales[i])) for i in range(k)])
        self.ws_bytes = gnn_muon_workspace(self)


def gnn_muon_workspace(tensors: MuonTensors) -> int:
    nb = ctypes.c_size_t()
    call("gnn_muon_workspace", tensors.c, tensors.count, ctypes.byref(nb))
    return nb.value


def gnn_muon_step(tensors: MuonTensors, lr: float, momentum: float = 0.95, nesterov: bool = True,
                  weight_decay: float = 0.0, grad_scale: float = 1.0, steps: int = 5, coeffs=NS_COEFFS,
                  eps: float = 1e-7, norms=None, ws=None, stream=None) -> None:
    """One Muon step over every matrix: m = momentum m + g, the update (with
    nesterov g + momentum m, else m) orthogonalised (coeffs within gnn_orthogonalise's
    limits), params (1 - lr weight_decay) - lr scale update.  norms (fp32, one a
    matrix) receives the updates' norms; a matrix whose norm is not finite is left as
    it is."""
    if tensors.count == 0:
        return
    first = tensors._keep["params"][0]
    at, size, ws = _ws(ws, tensors.ws_bytes, first, stream)
    call("gnn_muon_step", tensors.c, tensors.count, tensors.param_type, tensors.grad_type, tensors.m_type, lr, momentum,
         int(nesterov), weight_decay, grad_scale,
         _coeffs(coeffs, steps), steps, eps,
         _f32(norms, tensors.count, "norms"), at, size, _current(first, stream))


# ---------------------------------------------------------------- epoch control (host only)
def gnn_ldr_init(lam: float = 0.9, delta: int = 5, b_min: int = 1, b_max: int = 8) -> LdrState:
    st = LdrState()
    call("gnn_ldr_init", ctypes.byref(st), float(lam), delta, b_min, b_max)
    return st


def gnn_ldr_update(st: LdrState, partition_losses: Sequence[float], epoch_seconds: float):
    """Reports one epoch; returns (base width, asynchronous?) for the next."""
    n = len(partition_losses)
    arr = (ctypes.c_double * max(n, 1))(*[float(x) for x in partition_losses])
    call("gnn_ldr_update", ctypes.byref(st), arr, n, float(epoch_seconds))
    return st.base_bits, bool(st.async_next)
