"""Host-side composition of the libmoe calls into a layer step.

PyTorch only allocates device buffers and supplies the stream; every step of
the layer runs in libmoe's kernels.  Nothing here synchronises the host with the
device: the row split per expert stays on the device (cu_seqlens).

    MoE forward:  moe_route -> moe_dispatch -> moe_expert_ffn -> moe_combine
                  (or moe_dispatch writing index maps only -> moe_expert_ffn_gather,
                  whose gate/up GEMM reads the rows of x itself)
    backward:     moe_permute_bwd (dh, d_gate, dx from dxs) -> moe_route_bwd
    MoD front:    mod_select (scores, capacity top-C, gather, skip copy) -> MoE on the
                  selected tokens -> moe_combine(row_scale = score, residual = x,
                  out_row = selected rows); route backward through
                  moe_permute_bwd(d_scale) and moe_route_bwd(MOE_ROUTE_MOD_LINEAR).
    MoE block:    moe_combine_norm (the norm before it) -> moe_route_group -> moe_dispatch ->
                  moe_expert_ffn -> moe_combine_norm (combine, norm after the block, gate and
                  residual scale, residual, norm before the next block); backward in the
                  reverse order, its expert activations kept in 8 bits where asked.
    expert tensors: ExpertMuon updates them with the gradients of a backward (moe_muon_step);
                  ExpertsW4 holds them in 4 bits, for the forwards' w_gate (moe_expert_ffn_w4).
"""
from __future__ import annotations

import math

import torch

from . import _lib as L

_TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
_CDT = {"f32": L.MOE_F32, "bf16": L.MOE_BF16}


def _ws(nbytes: int, device):
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


class _Holder:
    """Which forward the expert tensors xs, act and gu hold, of all layers that share them."""

    def __init__(self):
        self.forward = None  # none that is known, or one that has not come to its end
        self.shared = False


class MoEBuffers:
    """Device buffers of one MoE layer call (T tokens, H, E, K, Hp).

    ``experts``: buffers of another layer of the same sizes, whose xs, act, gu, dh, dxs and FFN
    workspaces serve this one too.  Such layers run one after the other on one stream, and a
    layer's backward needs an ExpertCheckpoint of its forward (moe_block_backward) unless no
    other ran between: moe_forward and moe_block_forward note whose tensors they are, and the
    backward of a forward that is gone is refused.  A captured graph notes that at its capture
    alone: such graphs are replayed in the order of their captures."""

    def __init__(self, T, H, E, K, Hp, dtype: str, device, backward: bool = True, train: bool = False,
                 experts: MoEBuffers | None = None):
        self.T, self.H, self.E, self.K, self.Hp, self.dtype = T, H, E, K, Hp, dtype
        self.cdt = _CDT[dtype]
        tdt = _TDT[dtype]
        R = T * K
        dev = device
        f32, i32 = torch.float32, torch.int32
        if experts is not None:
            e = experts
            if (T, H, E, K, Hp, dtype, train) != (e.T, e.H, e.E, e.K, e.Hp, e.dtype, e.gu is not None) or \
                    backward and not hasattr(e, "dh") or torch.empty(0, device=dev).device != e.xs.device:
                raise ValueError("MoEBuffers: the buffers to share are of other sizes or another device, or lack a "
                                 "backward's")
        self.forward = object()  # this layer's last forward
        self.holder = _Holder() if experts is None else experts.holder
        self.holder.shared = experts is not None

        def rows(name, width):
            return torch.empty((R, width), dtype=tdt, device=dev) if experts is None else getattr(experts, name)
        self.logits = torch.empty((T, E), dtype=f32, device=dev)
        self.idx = torch.empty((T, K), dtype=i32, device=dev)
        self.gate = torch.empty((T, K), dtype=f32, device=dev)
        self.cu = torch.empty((E + 1,), dtype=i32, device=dev)
        self.dst_row = torch.empty((R,), dtype=i32, device=dev)
        self.src_tok = torch.empty((R,), dtype=i32, device=dev)
        self.xs = rows("xs", H)
        self.act = rows("act", Hp)
        self.h = torch.empty((R, H), dtype=tdt, device=dev)
        self.y = torch.empty((T, H), dtype=tdt, device=dev)
        self.ws_dispatch_bytes = L.moe_workspace_bytes(L.MOE_OP_DISPATCH, T, H, E, K, Hp)
        self.ws_dispatch = _ws(self.ws_dispatch_bytes, dev)
        self.ws_route_bytes = L.moe_workspace_bytes(L.MOE_OP_ROUTE, T, H, E, K, Hp)
        self.ws_route = _ws(self.ws_route_bytes, dev)
        # the expert FFN's optional workspace (bf16: the down projection's
        # last round split along K)
        self.ws_ffn_bytes = L.moe_workspace_bytes(L.MOE_OP_EXPERT_FFN, T, H, E, K, Hp) if dtype == "bf16" else 0
        self.ws_ffn = _ws(self.ws_ffn_bytes, dev) if experts is None else experts.ws_ffn
        if backward:
            self.dh = rows("dh", H)
            self.d_gate = torch.empty((T, K), dtype=f32, device=dev)
            self.d_logits = torch.empty((T, E), dtype=f32, device=dev)
            self.dw_router = torch.empty((H, E), dtype=f32, device=dev)
            self.dx = torch.empty((T, H), dtype=tdt, device=dev)
            self.ws_bwd_bytes = L.moe_workspace_bytes(L.MOE_OP_ROUTE_BWD, T, H, E, K, Hp)
            self.ws_bwd = _ws(self.ws_bwd_bytes, dev)
        self.gu = None
        if train:  # the expert backward: saved [g | u], dxs, fp32 weight gradients
            self.gu = rows("gu", 2 * Hp)
            self.dxs = rows("dxs", H)
            self.dw_gate = torch.empty((E, H, Hp), dtype=f32, device=dev)
            self.dw_up = torch.empty((E, H, Hp), dtype=f32, device=dev)
            self.dw_down = torch.empty((E, H, Hp), dtype=f32, device=dev)
            self.ws_ffn_bwd_bytes = L.moe_workspace_bytes(L.MOE_OP_EXPERT_FFN_BWD, T, H, E, K, Hp)
            self.ws_ffn_bwd = _ws(self.ws_ffn_bwd_bytes, dev) if experts is None else experts.ws_ffn_bwd


def _dtype_of(w):
    if w.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"expert tensors are bf16 or fp32, not {w.dtype}")
    return L.MOE_F32 if w.dtype == torch.float32 else L.MOE_BF16


def _check_three(what, tensors, n, device, types=(torch.float32, torch.bfloat16), optional=False):
    """Three expert tensors (optional: or None, or raw addresses) that three calls, one after the other, are to take: what the
    third one would refuse is refused before the first is made."""
    if len(tensors) != 3:
        raise ValueError(f"{what}: one for each of the three expert tensors")
    for t in tensors:
        if optional and (t is None or type(t) is int):
            continue
        if not torch.is_tensor(t):
            raise ValueError(f"{what}: tensors, not {type(t).__name__}")
        if t.dtype not in types or t.numel() < n or not t.is_contiguous() or t.device != device or t.data_ptr() % 16:
            raise ValueError(f"{what}: contiguous 16-byte aligned tensors of {' or '.join(map(str, types))} and {n} "
                             f"elements on {device}, not {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


class ExpertsW4:
    """The experts' three tensors [E, H, Hp] in 4 bits (moe_w4_pack), in the place of w_gate, w_up and
    w_down of moe_forward, mod_forward and moe_block_forward (as w_gate; w_up and w_down are then None).
    For serving: such a forward keeps nothing that a backward could use, and chooses by itself whether dispatch lays the
    rows side by side (fused_gather is not asked).  Up to some 200 rows an expert it is the faster one too."""

    def __init__(self, E, H, Hp, device, group=64):
        if group not in (32, 64, 128):
            raise ValueError("ExpertsW4: groups of 32, 64 or 128 weights share a scale")
        self.E, self.H, self.Hp, self.group = E, H, Hp, group

        def packed(out, inp):
            blocks = -(-inp // 128)
            return (torch.empty((E, out, blocks * 16), dtype=torch.int32, device=device),
                    torch.empty((E, out, blocks * 128 // group), dtype=torch.bfloat16, device=device))
        self.q_gate, self.s_gate = packed(Hp, H)
        self.q_up, self.s_up = packed(Hp, H)
        self.q_down, self.s_down = packed(H, Hp)

    def _each(self, w_gate, w_up, w_down):
        _check_three("ExpertsW4", (w_gate, w_up, w_down), self.E * self.H * self.Hp, self.q_gate.device)
        return ((w_gate, 0, self.q_gate, self.s_gate), (w_up, 0, self.q_up, self.s_up),
                (w_down, 1, self.q_down, self.s_down))

    def pack(self, w_gate, w_up, w_down, stream=None):
        """From bf16 or fp32 tensors; returns self."""
        for w, axis, q, s in self._each(w_gate, w_up, w_down):
            L.moe_w4_pack(w, self.E, self.H, self.Hp, axis, self.group, _dtype_of(w), q, s, stream=stream)
        return self

    def unpack(self, w_gate, w_up, w_down, stream=None):
        """The weights that the packed form stands for, into bf16 or fp32 tensors."""
        for w, axis, q, s in self._each(w_gate, w_up, w_down):
            L.moe_w4_unpack(q, s, self.E, self.H, self.Hp, axis, self.group, _dtype_of(w), w, stream=stream)


class ExpertMuon:
    """The momentum of a layer's three expert tensors and their orthogonalised update (moe_muon_step)
    from the gradients that a backward left in ``b`` (train=True)."""

    def __init__(self, b: MoEBuffers, beta=0.95, nesterov=True, steps=5, coef=(3.4445, -4.7750, 2.0315), eps=1e-7):
        if b.gu is None:
            raise ValueError("ExpertMuon: the buffers were made without train=True")
        self.E, self.H, self.Hp = b.E, b.H, b.Hp
        self.beta, self.nesterov, self.steps, self.coef, self.eps = beta, nesterov, steps, coef, eps
        self.m_gate, self.m_up, self.m_down = (torch.zeros_like(b.dw_gate) for _ in range(3))
        self.ws_bytes = L.moe_workspace_bytes(L.MOE_OP_MUON_STEP, 0, b.H, b.E, 0, b.Hp)
        self.ws = _ws(self.ws_bytes, b.dw_gate.device)

    def step(self, b: MoEBuffers, w_gate, w_up, w_down, lr, weight_decay=0.0, scale=None, low=(None, None, None),
             stream=None):
        """w <- (1 - lr weight_decay) w - lr scale O for the three tensors, in place.  scale: 0.2 sqrt(max(H, Hp))
        unless given, which makes the update's elements about 0.2 lr in size.  low: for fp32 weights, the bf16
        tensors that the forward reads, written too."""
        if (b.E, b.H, b.Hp) != (self.E, self.H, self.Hp):
            raise ValueError("ExpertMuon: the buffers are of another layer's sizes")
        n, dev = self.E * self.H * self.Hp, self.m_gate.device
        _check_three("ExpertMuon", (w_gate, w_up, w_down), n, dev)
        _check_three("ExpertMuon, low", low, n, dev, (torch.bfloat16,), optional=True)
        if scale is None:
            scale = 0.2 * math.sqrt(max(self.H, self.Hp))
        for w, dw, m, lo in ((w_gate, b.dw_gate, self.m_gate, low[0]), (w_up, b.dw_up, self.m_up, low[1]),
                             (w_down, b.dw_down, self.m_down, low[2])):
            L.moe_muon_step(w, dw, m, self.E, self.H, self.Hp, _dtype_of(w), self.beta, self.nesterov, lr, weight_decay,
                            scale, self.steps, *self.coef, self.eps, w, lo, m, self.ws, self.ws_bytes, stream=stream)


def _check_w4(b: MoEBuffers, w_gate, w_up, w_down):
    """The ExpertsW4 that a forward was given for its expert tensors, or None."""
    if not isinstance(w_gate, ExpertsW4):
        return None
    if b.gu is not None or b.dtype != "bf16":
        raise ValueError("ExpertsW4: 4-bit experts serve bf16 forwards alone (buffers without train=True)")
    if w_up is not None or w_down is not None:
        raise ValueError("ExpertsW4: it stands for all three tensors, w_up and w_down are None")
    if (w_gate.E, w_gate.H, w_gate.Hp) != (b.E, b.H, b.Hp):
        raise ValueError("ExpertsW4: of another layer's sizes")
    return w_gate


def _dispatch_and_experts(b: MoEBuffers, x, w_gate, w_up, w_down, fused_gather, stream):
    """From the routing in b to the expert outputs b.h, with the tensors as they are or in 4 bits."""
    T, H, E, K, Hp, dt = b.T, b.H, b.E, b.K, b.Hp, b.cdt
    w4 = _check_w4(b, w_gate, w_up, w_down)
    if w4 is not None:
        # where the products want the rows side by side, dispatch lays them there
        fused_gather = L.moe_workspace_bytes(L.MOE_OP_EXPERT_FFN_W4, T, H, E, K, Hp) == 0
    L.moe_dispatch(x, b.idx, T, H, E, K, dt, b.cu, b.dst_row, b.src_tok, None if fused_gather else b.xs,
                   b.ws_dispatch, b.ws_dispatch_bytes, stream=stream)
    if w4 is not None:
        L.moe_expert_ffn_w4(x if fused_gather else b.xs, b.src_tok if fused_gather else None, T, b.cu, T * K, w4.q_gate,
                            w4.s_gate, w4.q_up, w4.s_up, w4.q_down, w4.s_down, E, H, Hp, w4.group, dt, b.act, b.h,
                            stream=stream)
    elif fused_gather:
        L.moe_expert_ffn_gather(x, b.src_tok, T, b.cu, T * K, w_gate, w_up, w_down, E, H, Hp, dt, b.act, b.gu, b.h,
                                b.ws_ffn, b.ws_ffn_bytes, stream=stream)
    else:
        L.moe_expert_ffn_ex(b.xs, b.cu, T * K, w_gate, w_up, w_down, E, H, Hp, dt, b.act, b.gu, b.h,
                            b.ws_ffn, b.ws_ffn_bytes, stream=stream)


def _forward_begins(b: MoEBuffers):
    """A forward of b begins: no other's activations are whole from here on, and an older one's
    routing in b is gone."""
    b.holder.forward = None
    b.forward = object()


def moe_forward(b: MoEBuffers, x, w_router, logit_bias, w_gate, w_up, w_down, stream=None,
                row_scale=None, residual=None, out_row=None, y=None, route_flags=0, fused_gather=None):
    """One MoE forward pass into the buffers of ``b`` (y defaults to ``b.y``);
    ``route_flags``: MOE_ROUTE_RENORM / MOE_ROUTE_BIAS_SELECT gate options.
    ``w_gate`` may be ExpertsW4 (and w_up, w_down None).
    ``fused_gather``: dispatch writes only the index maps and the expert FFN
    reads the rows of x itself (moe_expert_ffn_gather); off by default (the
    row-by-row operand fetch measured 7-11% slower than the gather kernel plus
    the FFN on the dispatched rows), and never with train=True buffers (the
    expert backward reads the dispatched rows)."""
    T, H, E, K, Hp, dt = b.T, b.H, b.E, b.K, b.Hp, b.cdt
    if fused_gather is None or b.gu is not None:
        fused_gather = False
    _check_w4(b, w_gate, w_up, w_down)
    _forward_begins(b)
    L.moe_route_ex(x, w_router, logit_bias, T, H, E, K, dt, route_flags, b.logits, b.idx, b.gate, b.ws_route,
                   b.ws_route_bytes, stream=stream)
    _dispatch_and_experts(b, x, w_gate, w_up, w_down, fused_gather, stream)
    b.holder.forward = b.forward
    L.moe_combine(b.h, b.gate, b.dst_row, row_scale, residual, out_row, T, H, K, dt,
                  b.y if y is None else y, stream=stream)


def moe_backward(b: MoEBuffers, x, w_router, dy, dxs, stream=None, row_scale=None, out_row=None,
                 d_scale=None, route_flags=0):
    """Gate and dispatch/combine backward: dh, d_gate, d_logits, dw_router and
    dx = (adjoint of the gather applied to dxs) + router contribution."""
    T, H, E, K, dt = b.T, b.H, b.E, b.K, b.cdt
    L.moe_permute_bwd(dy, b.h, b.gate, b.dst_row, row_scale, out_row, dxs, T, H, K, dt, b.dh,
                      b.d_gate, d_scale, b.dx, stream=stream)
    renorm = L.MOE_ROUTE_GATE_RENORM if route_flags & L.MOE_ROUTE_RENORM else 0
    L.moe_route_bwd(L.MOE_ROUTE_SOFTMAX_TOPK | renorm, b.d_gate, b.logits, b.idx, x, w_router, T, H, E, K, dt,
                    b.d_logits, b.dw_router, b.dx, b.ws_bwd, b.ws_bwd_bytes, stream=stream)


def moe_train_backward(b: MoEBuffers, x, w_router, w_gate, w_up, w_down, dy, stream=None, route_flags=0):
    """Full backward of the layer (buffers made with train=True, forward run
    with them, and the last one in them where layers share expert tensors): dh and
    d_gate, the expert backward (dxs and the three weight gradients), dx = sum_k
    dxs[row(t,k)] plus the router's share, dw_router."""
    if b.holder.shared and b.holder.forward is not b.forward:
        raise ValueError("moe_train_backward: the layer's forward must be the last one in the expert tensors it shares")
    T, H, E, K, Hp, dt = b.T, b.H, b.E, b.K, b.Hp, b.cdt
    L.moe_permute_bwd(dy, b.h, b.gate, b.dst_row, None, None, None, T, H, K, dt, b.dh, b.d_gate, None, None,
                      stream=stream)
    L.moe_expert_ffn_bwd(b.xs, b.cu, T * K, w_gate, w_up, w_down, E, H, Hp, dt, b.gu, b.act, b.dh, b.dxs,
                         b.dw_gate, b.dw_up, b.dw_down, b.ws_ffn_bwd, b.ws_ffn_bwd_bytes, stream=stream)
    L.moe_permute_bwd(None, None, b.gate, b.dst_row, None, None, b.dxs, T, H, K, dt, None, None, None, b.dx,
                      stream=stream)
    renorm = L.MOE_ROUTE_GATE_RENORM if route_flags & L.MOE_ROUTE_RENORM else 0
    L.moe_route_bwd(L.MOE_ROUTE_SOFTMAX_TOPK | renorm, b.d_gate, b.logits, b.idx, x, w_router, T, H, E, K, dt,
                    b.d_logits, b.dw_router, b.dx, b.ws_bwd, b.ws_bwd_bytes, stream=stream)


class MoDBuffers:
    """Buffers of the MoD front end: B sequences of L tokens, capacity C."""

    def __init__(self, B, Lseq, C, H, E, K, Hp, dtype: str, device, backward: bool = True):
        self.B, self.L, self.C, self.H = B, Lseq, C, H
        self.cdt = _CDT[dtype]
        tdt = _TDT[dtype]
        n = B * Lseq
        self.score = torch.empty((n,), dtype=torch.float32, device=device)
        self.sel = torch.empty((B * C,), dtype=torch.int32, device=device)  # flat token rows
        self.sel_score = torch.empty((B * C,), dtype=torch.float32, device=device)
        self.mask = torch.empty((n,), dtype=torch.uint8, device=device)
        self.x_sel = torch.empty((B * C, H), dtype=tdt, device=device)
        self.y = torch.empty((n, H), dtype=tdt, device=device)
        self.moe = MoEBuffers(B * C, H, E, K, Hp, dtype, device, backward=backward)
        if backward:
            self.d_score = torch.empty((B * C,), dtype=torch.float32, device=device)
            self.dw_mod = torch.empty((H,), dtype=torch.float32, device=device)
            self.ws_lin_bytes = L.moe_workspace_bytes(L.MOE_OP_ROUTE_BWD, B * C, H, 1, 1, 0)
            self.ws_lin = _ws(self.ws_lin_bytes, device)


def mod_forward(m: MoDBuffers, x, w_mod, w_router, w_gate, w_up, w_down, stream=None):
    """MoD + MoE forward: y = x + s * MoE(x) on the selected tokens, y = x elsewhere."""
    b = m.moe
    _check_w4(b, w_gate, w_up, w_down)
    L.mod_select(x, w_mod, m.B, m.L, m.H, m.C, m.cdt, m.score, m.sel, m.sel_score, m.mask, m.x_sel,
                 m.y, stream=stream)
    moe_forward(b, m.x_sel, w_router, None, w_gate, w_up, w_down, stream=stream,
                row_scale=m.sel_score, residual=x, out_row=m.sel, y=m.y)


def mod_route_backward(m: MoDBuffers, w_router, w_mod, dy, stream=None):
    """Route backward of the MoD + MoE layer with the expert outputs held fixed:
    d_gate of the MoE router, d_score = <dy, MoE(x)> of the MoD router, dw_router,
    dw_mod and their input gradients accumulated into m.moe.dx."""
    b = m.moe
    T, H, E, K, dt = b.T, b.H, b.E, b.K, b.cdt
    L.moe_permute_bwd(dy, b.h, b.gate, b.dst_row, m.sel_score, m.sel, None, T, H, K, dt, b.dh,
                      b.d_gate, m.d_score, None, stream=stream)
    L.moe_route_bwd(L.MOE_ROUTE_SOFTMAX_TOPK | L.MOE_ROUTE_DX_WRITE, b.d_gate, b.logits, b.idx, m.x_sel, w_router, T, H, E,
                    K, dt, b.d_logits, b.dw_router, b.dx, b.ws_bwd, b.ws_bwd_bytes, stream=stream)
    L.moe_route_bwd(L.MOE_ROUTE_MOD_LINEAR, m.d_score, None, None, m.x_sel, w_mod, T, H, 1, 1, dt,
                    None, m.dw_mod, b.dx, m.ws_lin, m.ws_lin_bytes, stream=stream)


class GroupGate:
    """Options of the group-limited gate (moe_gate): expert groups, how many of them a token
    may use, and the mode bits and scale of its gates."""

    def __init__(self, groups=1, topk_groups=None, sigmoid=False, renorm=False, group_max=False, scale=1.0):
        self.groups, self.topk_groups = groups, groups if topk_groups is None else topk_groups
        self.mode = (L.MOE_GATE_SIGMOID if sigmoid else L.MOE_GATE_SOFTMAX) | (L.MOE_GATE_RENORM if renorm else 0) | \
            (L.MOE_GATE_GROUP_MAX if group_max else 0)
        self.scale = scale


class ExpertCheckpoint:
    """What the expert FFN's backward reads of the forward, in 8 bits: the dispatched rows and
    [g | u] (moe_ckpt_pack), 1.03 bytes a value instead of 2.  act is computed again.  One for
    each layer, so that layers whose buffers share these tensors (MoEBuffers(experts=...)) can
    save from them and restore into them; what else a backward reads, each layer keeps.  It
    serves the backward of the forward that it was saved from."""

    def __init__(self, b: MoEBuffers):
        if b.gu is None:
            raise ValueError("ExpertCheckpoint: the buffers were made without train=True")
        self.forward = None  # the forward that it holds
        dev, R = b.gu.device, b.T * b.K
        self.gu = torch.empty((R, 2 * b.Hp), dtype=torch.int8, device=dev)
        self.gu_scale = torch.empty((R, (2 * b.Hp + 31) // 32), dtype=torch.uint8, device=dev)
        self.xs = torch.empty((R, b.H), dtype=torch.int8, device=dev)
        self.xs_scale = torch.empty((R, (b.H + 31) // 32), dtype=torch.uint8, device=dev)

    def save(self, b: MoEBuffers, stream=None):
        if b.holder.shared and b.holder.forward is not b.forward:
            raise ValueError("ExpertCheckpoint: the expert tensors hold another layer's forward")
        R = b.T * b.K
        self.forward = None
        L.moe_ckpt_pack(b.gu, R, 2 * b.Hp, b.cdt, self.gu, self.gu_scale, stream=stream)
        L.moe_ckpt_pack(b.xs, R, b.H, b.cdt, self.xs, self.xs_scale, stream=stream)
        self.forward = b.forward

    def restore(self, b: MoEBuffers, stream=None):
        if self.forward is None:
            raise ValueError("ExpertCheckpoint: nothing has been saved")
        R = b.T * b.K
        b.holder.forward = None
        L.moe_ckpt_swiglu(self.gu, self.gu_scale, R, b.Hp, b.cdt, b.gu, b.act, stream=stream)
        L.moe_ckpt_unpack(self.xs, self.xs_scale, R, b.H, b.cdt, b.xs, stream=stream)
        b.holder.forward = self.forward


class MoEBlockBuffers:
    """Buffers of a MoE block: MoEBuffers of its layer (``moe``), the normed input ``x0``, the
    residual stream ``y`` behind the block and the normed input ``xn`` of the next one; for
    training (bf16, as the expert FFN's backward) the gradients of all of them and of the norm
    weights.  ``experts``: MoEBuffers whose expert tensors ``moe`` shares."""

    def __init__(self, T, H, E, K, Hp, dtype: str, device, train: bool = False, experts: MoEBuffers | None = None):
        tdt, f32 = _TDT[dtype], torch.float32
        self.moe = MoEBuffers(T, H, E, K, Hp, dtype, device, backward=train, train=train, experts=experts)
        self.forward = self.moe.forward  # the block's last forward
        self.x0, self.y, self.xn = (torch.empty((T, H), dtype=tdt, device=device) for _ in range(3))
        if train:
            self.d_x = torch.empty((T, H), dtype=tdt, device=device)
            self.dw_pre, self.dw_post, self.d_res_scale, self.dw_next = (
                torch.empty((H,), dtype=f32, device=device) for _ in range(4))
            self.ws_norm_bytes = L.moe_workspace_bytes(L.MOE_OP_COMBINE_NORM_BWD, T, H, 0, K, 0)
            self.ws_norm = _ws(self.ws_norm_bytes, device)


def moe_block_forward(m: MoEBlockBuffers, x, w_pre, w_router, sel_bias, gate: GroupGate, w_gate, w_up, w_down,
                      w_post=None, res_scale=None, w_next=None, eps=1e-5, x0=None, ckpt: ExpertCheckpoint | None = None,
                      stream=None):
    """One MoE block: m.y = x + res_scale * norm(MoE(norm(x))), m.xn = norm(m.y).

    w_pre, w_post, w_next (float [H]): weights of the norms before the block, after it and
    before the next one; w_post and w_next may be None (no such norm).  x0: norm(x) where
    the block before has written it (its m.xn); w_pre is then unused.  ckpt: keep the expert
    activations there, so that blocks which share m.moe's may run before the backward.  w_gate
    may be ExpertsW4 (and w_up, w_down None)."""
    b = m.moe
    T, H, E, K, Hp, dt = b.T, b.H, b.E, b.K, b.Hp, b.cdt
    _check_w4(b, w_gate, w_up, w_down)
    _forward_begins(b)
    m.forward = b.forward
    if x0 is None:
        x0 = m.x0
        L.moe_combine_norm(None, None, None, None, x, None, None, w_pre, eps, T, H, 0, dt, None, x0, stream=stream)
    L.moe_route_group(x0, w_router, sel_bias, T, H, E, K, dt, gate.groups, gate.topk_groups, gate.mode, gate.scale,
                      b.logits, b.idx, b.gate, b.ws_route, b.ws_route_bytes, stream=stream)
    _dispatch_and_experts(b, x0, w_gate, w_up, w_down, False, stream)
    b.holder.forward = b.forward
    if ckpt is not None:
        ckpt.save(b, stream=stream)
    L.moe_combine_norm(b.h, b.gate, b.dst_row, None, x, w_post, res_scale, w_next, eps, T, H, K, dt, m.y,
                       None if w_next is None else m.xn, stream=stream)


def moe_block_backward(m: MoEBlockBuffers, x, w_pre, w_router, gate: GroupGate, w_gate, w_up, w_down, dy, dxn=None,
                       w_post=None, res_scale=None, w_next=None, eps=1e-5, x0=None,
                       ckpt: ExpertCheckpoint | None = None, stream=None):
    """Backward of moe_block_forward on the buffers it filled (with ckpt: on its checkpoint),
    given dy = dL/dy and, with w_next, dxn = dL/dxn.  Leaves m.d_x = dL/dx, the weight
    gradients in m.moe (dw_gate, dw_up, dw_down, dw_router) and those of the norms.  With x0
    given (the norm belongs to the block before) m.d_x holds the residual's share alone and
    m.moe.dx = dL/dx0."""
    b = m.moe
    if m.forward is not b.forward:
        raise ValueError("moe_block_backward: another forward has run in the block's buffers")
    if ckpt is None and b.holder.forward is not b.forward:
        raise ValueError("moe_block_backward: without ckpt the block's forward must be the last one in its buffers")
    if ckpt is not None and ckpt.forward is not b.forward:
        raise ValueError("moe_block_backward: ckpt does not hold the block's last forward")
    T, H, E, K, Hp, dt = b.T, b.H, b.E, b.K, b.Hp, b.cdt
    L.moe_combine_norm_bwd(dy, dxn, b.h, b.gate, b.dst_row, None, None if w_next is None else m.y, w_post, res_scale,
                           w_next, eps, T, H, K, dt, m.d_x, b.dh, b.d_gate, None,
                           None if w_post is None else m.dw_post, None if res_scale is None else m.d_res_scale,
                           None if w_next is None else m.dw_next, m.ws_norm, m.ws_norm_bytes, stream=stream)
    if ckpt is not None:
        ckpt.restore(b, stream=stream)
    L.moe_expert_ffn_bwd(b.xs, b.cu, T * K, w_gate, w_up, w_down, E, H, Hp, dt, b.gu, b.act, b.dh, b.dxs,
                         b.dw_gate, b.dw_up, b.dw_down, b.ws_ffn_bwd, b.ws_ffn_bwd_bytes, stream=stream)
    L.moe_permute_bwd(None, None, b.gate, b.dst_row, None, None, b.dxs, T, H, K, dt, None, None, None, b.dx,
                      stream=stream)
    L.moe_gate_bwd(b.d_gate, b.logits, b.idx, T, E, K, gate.mode, gate.scale, b.d_logits, stream=stream)
    L.moe_route_bwd(L.MOE_ROUTE_LOGIT_GRAD, b.d_logits, None, None, m.x0 if x0 is None else x0, w_router, T, H, E, K,
                    dt, None, b.dw_router, b.dx, b.ws_bwd, b.ws_bwd_bytes, stream=stream)
    if x0 is None:
        L.moe_combine_norm_bwd(m.d_x, b.dx, None, None, None, None, x, None, None, w_pre, eps, T, H, 0, dt, m.d_x,
                               None, None, None, None, None, m.dw_pre, m.ws_norm, m.ws_norm_bytes, stream=stream)
