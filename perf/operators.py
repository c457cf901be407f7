"""The operators around the expert products, as cases to time and compare: the routing gate with expert groups, the
combine fused with the norms around the block, and the 8-bit activation checkpoint.

``run`` computes a case in its plain form (elementary torch operations) or, where ``own`` is true, through the
library's calls.  ``exact`` states the same result in 64 bits, written apart from the plain form.

Kinds of cases:
  gate       scores, balance bias, expert groups, top-K and gates from router logits
  gate_bwd   the gradient of those gates with respect to the logits
  norm       combine, norm after the block, gate and residual scale, residual, norm before the next block
  norm_bwd   the gradients of all of that
  ckpt       [g | u] of the expert FFN kept in 8 bits, and g, u and silu(g) u restored for its backward
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
BLOCK = 32  # values that share one power of two in a checkpoint
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one token of a decoding step through a 384-expert router with limited groups
        _gate("gate_one_token", 1, 384, 8, 8, 4, score="sigmoid", bias=True, renorm=True, scale=2.5),
        # a softmax router over groups ranked by their best expert, a training batch
        _gate("gate_softmax_E64", 16384, 64, 6, 8, 3, score="softmax", group_max=True, scale=16.0),
        # a long prefill batch of the 384-expert router, six experts out of service
        _gate("gate_sigmoid_E384", 32768, 384, 8, 8, 4, score="sigmoid", bias=True, renorm=True, scale=2.5, masked=6),
        # the backward of a training batch: gates that sum to one, sigmoid scores
        _gate("gate_bwd_sigmoid_E384", 8192, 384, 8, 8, 4, kind="gate_bwd", score="sigmoid", bias=True, renorm=True,
              scale=2.5),
        # the backward through the whole softmax row
        _gate("gate_bwd_softmax_E64", 16384, 64, 6, 8, 3, kind="gate_bwd", score="softmax", group_max=True, scale=16.0),
        # a decoding step of seven sequences at the widest layer
        _norm("norm_seven_tokens_H7168", 7, 7168, 8),
        # a prompt of the two-expert layer, without the norm after the block
        _norm("norm_T8192_H4096_K2", 8192, 4096, 2, post=False),
        # the widest layer's batch with both norms: the largest forward
        _norm("norm_T8192_H7168_K8", 8192, 7168, 8),
        # a training batch of the fine-grained layer
        _norm("norm_bwd_T16384_H2048_K6", 16384, 2048, 6, kind="norm_bwd"),
        # an fp32 layer of odd sizes
        _norm("norm_bwd_f32_T1001_H1000_K3", 1001, 1000, 3, kind="norm_bwd", dtype="f32"),
        # the two-expert layer's routed rows, [g | u] of 2 x 14336
        _ckpt("ckpt_R16384_Hp14336", 16384, 14336),
        # a ragged fp32 layer
        _ckpt("ckpt_f32_R777_Hp1404", 777, 1404, dtype="f32"),
    ]


def _gate(name, T, E, K, groups, topk_groups, kind="gate", score="softmax", bias=False, renorm=False, group_max=False,
          scale=1.0, masked=0):
    return {"name": name, "kind": kind, "T": T, "E": E, "K": K, "groups": groups, "topk_groups": topk_groups,
            "score": score, "bias": bias, "renorm": renorm, "group_max": group_max, "scale": scale, "masked": masked}


def _norm(name, T, H, K, kind="norm", dtype="bf16", post=True, next=True, scale=True):
    return {"name": name, "kind": kind, "T": T, "H": H, "K": K, "dtype": dtype, "post": post, "next": next,
            "scale": scale}


def _ckpt(name, rows, Hp, dtype="bf16"):
    return {"name": name, "kind": "ckpt", "rows": rows, "Hp": Hp, "dtype": dtype}


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    kind = rng.choice(("gate", "gate", "gate_bwd", "norm", "norm", "norm_bwd", "ckpt"))
    if kind in ("gate", "gate_bwd"):
        groups = rng.choice((1, 1, 2, 4, 8, 16))
        size = _log(rng, max(1, 8 // groups), 512 // groups)
        E = groups * size
        T = _log(rng, 1, min(32768, 32768 * 384 // E))
        K = rng.randint(1, min(E, 10))
        kg = rng.randint(-(-K // size), groups)
        masked = rng.choice((0, 0, 1, 3)) if E >= 32 else 0
        c = _gate("", T, E, K, groups, kg, kind=kind, score=rng.choice(("softmax", "sigmoid")),
                  bias=rng.random() < 0.6, renorm=rng.random() < 0.5, group_max=rng.random() < 0.4,
                  scale=rng.choice((1.0, 2.5)), masked=masked)
    elif kind in ("norm", "norm_bwd"):
        H = 8 * _log(rng, 8, 1024)
        K = rng.randint(0, 8)
        T = _log(rng, 1, min(16384, 16384 * 2048 * 9 // (H * (K + 3))))
        post = K > 0 and rng.random() < 0.6
        if kind == "norm_bwd" and post and K == 1:
            K = 2  # the gradient of a lone row's gate is zero but for eps: nothing to compare
        c = _norm("", T, H, K, kind=kind, dtype=rng.choice(("bf16", "bf16", "f32")), post=post,
                  next=K == 0 or rng.random() < 0.7, scale=K > 0 and rng.random() < 0.6)
    else:
        Hp = 4 * _log(rng, 8, 3584)
        dtype = rng.choice(("bf16", "bf16", "f32"))
        Hp += Hp % 8 if dtype == "bf16" else 0
        c = _ckpt("", _log(rng, 1, min(65536, 16384 * 7168 // Hp)), Hp, dtype=dtype)
    del c["name"]
    return c


def work(case):
    c = case
    if c["kind"] == "gate":
        n = c["T"] * c["E"]
        return {"bytes": 4 * n + 4 * c["E"] * c["bias"] + 8 * c["T"] * c["K"], "flops": 4 * n}
    if c["kind"] == "gate_bwd":
        n, k = c["T"] * c["E"], c["T"] * c["K"]
        whole = c["score"] == "softmax" and not c["renorm"]  # every logit of a row, or the chosen ones alone
        return {"bytes": 4 * n + 8 * k + 4 * (n if whole else k), "flops": 4 * n if whole else 10 * k}
    s = 2 if c["dtype"] == "bf16" else 4
    if c["kind"] == "ckpt":
        n = 2 * c["rows"] * c["Hp"]
        held = n + c["rows"] * -(-2 * c["Hp"] // BLOCK)
        return {"bytes": s * (n + n + n // 2) + 2 * held, "flops": 6 * n}
    n, K = c["T"] * c["H"], c["K"]
    if c["kind"] == "norm":
        rows = K + 1 + (K > 0) + c["next"]  # h, residual; y where there is a block, xn
        extra = c["H"] * (c["post"] + c["next"] + c["scale"])
        return {"bytes": n * s * rows + 4 * extra + 4 * c["T"] * (2 * K + c["scale"]), "flops": n * (2 * K + 10)}
    rows = (1 + 2 * c["next"] + K) + (1 + K)  # dy, y, dxn, h; d_res, dh
    extra = 2 * c["H"] * (c["post"] + c["next"] + c["scale"])
    return {"bytes": n * s * rows + 4 * extra + 4 * c["T"] * (3 * K + 2 * c["scale"]), "flops": n * (6 * K + 30)}


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    c, g = case, torch.Generator(device="cuda")
    g.manual_seed(seed)
    if c["kind"] in ("gate", "gate_bwd"):
        # logits of x ~ N(0, 1) through W_r ~ N(0, 0.02) at H = 7168 have this spread
        s = {"logits": 1.7 * _randn(g, c["T"], c["E"]), "bias": 0.05 * _randn(g, c["E"]) if c["bias"] else None}
        if c["masked"]:
            off = torch.randperm(c["E"], generator=g, device="cuda")[:c["masked"]]
            s["logits"][:, off] = -math.inf
        if c["kind"] == "gate_bwd":
            s["d_gate"] = _randn(g, c["T"], c["K"])
        return s
    dtype = TYPES[c["dtype"]]
    if c["kind"] == "ckpt":
        # pre-activations whose rows differ in size
        rows = torch.exp(0.5 * _randn(g, c["rows"], 1))
        return {"gu": (_randn(g, c["rows"], 2 * c["Hp"]) * rows).to(dtype)}
    T, H, K = c["T"], c["H"], c["K"]
    s = {"residual": _randn(g, T, H).to(dtype)}
    for name in ("h", "gate", "dst_row", "row_scale", "w_post", "res_scale", "w_next"):
        s[name] = None
    if K:
        s["h"] = torch.empty((T * K, H), dtype=dtype, device="cuda")
        for k in range(K):  # in parts, so that the fp32 draws stay small
            s["h"][k * T:(k + 1) * T] = _randn(g, T, H).to(dtype)
        gate = torch.exp(_randn(g, T, K))
        s["gate"] = gate / gate.sum(dim=1, keepdim=True)
        s["dst_row"] = torch.randperm(T * K, generator=g, device="cuda").to(torch.int32)
    if c["scale"]:
        s["row_scale"] = _randn(g, T)
        s["res_scale"] = 0.5 + 0.1 * _randn(g, H)
    if c["post"]:
        s["w_post"] = 1 + 0.1 * _randn(g, H)
    if c["next"]:
        s["w_next"] = 1 + 0.1 * _randn(g, H)
    if c["kind"] == "norm_bwd":
        s["dy"] = _randn(g, T, H).to(dtype)
        s["dxn"] = _randn(g, T, H).to(dtype) if c["next"] else None
    return s


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=dict(case))
    if case["kind"] == "gate_bwd":  # what the forward left
        s["idx"] = _choose(s["logits"], s["bias"], case)[0].to(torch.int32)
    if case["kind"] == "norm_bwd":
        s["y"] = _norm_forward(s, case)[0].to(TYPES[case["dtype"]])
        del s["residual"]
    return s


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["kind"]](state, state["case"])


# ---- plain forms -----------------------------------------------------------------------------------------------------


def _choose(logits, bias, c):
    """Chosen experts [T, K] and the scores of all experts, in 64 bits: a choice hangs on the order of near scores."""
    T, E, G = c["T"], c["E"], c["groups"]
    z = logits.double()
    if c["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-z))
    else:
        e = torch.exp(z - z.amax(dim=1, keepdim=True))
        s = e / e.sum(dim=1, keepdim=True)
    sel = s if bias is None else s + bias.double()
    sel = torch.where(z == -math.inf, -math.inf, sel)
    if c["topk_groups"] < G:
        best = torch.sort(sel.view(T, G, E // G), dim=2, descending=True).values
        rank = best[:, :, 0]
        if not c["group_max"] and E // G > 1:
            second = best[:, :, 1]
            rank = torch.where(second == -math.inf, rank, rank + second)
        order = torch.sort(rank, dim=1, descending=True, stable=True).indices
        # the place of each group in that order; experts of the groups behind are left out
        place = torch.sort(order, dim=1).indices
        left = (place < c["topk_groups"]).repeat_interleave(E // G, dim=1)
        # left-out experts sort behind masked ones of the groups that stay
        behind = torch.sort(torch.where(left, sel, -math.inf), dim=1, descending=True, stable=True).indices
        kept = torch.sort(left.gather(1, behind).to(torch.int8), dim=1, descending=True, stable=True).indices
        return behind.gather(1, kept)[:, :c["K"]], s
    return torch.sort(sel, dim=1, descending=True, stable=True).indices[:, :c["K"]], s


def _plain_gate(state, c):
    idx, s = _choose(state["logits"], state["bias"], c)
    gate = s.gather(1, idx)
    if c["renorm"]:
        gate = gate / gate.sum(dim=1, keepdim=True)
    return {"idx": idx.to(torch.int32), "gate": (gate * c["scale"]).float()}


def _plain_gate_bwd(state, c):
    z, idx, dg = state["logits"], state["idx"].long(), state["d_gate"]
    if c["score"] == "sigmoid":
        l = z.gather(1, idx)
        s, rest = 1 / (1 + torch.exp(-l)), 1 / (1 + torch.exp(l))
        if c["renorm"]:
            q = s / s.sum(dim=1, keepdim=True)
            d = q * rest * (dg - (dg * q).sum(dim=1, keepdim=True))
        else:
            d = dg * s * rest
        return {"d_logits": torch.zeros_like(z).scatter_(1, idx, c["scale"] * d)}
    e = torch.exp(z - z.amax(dim=1, keepdim=True))
    if c["renorm"]:
        q = e.gather(1, idx)
        q = q / q.sum(dim=1, keepdim=True)
        d = q * (dg - (dg * q).sum(dim=1, keepdim=True))
        return {"d_logits": torch.zeros_like(z).scatter_(1, idx, c["scale"] * d)}
    p = e / e.sum(dim=1, keepdim=True)
    g = torch.zeros_like(z).scatter_(1, idx, dg)
    return {"d_logits": c["scale"] * p * (g - (dg * p.gather(1, idx)).sum(dim=1, keepdim=True))}


def _rows(state, c):
    """The block's output rows of each token, [T, K, H] in 32 bits."""
    return state["h"].float()[state["dst_row"].long()].view(c["T"], c["K"], c["H"])


def _rms(x):
    return 1 / torch.sqrt((x * x).mean(dim=1, keepdim=True) + EPS)


def _norm_forward(state, c):
    y = state["residual"].float()
    if c["K"]:
        n = (_rows(state, c) * state["gate"][:, :, None]).sum(dim=1)
        if c["post"]:
            n = n * _rms(n) * state["w_post"]
        if c["scale"]:
            n = n * state["res_scale"] * state["row_scale"][:, None]
        y = y + n
    return y, y * _rms(y) * state["w_next"] if c["next"] else None


def _plain_norm(state, c):
    y, xn = _norm_forward(state, c)
    dtype = TYPES[c["dtype"]]
    out = {"y": y.to(dtype)} if c["K"] else {}
    if c["next"]:
        out["xn"] = xn.to(dtype)
    return out


def _plain_norm_bwd(state, c):
    dtype, out = TYPES[c["dtype"]], {}
    D = state["dy"].float()
    if c["next"]:
        y, dxn = state["y"].float(), state["dxn"].float()
        v = y * _rms(y)
        out["dw_next"] = (dxn * v).sum(dim=0)
        t = dxn * state["w_next"]
        D = D + _rms(y) * (t - v * (t * v).mean(dim=1, keepdim=True))
    out["d_res"] = D.to(dtype)
    if not c["K"]:
        return out
    rows, gate = _rows(state, c), state["gate"]
    z = (rows * gate[:, :, None]).sum(dim=1)
    u = z * _rms(z) if c["post"] else z
    n = u * state["w_post"] if c["post"] else u
    P = D
    if c["scale"]:
        out["d_scale"] = (D * state["res_scale"] * n).sum(dim=1)
        P = P * state["row_scale"][:, None]
        out["d_res_scale"] = (P * n).sum(dim=0)
        P = P * state["res_scale"]
    if c["post"]:
        out["dw_post"] = (P * u).sum(dim=0)
        P = P * state["w_post"]
        P = _rms(z) * (P - u * (P * u).mean(dim=1, keepdim=True))
    out["d_gate"] = (rows * P[:, None, :]).sum(dim=2)
    dh = torch.empty_like(state["h"])
    dh[state["dst_row"].long()] = (gate[:, :, None] * P[:, None, :]).to(dtype).view(-1, c["H"])
    out["dh"] = dh
    return out


def _plain_ckpt(state, c):
    x = state["gu"].float()
    rows, n = x.shape
    x = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(rows, -1, BLOCK)
    m, e = torch.frexp(x.abs().amax(dim=2, keepdim=True))  # amax = m 2^e, 1/2 <= m < 1
    e = torch.clamp(e - 7 + (m > 127 / 128).int(), min=-126)  # the least with amax <= 127 * 2^e
    held = torch.round(torch.ldexp(x, -e)).to(torch.int8)  # halves to even
    x = torch.ldexp(held.float(), e).view(rows, -1)[:, :n]
    g, u = x[:, :n // 2], x[:, n // 2:]
    dtype = TYPES[c["dtype"]]
    return {"gu": x.to(dtype), "act": (g / (1 + torch.exp(-g)) * u).to(dtype)}


_PLAIN = {"gate": _plain_gate, "gate_bwd": _plain_gate_bwd, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd,
          "ckpt": _plain_ckpt}


# ---- through the library ---------------------------------------------------------------------------------------------


def _buffers(state, make):
    """A program's output buffers and workspace: made at its first call, kept beside its inputs."""
    if "buffers" not in state:
        state["buffers"] = make()
    return state["buffers"]


def _empty(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _mode(L, c):
    mode = L.MOE_GATE_SIGMOID if c["score"] == "sigmoid" else L.MOE_GATE_SOFTMAX
    return mode | (L.MOE_GATE_RENORM if c["renorm"] else 0) | (L.MOE_GATE_GROUP_MAX if c["group_max"] else 0)


def _own_gate(state, c):
    from token_dispatch_gb300 import _lib as L
    T, K = c["T"], c["K"]
    b = _buffers(state, lambda: {"idx": _empty(T, K, dtype=torch.int32), "gate": _empty(T, K)})
    L.moe_gate(state["logits"], state["bias"], T, c["E"], K, c["groups"], c["topk_groups"], _mode(L, c), c["scale"],
               b["idx"], b["gate"])
    return b


def _own_gate_bwd(state, c):
    from token_dispatch_gb300 import _lib as L
    b = _buffers(state, lambda: {"d_logits": _empty(c["T"], c["E"])})
    L.moe_gate_bwd(state["d_gate"], state["logits"], state["idx"], c["T"], c["E"], c["K"], _mode(L, c), c["scale"],
                   b["d_logits"])
    return b


def _own_norm(state, c):
    from token_dispatch_gb300 import _lib as L
    T, H, dtype = c["T"], c["H"], TYPES[c["dtype"]]

    def make():
        b = {"y": _empty(T, H, dtype=dtype)} if c["K"] else {}
        if c["next"]:
            b["xn"] = _empty(T, H, dtype=dtype)
        return b
    b = _buffers(state, make)
    L.moe_combine_norm(state["h"], state["gate"], state["dst_row"], state["row_scale"], state["residual"],
                       state["w_post"], state["res_scale"], state["w_next"], EPS, T, H, c["K"],
                       L.MOE_BF16 if c["dtype"] == "bf16" else L.MOE_F32, b.get("y"), b.get("xn"))
    return b


def _own_norm_bwd(state, c):
    from token_dispatch_gb300 import _lib as L
    T, H, K, dtype = c["T"], c["H"], c["K"], TYPES[c["dtype"]]

    def make():
        b = {"d_res": _empty(T, H, dtype=dtype)}
        if K:
            b.update(dh=_empty(T * K, H, dtype=dtype), d_gate=_empty(T, K))
        if c["scale"]:
            b.update(d_scale=_empty(T), d_res_scale=_empty(H))
        if c["post"]:
            b["dw_post"] = _empty(H)
        if c["next"]:
            b["dw_next"] = _empty(H)
        return b, _empty(L.moe_workspace_bytes(L.MOE_OP_COMBINE_NORM_BWD, T, H, 0, K, 0), dtype=torch.uint8)
    b, ws = _buffers(state, make)
    L.moe_combine_norm_bwd(state["dy"], state["dxn"], state["h"], state["gate"], state["dst_row"], state["row_scale"],
                           state["y"], state["w_post"], state["res_scale"], state["w_next"], EPS, T, H, K,
                           L.MOE_BF16 if c["dtype"] == "bf16" else L.MOE_F32, b["d_res"], b.get("dh"),
                           b.get("d_gate"), b.get("d_scale"), b.get("dw_post"), b.get("d_res_scale"),
                           b.get("dw_next"), ws, ws.numel())
    return b


def _own_ckpt(state, c):
    from token_dispatch_gb300 import _lib as L
    rows, Hp, dtype = c["rows"], c["Hp"], TYPES[c["dtype"]]
    b, q, e = _buffers(state, lambda: (
        {"gu": _empty(rows, 2 * Hp, dtype=dtype), "act": _empty(rows, Hp, dtype=dtype)},
        _empty(rows, 2 * Hp, dtype=torch.int8), _empty(rows, -(-2 * Hp // BLOCK), dtype=torch.uint8)))
    cdt = L.MOE_BF16 if c["dtype"] == "bf16" else L.MOE_F32
    L.moe_ckpt_pack(state["gu"], rows, 2 * Hp, cdt, q, e)
    L.moe_ckpt_swiglu(q, e, rows, Hp, cdt, b["gu"], b["act"])
    return b


_OWN = {"gate": _own_gate, "gate_bwd": _own_gate_bwd, "norm": _own_norm, "norm_bwd": _own_norm_bwd, "ckpt": _own_ckpt}


# ---- in 64 bits, apart from the plain forms --------------------------------------------------------------------------


def exact(case, seed):
    s = _inputs(case, seed)
    if case["kind"] == "gate_bwd":
        s["idx"] = prepare(case, seed)["idx"]
    if case["kind"] == "norm_bwd":
        s["y"] = prepare(case, seed)["y"]
    return _EXACT[case["kind"]](s, case)


def _exact_gate(s, c):
    T, E, G, K = c["T"], c["E"], c["groups"], c["K"]
    z = s["logits"].cpu().numpy().astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        p = np.reciprocal(1 + np.exp(-z)) if c["score"] == "sigmoid" else np.exp(z - np.logaddexp.reduce(z, axis=1)[:, None])
    key = p + (0 if s["bias"] is None else s["bias"].cpu().numpy().astype(np.float64))
    key[np.isneginf(z)] = -np.inf
    tier = np.zeros((T, E), np.int64)  # 0: may be chosen, 1: its group is behind
    if c["topk_groups"] < G:
        parts = key.reshape(T, G, -1)
        top = parts.max(axis=2)
        if not c["group_max"] and E > G:
            rest = parts.copy()
            np.put_along_axis(rest, parts.argmax(axis=2)[:, :, None], -np.inf, axis=2)
            two = rest.max(axis=2)
            top = np.where(np.isneginf(two), top, top + np.where(np.isneginf(two), 0, two))
        # a group's place: how many are ahead of it, by value and then by number
        ahead = (top[:, None, :] > top[:, :, None]) | ((top[:, None, :] == top[:, :, None])
                                                       & (np.arange(G)[None, None, :] < np.arange(G)[None, :, None]))
        tier = np.repeat(ahead.sum(axis=2) >= c["topk_groups"], E // G, axis=1).astype(np.int64)
    order = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -key, tier), axis=1)[:, :K]
    gate = np.take_along_axis(p, order, axis=1)
    if c["renorm"]:
        gate /= gate.sum(axis=1, keepdims=True)
    return {"idx": order.astype(np.int32), "gate": c["scale"] * gate}


def _exact_gate_bwd(s, c):
    z = s["logits"].double().requires_grad_()
    p = torch.special.expit(z) if c["score"] == "sigmoid" else torch.softmax(z, dim=1)
    gate = torch.gather(p, 1, s["idx"].long())
    if c["renorm"]:
        gate = gate / gate.sum(dim=1, keepdim=True)
    return {"d_logits": torch.autograd.grad(c["scale"] * gate, z, s["d_gate"].double())[0]}


def _exact_block(leaf, dst_row, c):
    """The block's scaled and normed output from fp64 leaves."""
    o = torch.einsum("tk,tkh->th", leaf["gate"], leaf["h"][dst_row.long()].reshape(c["T"], c["K"], c["H"]))
    if c["post"]:
        o = o / (o.square().mean(dim=1, keepdim=True) + EPS).sqrt() * leaf["w_post"]
    if c["scale"]:
        o = torch.einsum("th,t,h->th", o, leaf["row_scale"], leaf["res_scale"])
    return o


def _leaves(s):
    return {k: v.double() for k, v in s.items() if v is not None and k not in ("dst_row", "case")}


def _exact_norm(s, c):
    x = _leaves(s)
    y = x["residual"] + _exact_block(x, s["dst_row"], c) if c["K"] else x["residual"]
    out = {"y": y} if c["K"] else {}
    if c["next"]:
        out["xn"] = y / (y.square().mean(dim=1, keepdim=True) + EPS).sqrt() * x["w_next"]
    return out


def _exact_norm_bwd(s, c):
    x, out = {k: v.requires_grad_() for k, v in _leaves(s).items()}, {}
    d = x["dy"].detach()
    if c["next"]:  # the next norm at the stored y
        xn = x["y"] / (x["y"].square().mean(dim=1, keepdim=True) + EPS).sqrt() * x["w_next"]
        more, out["dw_next"] = torch.autograd.grad(xn, (x["y"], x["w_next"]), x["dxn"].detach())
        d = d + more
    out["d_res"] = d
    if c["K"]:
        names = {"h": "dh", "gate": "d_gate"}
        if c["post"]:
            names["w_post"] = "dw_post"
        if c["scale"]:
            names.update(row_scale="d_scale", res_scale="d_res_scale")
        got = torch.autograd.grad(_exact_block(x, s["dst_row"], c), [x[k] for k in names], d)
        out.update(zip(names.values(), got))
    return out


def _exact_ckpt(s, c):
    x = s["gu"].double()
    n = x.shape[1]
    x = torch.cat([x, x.new_zeros(x.shape[0], -n % BLOCK)], dim=1).unflatten(1, (-1, BLOCK))
    top = x.abs().amax(dim=2, keepdim=True)
    step = torch.exp2(torch.floor(torch.log2(top.clamp_min(2.0 ** -120))) - 7)
    for _ in range(3):  # the least power of two that the block fits in, whatever the logarithm's last bit
        step = torch.where(127 * step < top, 2 * step, step)
    x = (torch.round(x / step) * step).flatten(1)[:, :n]
    g, u = x.split(n // 2, dim=1)
    return {"gu": x, "act": torch.special.expit(g) * g * u}


_EXACT = {"gate": _exact_gate, "gate_bwd": _exact_gate_bwd, "norm": _exact_norm, "norm_bwd": _exact_norm_bwd,
          "ckpt": _exact_ckpt}
