"""The operators on the experts' weight tensors, as cases to time and compare: weights in 4 bits with group scales,
the expert FFN that reads them, and the orthogonalised update of a training step.

``run`` computes a case in its plain form (elementary torch operations) or, where ``own`` is true, through the
library's calls.  ``exact`` states the same result in 64 bits, written apart from the plain form.

Kinds of cases:
  ffn   act = silu(x Wg) * (x Wu), h = act Wd^T of routed rows, weights of 4 bits
  pack  a weight tensor brought into 4 bits, and restored
  orth  Newton-Schulz steps on a batch of matrices
  muon  momentum, Newton-Schulz steps, and the weights' update
"""
import math

import torch

own = False

EPS = 1e-7
COEF = (3.4445, -4.7750, 2.0315)
STEPS = 5
BETA, LR, DECAY = 0.95, 3e-4, 0.1
BLOCK = 128  # inputs of an output's row that lie together in the packed form
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one token of a decoding step through the 384-expert layer
        _ffn("ffn_T1_E384_H7168", 1, 7168, 384, 8, 2048, 128),
        # a decoding step of sixteen sequences through the two-expert layer
        _ffn("ffn_T16_E8_Hp14336", 16, 4096, 8, 2, 14336, 64),
        # a decoding step of sixty-four sequences through the fine-grained layer
        _ffn("ffn_T64_E64_H2048", 64, 2048, 64, 6, 1408, 32),
        # odd sizes: groups that end behind the rows, experts without rows
        _ffn("ffn_T23_H1000_Hp712", 23, 1000, 48, 3, 712, 64),
        # a prompt: some 380 rows an expert
        _ffn("ffn_T4096_E64_H2048", 4096, 2048, 64, 6, 1408, 128),
        # the fine-grained layer's up projection after training, brought into 4 bits
        _pack("pack_E64_2048x1408", 64, 2048, 1408, 0, 32),
        # a ragged fp32 down projection
        _pack("pack_f32_E5_1000x712", 5, 1000, 712, 1, 128, dtype="f32"),
        # the small fp32 layer's experts
        _orth("orth_E8_128x256", 8, 128, 256, dtype="f32"),
        # one tall matrix: the 384-expert router's weights
        _orth("orth_E1_7168x384", 1, 7168, 384, dtype="f32"),
        # odd sizes
        _orth("orth_E3_1001x777", 3, 1001, 777),
        # an update of the fine-grained layer's experts
        _muon("muon_E64_2048x1408", 64, 2048, 1408),
        # an update of the two-expert layer's: the largest
        _muon("muon_E8_4096x14336", 8, 4096, 14336),
    ]


def _ffn(name, T, H, E, K, Hp, group):
    return {"name": name, "kind": "ffn", "T": T, "H": H, "E": E, "K": K, "Hp": Hp, "group": group}


def _pack(name, E, rows, cols, axis, group, dtype="bf16"):
    return {"name": name, "kind": "pack", "E": E, "rows": rows, "cols": cols, "axis": axis, "group": group,
            "dtype": dtype}


def _orth(name, E, M, N, dtype="bf16"):
    return {"name": name, "kind": "orth", "E": E, "M": M, "N": N, "dtype": dtype}


def _muon(name, E, M, N, nesterov=True):
    return {"name": name, "kind": "muon", "E": E, "M": M, "N": N, "dtype": "bf16", "nesterov": nesterov}


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    kind = rng.choice(("ffn", "ffn", "ffn", "pack", "orth", "orth", "muon"))
    if kind == "ffn":
        H = 8 * _log(rng, 8, 896)
        Hp = 8 * _log(rng, 8, 1792)
        E = _log(rng, 1, max(1, min(384, 469762048 // (H * Hp))))
        K = rng.randint(1, min(E, 8))
        T = _log(rng, 1, max(1, min(4096, 24576 * 2048 * 1408 // (H * Hp * K))))
        c = _ffn("", T, H, E, K, Hp, rng.choice((32, 64, 128)))
    elif kind == "pack":
        rows, cols = 8 * _log(rng, 8, 896), 8 * _log(rng, 8, 896)
        E = _log(rng, 1, max(1, min(128, 64 * 2048 * 1408 // (rows * cols))))
        c = _pack("", E, rows, cols, rng.randint(0, 1), rng.choice((32, 64, 128)),
                  dtype=rng.choice(("bf16", "bf16", "f32")))
    else:
        m = _log(rng, 16, 4096)
        n = _log(rng, m, min(14336, 8 * m))
        n = max(n, min(m + m // 8, 14336))  # a lone nearly singular direction says nothing about the rest
        cost = m * m * (3 * n + m)
        E = _log(rng, 1, max(1, min(64, 64 * 1408 * 1408 * (3 * 2048 + 1408) // cost)))
        M, N = (m, n) if rng.random() < 0.5 else (n, m)
        if kind == "orth":
            c = _orth("", E, M, N, dtype=rng.choice(("bf16", "f32")))
        else:
            c = _muon("", E, M, N, nesterov=rng.random() < 0.7)
    del c["name"]
    return c


def _up(n, k):
    return -(-n // k) * k


def work(case):
    c = case
    if c["kind"] == "ffn":
        R = c["T"] * c["K"]
        met = c["E"] * (1 - (1 - c["K"] / c["E"]) ** c["T"])  # experts that have rows, on average
        n = c["H"] * c["Hp"]
        rows = 2 * c["H"] * (c["T"] + R) + 2 * R * c["Hp"]  # x, h, act
        return {"bytes": met * 3 * n * (0.5 + 2 / c["group"]) + rows, "flops": 6 * R * n}
    n = c["E"] * c["rows"] * c["cols"] if c["kind"] == "pack" else c["E"] * c["M"] * c["N"]
    s = 2 if c["dtype"] == "bf16" else 4
    if c["kind"] == "pack":
        return {"bytes": 2 * s * n + 2 * n * (0.5 + 2 / c["group"]), "flops": 4 * n}
    m, l = sorted((c["M"], c["N"]))
    flops = STEPS * c["E"] * (3 * m * m * l + m * m * m)  # half of each symmetric product
    if c["kind"] == "orth":
        return {"bytes": (s + 2) * n, "flops": flops}
    return {"bytes": (4 + 8 + 2 * s) * n, "flops": flops}


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _codes(g, E, out, inp, group):
    """Random codes and scales of a weight tensor with about the spread of 1 / sqrt(inp)."""
    blocks = _up(inp, BLOCK) // BLOCK
    q = torch.randint(-2 ** 31, 2 ** 31, (E, out, blocks * BLOCK // 8), generator=g, device="cuda", dtype=torch.int32)
    # scales of 5 significant bits
    s = torch.randint(16, 32, (E, out, blocks * BLOCK // group), generator=g, device="cuda", dtype=torch.int32)
    return q, (s.float() * 2.0 ** (-7 - math.ceil(math.log2(inp) / 2))).to(torch.bfloat16)


def _update(g, E, M, N):
    """What gradients of a weight matrix look like: noise, and a few directions that stand out of it."""
    u = _randn(g, E, M, N)
    return u.baddbmm_(_randn(g, E, M, 4), _randn(g, E, 4, N))


def _inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    c, g = case, torch.Generator(device="cuda")
    g.manual_seed(seed)
    if c["kind"] == "ffn":
        T, H, E, K, Hp, G = (c[k] for k in ("T", "H", "E", "K", "Hp", "group"))
        idx = torch.rand((T, E), generator=g, device="cuda").topk(K, dim=1).indices.reshape(-1)
        order = torch.sort(idx, stable=True).indices
        count = torch.bincount(idx, minlength=E)
        cu = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        cu[1:] = count.cumsum(0)
        s = {"x": _randn(g, T, H).bfloat16(), "src_tok": (order // K).to(torch.int32), "cu": cu,
             "most": int(count.max())}
        s["q_gate"], s["s_gate"] = _codes(g, E, Hp, H, G)
        s["q_up"], s["s_up"] = _codes(g, E, Hp, H, G)
        s["q_down"], s["s_down"] = _codes(g, E, H, Hp, G)
        return s
    dtype = TYPES[c["dtype"]]
    if c["kind"] == "pack":
        w = _randn(g, c["E"], c["rows"], c["cols"]) * torch.exp(0.5 * _randn(g, c["E"], c["rows"], 1))
        return {"w": (w / math.sqrt(c["rows"])).to(dtype)}
    E, M, N = c["E"], c["M"], c["N"]
    if c["kind"] == "orth":
        return {"x": (1e-3 * _update(g, E, M, N)).to(dtype)}
    return {"g": 1e-4 * _update(g, E, M, N), "m": 1e-3 * _update(g, E, M, N),
            "w": (_randn(g, E, M, N) / math.sqrt(M)).to(dtype)}


def prepare(case, seed):
    c, s = case, dict(_inputs(case, seed), case=dict(case))
    if c["kind"] == "ffn":  # buffers and workspace that a decoding loop keeps
        R = c["T"] * c["K"]
        s["act"] = torch.empty((R, c["Hp"]), dtype=torch.bfloat16, device="cuda")
        s["h"] = torch.empty((R, c["H"]), dtype=torch.bfloat16, device="cuda")
    return s


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["kind"]](state, state["case"])


# ---- plain forms -----------------------------------------------------------------------------------------------------


def _restore(q, scale, inp, group):
    """[.., out, inp] in 32 bits of packed codes and scales."""
    lead = q.shape[:-1]
    # words of a block lie by their place among four first, then by the run of 32 that they belong to
    words = q.view(*lead, -1, 4, 4).transpose(-1, -2).unsqueeze(-1)
    shifts = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], dtype=torch.int32, device=q.device)
    codes = ((words >> shifts) & 15).to(torch.int8).reshape(*lead, -1, group)
    return ((codes.float() - 8) * scale.float().unsqueeze(-1)).view(*lead, -1)[..., :inp]


def _plain_ffn(state, c):
    T, H, E, K, Hp, G = (c[k] for k in ("T", "H", "E", "K", "Hp", "group"))
    R, cu, most = T * K, state["cu"].long(), state["most"]
    x = state["x"].float()[state["src_tok"].long()]
    row = torch.arange(R, device="cuda")
    expert = (row[:, None] >= cu[None, 1:]).sum(dim=1)
    if R <= E:  # each row with its expert's weights
        def weights(name, inp):
            return _restore(state["q_" + name][expert], state["s_" + name][expert], inp, G)
        x = x[:, :, None]
    else:  # each expert's rows side by side
        def weights(name, inp):
            return _restore(state["q_" + name], state["s_" + name], inp, G)
        place = expert * most + row - cu[expert]
        x = torch.zeros((E * most, H), device="cuda").index_copy_(0, place, x).view(E, most, H).transpose(1, 2)
    gate = torch.bmm(weights("gate", H), x)
    act = gate / (1 + torch.exp(-gate)) * torch.bmm(weights("up", H), x)
    out = {"act": act, "h": torch.bmm(weights("down", Hp), act)}
    return {k: (v[:, :, 0] if R <= E else v.transpose(1, 2).reshape(E * most, -1)[place]).to(torch.bfloat16)
            for k, v in out.items()}


def _plain_pack(state, c):
    w = state["w"].float()
    w = w.transpose(1, 2) if c["axis"] == 0 else w
    E, out, inp = w.shape
    x = torch.nn.functional.pad(w, (0, -inp % c["group"])).reshape(E, out, -1, c["group"])
    a = x.abs().amax(dim=-1, keepdim=True) / 7
    s = ((a.view(torch.int32) + 0x7ffff) & ~0x7ffff).view(torch.float32)  # 5 significant bits, up
    s = torch.clamp(s, min=2.0 ** -126)
    x = (torch.round(x / s) * s).view(E, out, -1)[:, :, :inp]
    x = x.transpose(1, 2) if c["axis"] == 0 else x
    return {"w": x.to(TYPES[c["dtype"]]).contiguous()}


def _newton_schulz(u):
    """Orthogonalised u [E, M, N] in 32 bits."""
    a, b, c = COEF
    tall = u.shape[1] > u.shape[2]
    x = u.transpose(1, 2) if tall else u
    norm = torch.sqrt((x.double() ** 2).sum(dim=(1, 2), keepdim=True))
    x = x / (norm + EPS).float()
    left = STEPS
    while left:
        s = torch.bmm(x, x.transpose(1, 2))
        x = torch.baddbmm(x, torch.baddbmm(s, s, s, beta=b, alpha=c), x, beta=a)
        left -= 1
    return x.transpose(1, 2) if tall else x


def _plain_orth(state, c):
    return {"o": _newton_schulz(state["x"].float()).to(torch.bfloat16)}


def _plain_muon(state, c):
    m = BETA * state["m"] + state["g"]
    u = state["g"] + BETA * m if c["nesterov"] else m
    w = (1 - LR * DECAY) * state["w"].float() - LR * _scale(c) * _newton_schulz(u)
    return {"m": m, "w": w.to(torch.bfloat16).contiguous()}


def _scale(c):
    return 0.2 * math.sqrt(max(c["M"], c["N"]))


_PLAIN = {"ffn": _plain_ffn, "pack": _plain_pack, "orth": _plain_orth, "muon": _plain_muon}

# ---- the library's calls ---------------------------------------------------------------------------------------------


def _lib():
    from token_dispatch_gb300 import _lib as L
    return L


def _workspace(L, op, T=0, H=0, E=0, K=0, Hp=0):
    n = L.moe_workspace_bytes(op, T, H, E, K, Hp)
    return (torch.empty(n, dtype=torch.uint8, device="cuda") if n else None), n


def _own_ffn(state, c):
    L = _lib()
    T, H, E, K, Hp, G = (c[k] for k in ("T", "H", "E", "K", "Hp", "group"))
    ws, n = _workspace(L, L.MOE_OP_EXPERT_FFN_W4, T=T, H=H, E=E, K=K, Hp=Hp)
    L.moe_expert_ffn_w4(state["x"], state["src_tok"], T, state["cu"], T * K, state["q_gate"], state["s_gate"],
                        state["q_up"], state["s_up"], state["q_down"], state["s_down"], E, H, Hp, G, L.MOE_BF16,
                        state["act"], state["h"], ws, n)
    return {"act": state["act"], "h": state["h"]}


def _own_pack(state, c):
    L = _lib()
    E, rows, cols, axis, G = (c[k] for k in ("E", "rows", "cols", "axis", "group"))
    dt = L.MOE_BF16 if c["dtype"] == "bf16" else L.MOE_F32
    out, inp = (cols, rows) if axis == 0 else (rows, cols)
    q = torch.empty((E, out, _up(inp, BLOCK) // 8), dtype=torch.int32, device="cuda")
    s = torch.empty((E, out, _up(inp, BLOCK) // G), dtype=torch.bfloat16, device="cuda")
    w = torch.empty_like(state["w"])
    L.moe_w4_pack(state["w"], E, rows, cols, axis, G, dt, q, s)
    L.moe_w4_unpack(q, s, E, rows, cols, axis, G, dt, w)
    return {"w": w}


def _own_orth(state, c):
    L = _lib()
    E, M, N = c["E"], c["M"], c["N"]
    ws, n = _workspace(L, L.MOE_OP_ORTHOGONALIZE, H=M, E=E, Hp=N)
    o = torch.empty((E, M, N), dtype=torch.bfloat16, device="cuda")
    L.moe_orthogonalize(state["x"], E, M, N, L.MOE_BF16 if c["dtype"] == "bf16" else L.MOE_F32, STEPS, *COEF, EPS, o,
                        ws, n)
    return {"o": o}


def _own_muon(state, c):
    L = _lib()
    E, M, N = c["E"], c["M"], c["N"]
    ws, n = _workspace(L, L.MOE_OP_MUON_STEP, H=M, E=E, Hp=N)
    # a training program updates in place (m and w as their own outputs); here the state is needed again
    m, w = torch.empty_like(state["m"]), torch.empty_like(state["w"])
    L.moe_muon_step(state["w"], state["g"], state["m"], E, M, N, L.MOE_BF16, BETA, c["nesterov"], LR, DECAY,
                    _scale(c), STEPS, *COEF, EPS, w, None, m, ws, n)
    return {"m": m, "w": w}


_OWN = {"ffn": _own_ffn, "pack": _own_pack, "orth": _own_orth, "muon": _own_muon}

# ---- the definition in 64 bits ---------------------------------------------------------------------------------------


def _value(q, scale, inp, group):
    """[out, inp] weights in 64 bits of one expert: code k of an output, one by one in order of its inputs."""
    k = torch.arange(inp, device=q.device)
    block, run, word, i = k // 128, k % 128 // 32, k % 32 // 8, k % 8
    bits = 4 * (i // 2) + 16 * (i % 2)
    at = block * 16 + word * 4 + run
    code = (q[:, at].long() >> bits) & 15
    return (code - 8).double() * scale.double()[:, k // group]


def _exact_ffn(s, c):
    G, cu = c["group"], s["cu"].tolist()
    h = torch.zeros((c["T"] * c["K"], c["H"]), dtype=torch.float64, device="cuda")
    act = torch.zeros((c["T"] * c["K"], c["Hp"]), dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        rows = slice(cu[e], cu[e + 1])
        if cu[e] == cu[e + 1]:
            continue
        x = s["x"].double()[s["src_tok"][rows].long()]
        g = x @ _value(s["q_gate"][e], s["s_gate"][e], c["H"], G).T
        u = x @ _value(s["q_up"][e], s["s_up"][e], c["H"], G).T
        act[rows] = g * torch.sigmoid(g) * u
        h[rows] = act[rows] @ _value(s["q_down"][e], s["s_down"][e], c["Hp"], G).T
    return {"act": act, "h": h}


def _exact_pack(s, c):
    w = s["w"].double()
    axis = 1 + c["axis"]
    out = torch.empty_like(w)
    for lo in range(0, w.shape[axis], c["group"]):
        part = w.narrow(axis, lo, min(c["group"], w.shape[axis] - lo))
        step = (part.abs().amax(dim=axis, keepdim=True).float() / 7).double()  # the rule is stated in 32 bits
        m, e = torch.frexp(step)
        step = torch.clamp(torch.ldexp(torch.ceil(m * 32), e - 5), min=2.0 ** -126)
        # and so is the quotient that is rounded
        out.narrow(axis, lo, part.shape[axis]).copy_(torch.round((part.float() / step.float()).double()) * step)
    return {"w": out}


def _exact_orth(u):
    a, b, c = COEF
    out = []
    for x in u:
        x = x.double()
        x = x / (torch.linalg.norm(x) + EPS)
        for _ in range(STEPS):  # the same polynomial, by the Gram matrix of the shorter side
            if x.shape[0] <= x.shape[1]:
                t = x @ x.T
                x = a * x + b * (t @ x) + c * (t @ (t @ x))
            else:
                t = x.T @ x
                x = a * x + b * (x @ t) + c * ((x @ t) @ t)
        out.append(x)
    return torch.stack(out)


def exact(case, seed):
    c = case
    if c["kind"] in ("orth", "muon"):
        m, l = sorted((c["M"], c["N"]))
        if 6 * STEPS * c["E"] * m * m * l > 1e13:  # about ten seconds
            return None
    s = _inputs(case, seed)
    if c["kind"] == "ffn":
        return _exact_ffn(s, c)
    if c["kind"] == "pack":
        return _exact_pack(s, c)
    if c["kind"] == "orth":
        return {"o": _exact_orth(s["x"])}
    m = BETA * s["m"].double() + s["g"].double()
    o = _exact_orth(s["g"].double() + BETA * m if c["nesterov"] else m)
    w = (1 - LR * DECAY) * s["w"].double() - LR * _scale(c) * o
    return {"m": m, "w": w}
