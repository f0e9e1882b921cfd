"""Cases of the router, the gates' gradient, the 8-bit activation checkpoints and the
MXFP4 experts: inputs, one pass of each through the library's entry points (``own``) or
in its plain form (elementary torch operations), the work a pass cannot do without, and
the results in 64 bits.

Every layer here is one rank (R = 1), whose plan is the stable order of the slots by
expert: the operators read a plan only through slot_map, src_index and cu_seqlens, so
one rank stands for any number of them.
"""
import math

import torch

own = False

BLOCK = 32                     # columns per shared scale
INF = float("inf")


# ------------------------------------------------------------------ cases
def _route(op, name, N, E, K, score, dtype, groups=1, top_groups=1, group_top=1, renorm=True,
           bias=False, off=0, scale=1.0):
    return dict(op=op, name=name, N=N, E=E, K=K, score=score, dtype=dtype, groups=groups,
                top_groups=top_groups, group_top=group_top, renorm=renorm, bias=bias, off=off,
                scale=scale)


def listed():
    return [
        # one token of a serving step through a grouped sigmoid router with a balance bias
        _route("route", "route_one_token", 1, 256, 8, "sigmoid", "fp32", 8, 4, 2, True, True, 0, 2.5),
        # the router of a training step: 8 ranks x 8192 tokens, 384 experts
        _route("route", "route_sigmoid_groups", 65536, 384, 8, "sigmoid", "fp32", 8, 4, 2, True,
               True, 0, 2.5),
        # the same step with a plain softmax router on bfloat16 logits (many exact ties)
        _route("route", "route_softmax_bf16", 65536, 384, 8, "softmax", "bf16"),
        # backward of a small layer's sigmoid router, an odd number of tokens
        _route("route_grad", "route_grad_sigmoid", 8191, 64, 4, "sigmoid", "fp32", bias=True),
        # backward of a softmax router whose gates are not renormalised: dense rows
        _route("route_grad", "route_grad_softmax", 32768, 128, 8, "softmax", "bf16", renorm=False),
        # gates' gradient of a tiny float32 layer with odd sizes
        dict(op="gate_grad", name="gate_grad_small", N=251, K=3, E=16, W=76, dtype="fp32"),
        # gates' gradient of an FFN of hidden size 7168
        dict(op="gate_grad", name="gate_grad_wide", N=16384, K=8, E=384, W=7168, dtype="bf16"),
        # checkpoint of a layer's input, and the permute that reads it in the backward pass
        dict(op="checkpoint_x", name="checkpoint_x_wide", N=16384, K=8, E=384, W=7168, dtype="bf16"),
        # checkpoint of the gate/up projection of a tiny float32 layer, forward and backward
        dict(op="checkpoint_h", name="checkpoint_h_small", N=256, K=2, E=16, Hp=64, dtype="fp32"),
        # the same of a training layer of 32768 tokens, intermediate size 1408
        dict(op="checkpoint_h", name="checkpoint_h_train", N=32768, K=8, E=128, Hp=1408, dtype="bf16"),
        # a serving step of 16 sequences, one token each, over 4-bit experts
        dict(op="mx", name="mx_decode", N=16, K=8, E=256, H=4096, Hp=1536, dtype="bf16"),
        # a prompt batch over the same experts
        dict(op="mx", name="mx_prompt", N=65536, K=8, E=256, H=4096, Hp=1536, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "gate_grad", "checkpoint_x", "checkpoint_h", "mx", "mx"])
    dtype = rng.choice(["bf16", "fp32"])
    N = _log(rng, 1, 65536)
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, 2, 384 // groups)
        top_groups = rng.randint(max(1, groups // 2), groups)
        K = rng.randint(1, min(8, top_groups * (E // groups)))
        bias = rng.random() < 0.5
        off = rng.randint(0, E // 8) if bias else 0     # experts switched off by the bias
        case = _route(op, None, N, E, K, rng.choice(["softmax", "sigmoid"]), dtype, groups,
                      top_groups, rng.choice([1, 2]), rng.random() < 0.6, bias, off,
                      rng.choice([1.0, 2.5]))
        del case["name"]
        return case
    K, E = rng.randint(1, 8), rng.choice([8, 16, 60, 128, 384])
    eb = 4 if dtype == "fp32" else 2
    if op in ("gate_grad", "checkpoint_x"):
        W = (16 // eb) * _log(rng, 4, 7168 * eb // 16)
        N = min(N, max(1, 16384 * 8 * 7168 * 2 // (K * W * eb * 2)), 32768)
        return dict(op=op, N=N, K=K, E=E, W=W, dtype=dtype)
    if op == "checkpoint_h":
        Hp = BLOCK * _log(rng, 1, 2048 // BLOCK)
        N = min(N, max(1, 32768 * 8 * 1408 * 2 // (K * Hp * eb)), 32768)
        return dict(op=op, N=N, K=K, E=E, Hp=Hp, dtype=dtype)
    H, Hp = 64 * _log(rng, 1, 7168 // 64), 64 * _log(rng, 1, 2048 // 64)
    E = rng.choice([8, 16, 60, 128, 256])
    N = min(N, max(1, 65536 * 8 * 4096 * 1536 // (K * H * Hp)))
    return dict(op=op, N=N, K=K, E=E, H=H, Hp=Hp, dtype=dtype)


def work(case):
    c, op, N, K = case, case["op"], case["N"], case["K"]
    eb = 4 if c["dtype"] == "fp32" else 2
    if op == "route":
        return {"bytes": N * (c["E"] * eb + K * 8) + 4 * c["E"] * c["bias"], "flops": 6 * N * c["E"]}
    if op == "route_grad":
        dense = c["score"] == "softmax" and not c["renorm"]
        gathered = 0 if dense or c["score"] == "softmax" else K * eb
        read = N * (c["E"] * eb if dense else gathered)
        return {"bytes": read + N * (c["E"] * eb + K * 12), "flops": (6 if dense else 1) * N * c["E"]}
    NK = N * K
    if op == "gate_grad":
        return {"bytes": NK * c["W"] * 4 + N * c["W"] * eb + NK * 8, "flops": 2 * NK * c["W"]}
    if op == "checkpoint_x":
        W = c["W"]
        held = N * (W + -(-W // BLOCK))
        return {"bytes": N * W * eb + 2 * held + NK * W * eb + NK * 4, "flops": 4 * N * W + NK * W}
    if op == "checkpoint_h":
        Hp = c["Hp"]
        held = 2 * Hp + 2 * Hp // BLOCK
        forward = NK * (8 * Hp + eb * Hp + held)
        backward = NK * (held + 4 * Hp + eb * 3 * Hp + 12)
        return {"bytes": forward + backward, "flops": 40 * NK * Hp}
    touched = c["E"] * (1.0 - (1.0 - min(1.0, K / c["E"])) ** N)      # experts expected to have rows
    return {"bytes": int(N * c["H"] * eb + touched * c["H"] * c["Hp"] * 17 / 32 + NK * c["Hp"] * 4 + NK * 4),
            "flops": 2 * NK * c["H"] * c["Hp"]}


# ------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, dtype=torch.float32, std=1.0):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=g).to(dtype)


def _plan(g, N, E, K):
    """A skewed router's choice of K of E experts for every token, and its plan on one rank."""
    score = _normal(g, (N, E)) + 0.3 * _normal(g, (E,))
    topk = torch.sort(score, dim=1, descending=True).indices[:, :K].contiguous()
    order = torch.sort(topk.reshape(-1), stable=True).indices            # buffer position -> slot
    slot_map = torch.empty_like(order)
    slot_map[order] = torch.arange(N * K, device="cuda")
    counts = torch.bincount(topk.reshape(-1), minlength=E)
    cu = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    cu[1:] = torch.cumsum(counts, 0)
    gates = torch.softmax(torch.gather(score, 1, topk), 1)
    return slot_map.int(), order.int(), cu.int(), gates


def _fp4_codes(v):
    """e2m1 codes of v (|v| <= 6), to nearest, ties to the even code."""
    a = v.abs()
    code = torch.zeros(v.shape, dtype=torch.uint8, device=v.device)
    for mid, ties_up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False),
                         (3.5, True), (5.0, False)):
        code += (a >= mid) if ties_up else (a > mid)
    return code + 8 * torch.signbit(v).to(torch.uint8)


def _shared_exponent(amax, top):
    """The smallest e in [-127, 127] with amax <= top * 2^e."""
    m, e = torch.frexp(amax / top)                    # amax / top = m * 2^e, m in [0.5, 1)
    e = torch.where(m == 0.5, e - 1, e)
    return torch.where(amax == 0, -127, e).clamp(-127, 127)


def _pow2(e):
    """2^e as float32 for whole e in [-127, 127], from its bits."""
    return torch.where(e > -127, (e.int() + 127) << 23, 1 << 22).int().view(torch.float32)


def _pack_weight(w, H):
    """One expert's weight [H, Hp] in 4 bits: the packed values and the scales, both in the
    order the product reads them (tiles of 16 columns by 128 k; a lane's 32 values lie together)."""
    Hp = w.shape[1]
    KT, KC = -(-H // 128), -(-H // 512)
    wt = torch.zeros((Hp, KC * 512), dtype=torch.float32, device=w.device)
    wt[:, :H] = w.t()
    blocks = wt.view(Hp, -1, BLOCK)
    e = _shared_exponent(blocks.abs().amax(-1), 6.0)
    code = _fp4_codes(blocks * _pow2(-e).unsqueeze(-1))
    q = code[..., 0::2] | (code[..., 1::2] << 4)                         # [Hp, K/32, 16]
    q = q[:, :KT * 4].reshape(Hp // 16, 16, KT, 4, 16).permute(0, 2, 3, 1, 4)
    e[:, -(-H // 32):] = -127                                            # k past H: scale byte 0
    s = (e + 127).to(torch.uint8).view(Hp // 16, 16, KC, 4, 4).permute(0, 2, 4, 1, 3)
    return q.reshape(Hp // 16, KT, 64, 16), s.reshape(Hp // 16, KC, 64, 4)


def prepare(case, seed):
    c, op, N, K, E = case, case["op"], case["N"], case["K"], case["E"]
    g = _rng(seed)
    dt = _dtype(c)
    st = {"case": c}
    f32 = dict(dtype=torch.float32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    if op in ("route", "route_grad"):
        st["logits"] = (_normal(g, (N, E)) + 0.5 * _normal(g, (E,))).to(dt)
        st["bias"] = None
        if c["bias"]:
            st["bias"] = _normal(g, (E,), std=0.05)
            if c["off"]:
                gone = torch.randperm(E, generator=g, device="cuda")[:c["off"]]
                st["bias"][gone] = -INF
        if op == "route_grad":
            st["ids"], st["gates"] = _route_plain(st["logits"], st["bias"], c)
            st["dgates"] = _normal(g, (N, K))
    else:
        st["slot_map"], st["src_index"], cu, gates = _plan(g, N, E, K)
        if op == "gate_grad":
            st["out"] = _normal(g, (N * K, c["W"]))
            st["dy"] = _normal(g, (N, c["W"]), dt)
        elif op == "checkpoint_x":
            st["x"] = _normal(g, (N, c["W"]), dt)
        elif op == "checkpoint_h":
            st["h"] = _normal(g, (N * K, 2 * c["Hp"]))
            st["da"] = _normal(g, (N * K, c["Hp"]))
            st["gates"] = gates.contiguous()
        else:
            H, Hp = c["H"], c["Hp"]
            st["x"] = _normal(g, (N, H), dt)
            KT, KC = -(-H // 128), -(-H // 512)
            st["wq"] = torch.empty((E, Hp // 16, KT, 64, 16), dtype=torch.uint8, device="cuda")
            st["ws"] = torch.empty((E, Hp // 16, KC, 64, 4), dtype=torch.uint8, device="cuda")
            for e in range(E):
                st["wq"][e], st["ws"][e] = _pack_weight(_normal(g, (H, Hp), std=H ** -0.5), H)
            st["cu"] = cu
            st["bounds"] = cu.tolist()
    if not own:
        return st
    # the shape, the workspace and the output buffers that a layer keeps
    from redundant_expert_balancing_amd import _lib as L, checkpoint, mx
    st["L"] = L
    H, Hp = c.get("H", c.get("W", 64)), c.get("Hp", c.get("W", 64))
    ty = L.FP32 if c["dtype"] == "fp32" else L.BF16
    serving = op == "mx"
    sh = st["shape"] = L.Shape(1, N, E, K, 0 if serving else E, H, Hp,
                               L.INFER if serving else L.TRAIN, ty)
    NK = N * K
    if op in ("route", "route_grad"):
        st["router"] = L.Router(L.SIGMOID if c["score"] == "sigmoid" else L.SOFTMAX, ty, c["groups"],
                                c["top_groups"], c["group_top"], int(c["renorm"]), c["scale"])
    if op == "route":
        st["ids"], st["gates"] = torch.empty((N, K), **i32), torch.empty((N, K), **f32)
    elif op == "route_grad":
        st["dlogits"] = torch.empty((N, E), dtype=dt, device="cuda")
    elif op == "gate_grad":
        st["dgates"] = torch.empty((N, K), **f32)
    elif op == "checkpoint_x":
        st["q"], st["s"] = checkpoint.buffers(N, c["W"])
        st["xp"] = torch.empty((NK, c["W"]), dtype=dt, device="cuda")
    elif op == "checkpoint_h":
        st["q"], st["s"] = checkpoint.buffers(NK, 2 * Hp)
        st["act"], st["act_b"] = (torch.empty((NK, Hp), dtype=dt, device="cuda") for _ in range(2))
        st["dh"] = torch.empty((NK, 2 * Hp), dtype=dt, device="cuda")
        st["dgates"] = torch.empty((N, K), **f32)
    else:
        st["xq"], st["xs"] = mx.buffers(N, H)
        st["work"] = torch.empty((L.moonep_workspace_bytes(sh) // 4,), **i32)
        L.moonep_workspace_init(sh, st["work"])
        st["c"] = torch.empty((NK, Hp), **f32)
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    c, L, sh = st["case"], st["L"], st["shape"]
    op = c["op"]
    if op == "route":
        L.moonep_route(sh, st["router"], st["logits"], st["bias"], st["ids"], st["gates"])
        return st["ids"], st["gates"]
    if op == "route_grad":
        L.moonep_route_backward(sh, st["router"], st["logits"], st["bias"], st["ids"], st["gates"],
                                st["dgates"], st["dlogits"])
        return st["dlogits"]
    if op == "gate_grad":
        L.moonep_gate_grad(sh, c["W"], st["out"], st["slot_map"], st["dy"], st["dgates"])
        return st["dgates"]
    if op == "checkpoint_x":
        L.moonep_checkpoint_quantize(sh, c["W"], st["x"], st["q"], st["s"])
        L.moonep_checkpoint_dispatch(sh, c["W"], st["q"], st["s"], st["slot_map"], st["xp"])
        return st["xp"]
    if op == "checkpoint_h":
        L.moonep_swiglu_checkpoint(sh, st["h"], st["act"], st["q"], st["s"])
        L.moonep_swiglu_backward_checkpoint(sh, st["q"], st["s"], st["da"], st["src_index"],
                                            st["gates"], st["act_b"], st["dh"], st["dgates"])
        return st["act"], st["act_b"], st["dh"], st["dgates"]
    L.moonep_mx_quantize(sh, c["N"], c["H"], st["x"], st["xq"], st["xs"])
    L.moonep_mx_grouped_gemm(sh, st["xq"], st["xs"], st["src_index"], st["wq"], st["ws"], st["cu"],
                             st["c"], st["work"])
    return st["c"]


def _run_plain(st):
    c = st["case"]
    op, dt = c["op"], _dtype(c)
    if op == "route":
        return _route_plain(st["logits"], st["bias"], c)
    if op == "route_grad":
        return _route_grad_plain(st["logits"], st["bias"], st["ids"], st["gates"], st["dgates"], c)
    if op == "gate_grad":
        rows = st["out"][st["slot_map"].long()].view(c["N"], c["K"], c["W"])
        return (rows * st["dy"].float().unsqueeze(1)).sum(-1)
    if op == "checkpoint_x":
        held = _e4m3_plain(st["x"].float())
        return held.to(dt)[st["src_index"].long() // c["K"]]
    if op == "checkpoint_h":
        act = _swiglu_plain(*_split(st["h"]))
        gate, up = _split(_e4m3_plain(st["h"]))
        w = st["gates"].reshape(-1)[st["src_index"].long()]
        act_b, da = _swiglu_plain(gate, up), st["da"]
        dgates = torch.empty_like(w)
        dgates[st["src_index"].long()] = (act_b * da).sum(-1)
        dag = da * w.unsqueeze(1)
        s = 1.0 / (1.0 + torch.exp(-gate))
        dh = _join(dag * up * s * (1.0 + gate * (1.0 - s)), dag * gate * s)
        return (act.to(dt), (act_b * w.unsqueeze(1)).to(dt), dh.to(dt),
                dgates.view(c["N"], c["K"]))
    H, Hp, K = c["H"], c["Hp"], c["K"]
    x = st["x"].float()
    blocks = x.view(c["N"], H // BLOCK, BLOCK)
    e = _shared_exponent(blocks.abs().amax(-1), 6.0).unsqueeze(-1)
    x = (_fp4_values(_fp4_codes(blocks * _pow2(-e))) * _pow2(e)).view(c["N"], H)
    token = st["src_index"].long() // K
    out = torch.empty((c["N"] * K, Hp), dtype=torch.float32, device="cuda")
    for i in range(c["E"]):
        lo, hi = st["bounds"][i], st["bounds"][i + 1]
        if hi > lo:
            out[lo:hi] = x[token[lo:hi]] @ _weight_plain(st["wq"][i], st["ws"][i], H).t()
    return out


def _route_plain(logits, bias, c):
    """Chosen experts and gates: selection in 64 bits (values next to a border), gates in 32."""
    N, E = logits.shape
    l = logits.double()
    if bias is not None:
        l = torch.where(bias == -INF, -INF, l)
    masked = l == -INF
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        ex = torch.where(masked, 0.0, torch.exp(l - l.amax(1, keepdim=True)))
        s = ex / ex.sum(1, keepdim=True)
    biased = s if bias is None else s + bias.double()
    key = torch.where(masked, -INF, l if bias is None else biased)
    if c["groups"] > 1:
        G = c["groups"]
        if c["group_top"] == 1:
            score = key.view(N, G, -1).amax(-1)
        else:
            best = torch.where(masked, -INF, biased).view(N, G, -1).sort(-1, descending=True).values
            second = best[..., 1]
            score = best[..., 0] + torch.where(second == -INF, 0.0, second)
        rank = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        kept = torch.zeros((N, G), dtype=torch.bool, device=l.device).scatter_(1, rank, True)
        kept = kept.unsqueeze(-1).expand(N, G, E // G).reshape(N, E)
        key = torch.where(kept, key, -INF)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["K"]]
    chosen = torch.gather(key, 1, ids) != -INF
    lk = torch.gather(l, 1, ids).float()
    if not c["renorm"]:
        if c["score"] == "sigmoid":
            gates = 1.0 / (1.0 + torch.exp(-lk))
        else:
            lf = l.float()
            m = lf.amax(1, keepdim=True)
            gates = torch.exp(lk - m) / torch.exp(lf - m).sum(1, keepdim=True)
    elif c["score"] == "sigmoid":
        gates = torch.where(chosen, 1.0 / (1.0 + torch.exp(-lk)), 0.0)
        gates = gates / gates.sum(1, keepdim=True)
    else:
        ex = torch.where(chosen, torch.exp(lk - torch.where(chosen, lk, -INF).amax(1, keepdim=True)), 0.0)
        gates = ex / ex.sum(1, keepdim=True)
    return ids.int(), torch.where(chosen, gates * c["scale"], 0.0)


def _route_grad_plain(logits, bias, ids, gates, dgates, c):
    l = logits.float()
    if bias is not None:
        l = torch.where(bias == -INF, -INF, l)
    ids = ids.long()
    out = torch.zeros_like(l)
    if c["renorm"]:
        d = gates * (dgates - (gates / c["scale"] * dgates).sum(1, keepdim=True))
    else:
        d = gates * dgates
    if c["score"] == "sigmoid":
        lk = torch.gather(l, 1, ids)
        d = torch.where(gates == 0, 0.0, d / (1.0 + torch.exp(lk)))
    elif not c["renorm"]:
        ex = torch.exp(l - l.amax(1, keepdim=True))
        out = -ex / ex.sum(1, keepdim=True) * d.sum(1, keepdim=True)
    return out.scatter_add_(1, ids, d).to(logits.dtype)


def _e4m3_plain(v):
    """v [rows, W] rounded to e4m3 with a power-of-two scale per 32 columns, as float32."""
    rows, W = v.shape
    pad = torch.zeros((rows, -(-W // BLOCK) * BLOCK), dtype=torch.float32, device=v.device)
    pad[:, :W] = v
    blocks = pad.view(rows, -1, BLOCK)
    e = _shared_exponent(blocks.abs().amax(-1), 448.0).unsqueeze(-1)
    q = (blocks * _pow2(-e)).to(torch.float8_e4m3fn).float()
    return (q * _pow2(e)).view(rows, -1)[:, :W]


def _split(h):
    """Gate and up columns of h [rows, 2*Hp], interleaved in blocks of 32."""
    v = h.view(h.shape[0], -1, 2, BLOCK)
    return v[:, :, 0].reshape(h.shape[0], -1), v[:, :, 1].reshape(h.shape[0], -1)


def _join(gate, up):
    rows = gate.shape[0]
    return torch.stack((gate.view(rows, -1, BLOCK), up.view(rows, -1, BLOCK)), 2).reshape(rows, -1)


def _swiglu_plain(gate, up):
    return gate / (1.0 + torch.exp(-gate)) * up


def _fp4_values(code):
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    v = table[(code & 7).long()]
    return torch.where(code >= 8, -v, v)


def _weight_plain(q, s, H):
    """One expert's weight [Hp, H] in float32 from its packed values and scales."""
    NT, KT = q.shape[:2]
    code = torch.stack((q & 15, q >> 4), -1).view(NT, KT, 4, 16, 32)
    v = _fp4_values(code).permute(0, 3, 1, 2, 4).reshape(NT * 16, KT * 4, 32)
    e = s.view(NT, -1, 4, 16, 4).permute(0, 3, 1, 4, 2).reshape(NT * 16, -1)[:, :KT * 4].int() - 127
    return (v * _pow2(e).unsqueeze(-1)).reshape(NT * 16, -1)[:, :H]


# ------------------------------------------------------------------ results in 64 bits
def exact(case, seed):
    c, op, N, K = case, case["op"], case["N"], case["K"]
    st = _inputs(case, seed)
    if op == "route":
        return _route_exact(st, c)
    if op == "route_grad":
        return _route_grad_exact(st, c)
    if op == "gate_grad":
        out = torch.empty((N, K), dtype=torch.float64, device="cuda")
        where = st["slot_map"].long().view(N, K)
        for k in range(K):
            for lo in range(0, N, 4096):
                rows = st["out"][where[lo:lo + 4096, k]].double()
                out[lo:lo + 4096, k] = (rows * st["dy"][lo:lo + 4096].double()).sum(-1)
        return out
    if op == "checkpoint_x":
        held = torch.empty(st["x"].shape, dtype=torch.float64, device="cuda")
        for lo in range(0, N, 4096):
            held[lo:lo + 4096] = _blockwise_exact(st["x"][lo:lo + 4096].double(), 448.0, 3, -6)
        return held[torch.div(st["src_index"].long(), K, rounding_mode="floor")]
    if op == "checkpoint_h":
        Hp, NK = c["Hp"], N * K
        act, act_b = (torch.empty((NK, Hp), dtype=torch.float64, device="cuda") for _ in range(2))
        dh = torch.empty((NK, 2 * Hp), dtype=torch.float64, device="cuda")
        dg = torch.empty(NK, dtype=torch.float64, device="cuda")
        col = torch.arange(Hp, device="cuda")
        gc = 2 * BLOCK * (col // BLOCK) + col % BLOCK
        uc = gc + BLOCK
        src = st["src_index"].long()
        flat = st["gates"].double().reshape(-1)
        for lo in range(0, NK, 16384):
            h, da = st["h"][lo:lo + 16384].double(), st["da"][lo:lo + 16384].double()
            at = src[lo:lo + 16384]
            act[lo:lo + 16384] = h[:, gc] * torch.sigmoid(h[:, gc]) * h[:, uc]
            hq = _blockwise_exact(h, 448.0, 3, -6)
            gate, up, w = hq[:, gc], hq[:, uc], flat[at].unsqueeze(1)
            sg = torch.sigmoid(gate)
            a = gate * sg * up
            act_b[lo:lo + 16384] = w * a
            dg[at] = (a * da).sum(1)
            dh[lo:lo + 16384, gc] = w * da * up * (sg + gate * sg * torch.sigmoid(-gate))
            dh[lo:lo + 16384, uc] = w * da * gate * sg
        return act, act_b, dh, dg.view(N, K)
    x = _blockwise_exact(st["x"].double(), 6.0, 1, 0)
    out = torch.empty((N * K, c["Hp"]), dtype=torch.float64, device="cuda")
    token = torch.div(st["src_index"].long(), K, rounding_mode="floor")
    for i in range(c["E"]):
        lo, hi = st["bounds"][i], st["bounds"][i + 1]
        if hi > lo:
            w = _weight_exact(st["wq"][i], st["ws"][i], c["H"])
            out[lo:hi] = torch.matmul(x[token[lo:hi]], w)
    return out


def _inputs(case, seed):
    """The inputs alone, whichever side is measured."""
    global own
    kept, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = kept


def _blockwise_exact(v, top, mantissa, emin):
    """v rounded to nearest even in a small float type (largest value ``top``, ``mantissa``
    stored bits, smallest normal exponent ``emin``) with a power-of-two scale per 32 columns."""
    rows, W = v.shape
    out = torch.empty_like(v)
    for lo in range(0, W, BLOCK):
        b = v[:, lo:lo + BLOCK]
        amax = b.abs().max(1, keepdim=True).values
        scale = torch.exp2(torch.ceil(torch.log2(amax.clamp_min(1e-300) / top)).clamp(-127, 127))
        # the logarithm rounds: settle borders by the comparison itself
        scale = torch.where(amax > top * scale, 2 * scale, scale)
        scale = torch.where((amax <= top * scale / 2) & (scale > 2.0 ** -127), scale / 2, scale)
        r = b / scale
        expo = torch.floor(torch.log2(r.abs().clamp_min(1e-300))).clamp_min(emin)
        step = torch.exp2(expo - mantissa)
        out[:, lo:lo + BLOCK] = torch.round(r / step) * step * scale
    return out


def _weight_exact(q, s, H):
    """[H, Hp] in float64; the value of (k, n) is nibble k % 2 of byte (k % 32) / 2 of lane
    16 * (k / 32 % 4) + n % 16 of tile (n / 16, k / 128)."""
    n = torch.arange(q.shape[0] * 16, device="cuda").unsqueeze(0)
    k = torch.arange(H, device="cuda").unsqueeze(1)
    lane = 16 * ((k // 32) % 4) + n % 16
    byte = q[n // 16, k // 128, lane, (k % 32) // 2].int()
    code = torch.where(k % 2 == 0, byte & 15, byte >> 4)
    mag, expo = (code & 1).double(), ((code >> 1) & 3).double()
    val = torch.where(expo == 0, mag / 2, (1 + mag / 2) * torch.exp2(expo - 1))
    e = s[n // 16, k // 512, lane, (k // 128) % 4].double() - 127
    return torch.where(code >= 8, -val, val) * torch.exp2(e)


def _route_exact(st, c):
    l = st["logits"].double()
    N, E = l.shape
    bias = torch.zeros(E, dtype=torch.float64, device="cuda") if st["bias"] is None else st["bias"].double()
    live = torch.isfinite(bias).unsqueeze(0) & (l > -INF)
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        s = torch.softmax(torch.where(live, l, -INF), 1)
    rank = l if st["bias"] is None else s + bias
    rank = torch.where(live, rank, -INF)
    num = torch.arange(E, device="cuda")

    def first_best(v, taken):
        v = torch.where(taken, float("nan"), v)
        best = torch.nan_to_num(v, nan=-INF, neginf=-INF, posinf=INF).amax(1, keepdim=True)
        return torch.where((v == best), torch.arange(v.shape[1], device="cuda"), v.shape[1]).amin(1)

    if c["groups"] > 1:
        G, per = c["groups"], E // c["groups"]
        total = torch.empty((N, G), dtype=torch.float64, device="cuda")
        for i in range(G):
            part = (rank if c["group_top"] == 1 else torch.where(live, s + bias, -INF))[:, i * per:(i + 1) * per]
            total[:, i] = part.amax(1)
            if c["group_top"] == 2:
                at = first_best(part, torch.zeros_like(part, dtype=torch.bool))
                rest = torch.where(torch.arange(per, device="cuda") == at.unsqueeze(1), -INF, part).amax(1)
                total[:, i] += torch.where(rest == -INF, 0.0, rest)
        taken = torch.zeros((N, G), dtype=torch.bool, device="cuda")
        for _ in range(c["top_groups"]):
            at = first_best(total, taken)
            taken |= torch.arange(G, device="cuda") == at.unsqueeze(1)
        rank = torch.where(taken[:, num // per], rank, -INF)
    ids = torch.empty((N, c["K"]), dtype=torch.int64, device="cuda")
    taken = torch.zeros((N, E), dtype=torch.bool, device="cuda")
    for k in range(c["K"]):
        ids[:, k] = first_best(rank, taken)
        taken |= num == ids[:, k:k + 1]
    good = torch.gather(rank, 1, ids) > -INF
    gates = torch.where(good, torch.gather(s, 1, ids), 0.0)
    if c["renorm"]:
        gates = gates / gates.sum(1, keepdim=True)
    return ids.int(), gates * c["scale"]


def _route_grad_exact(st, c):
    l = st["logits"].double()
    if st["bias"] is not None:
        l = torch.where(st["bias"].unsqueeze(0) == -INF, -INF, l)
    gates, dg = st["gates"].double(), st["dgates"].double()
    pick = torch.zeros(l.shape, dtype=torch.float64, device="cuda")
    pick.scatter_(1, st["ids"].long(), gates)                            # gates at their experts
    grad = torch.zeros_like(pick).scatter_(1, st["ids"].long(), dg)
    mean = (pick * grad).sum(1, keepdim=True)
    if c["score"] == "sigmoid":
        inner = grad - mean / c["scale"] if c["renorm"] else grad
        return pick * inner * torch.sigmoid(-l).nan_to_num()
    if c["renorm"]:
        return pick * (grad - mean / c["scale"])
    return pick * grad - torch.softmax(l, 1) * mean
