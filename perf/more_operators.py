"""Cases of experts in 8-bit integers: the grouped product, its gate/up form with SwiGLU, the
dense product of a shared expert, and the gradient through frozen experts. Inputs, one pass of
each through the library's entry points (``own``) or in its plain form (elementary torch
operations), the work a pass cannot do without, and the results in 64 bits.

A pass begins at the activations (or the upstream gradient) in the layer's type: rounding them
to 8 bits is a part of it. Weights are held in 8 bits and are inputs.

Every layer here is one rank (R = 1), whose plan is the stable order of the slots by expert:
the operators read a plan only through src_index and cu_seqlens, so one rank stands for any
number of them.
"""
import math

import torch

own = False

BLOCK = 32                     # gate and up columns alternate in blocks of this many
LEAST = 2.0 ** -126            # the smallest scale


# ------------------------------------------------------------------ cases
def _case(op, name, N, K, E, H, Hp, dtype, saved=False, gather=True):
    """N tokens, K of E experts each (a dense product: 1 of 1), weights [H, Hp] (gate/up: [H, 2Hp])."""
    return dict(op=op, name=name, N=N, K=K, E=E, H=H, Hp=Hp, dtype=dtype, saved=saved, gather=gather)


def listed():
    return [
        # one token of a serving step over 256 experts
        _case("grouped", "grouped_one_token", 1, 8, 256, 4096, 1536, "bf16"),
        # a serving step of 16 sequences, one token each
        _case("grouped", "grouped_decode", 16, 8, 256, 4096, 1536, "bf16"),
        # a tiny float32 layer with sizes that fit no tile
        _case("grouped", "grouped_odd", 251, 3, 16, 76, 100, "fp32"),
        # a prompt batch
        _case("grouped", "grouped_prompt", 65536, 8, 256, 4096, 1536, "bf16"),
        # gate/up projection of a serving step of 64 sequences
        _case("swiglu", "swiglu_decode", 64, 8, 128, 4096, 1408, "bf16"),
        # the same in the forward pass of a training step, which keeps the pre-activation
        _case("swiglu", "swiglu_train", 32768, 8, 128, 4096, 1408, "bf16", saved=True),
        # down projection of a shared expert for one token, added to the routed experts' output
        _case("dense", "dense_one_token", 1, 1, 1, 2048, 7168, "bf16"),
        # the same for a prompt of 16384 tokens
        _case("dense", "dense_prompt", 16384, 1, 1, 2048, 7168, "bf16"),
        # gate/up projection of the shared expert, a serving step of 16 sequences
        _case("dense_swiglu", "shared_decode", 16, 1, 1, 7168, 2048, "bf16"),
        # the same for a prompt of 16384 tokens
        _case("dense_swiglu", "shared_prompt", 16384, 1, 1, 7168, 2048, "bf16"),
        # gradient through a small float32 layer's down projection
        _case("grad", "grad_small", 256, 2, 16, 64, 132, "fp32"),
        # gradient through the down projection of a training layer, from the tokens' gradient
        _case("grad", "grad_train", 32768, 8, 128, 1408, 4096, "bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "swiglu", "dense", "dense_swiglu", "grad"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    vec = 4 if dtype == "fp32" else 8
    dense = op.startswith("dense")
    H = vec * _log(rng, 4, 7168 // vec)
    if op in ("swiglu", "dense_swiglu"):
        Hp = BLOCK * _log(rng, 1, 2048 // BLOCK)
    else:
        Hp = vec * _log(rng, 4, 7168 // vec)
    E = 1 if dense else rng.choice([8, 16, 60, 128, 256])
    K = 1 if dense else rng.randint(1, 8)
    wide = 2 * Hp if op in ("swiglu", "dense_swiglu") else Hp
    # no more work than the largest listed case, in operations and in slots times width
    most = min(524288 * 4096 * 1536 // (K * H * wide), 262144 * 4096 // (K * max(H, wide)),
               16384 if dense else 65536)
    N = _log(rng, 1, max(1, most))
    return {k: v for k, v in _case(op, None, N, K, E, H, Hp, dtype, saved=rng.random() < 0.5,
                                   gather=rng.random() < 0.5).items() if k != "name"}


def _wide(case):
    """Columns of the weight: gate and up, or the output's."""
    return 2 * case["Hp"] if case["op"] in ("swiglu", "dense_swiglu") else case["Hp"]


def work(case):
    c, op, N, K, E, H = case, case["op"], case["N"], case["K"], case["E"], case["H"]
    W, NK = _wide(case), N * K
    eb = 4 if c["dtype"] == "fp32" else 2
    touched = E * (1.0 - (1.0 - min(1.0, K / E)) ** N)        # experts expected to have rows
    weights = int(touched * (H * W + 4 * W))
    index = 0 if op.startswith("dense") else 4 * NK + 4 * E
    flops = 2 * NK * H * W
    if op == "grouped":
        return {"bytes": N * H * eb + weights + index + NK * W * 4, "flops": flops}
    if op == "dense":
        return {"bytes": N * H * eb + weights + 2 * N * W * 4, "flops": flops}
    if op == "grad":
        rows = N if c["gather"] else NK
        return {"bytes": rows * W * eb + weights + index + 4 * NK * c["gather"] + NK * H * 4, "flops": flops}
    out = NK * c["Hp"] * eb + (NK * W * eb if c["saved"] else 0)
    return {"bytes": N * H * eb + weights + index + out, "flops": flops}


# ------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


def _normal(g, shape, std=1.0):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=g)


def _plan(g, N, E, K, rows):
    """A skewed router's choice of K of E experts for every token, and its plan on one rank whose
    weight has `rows` rows, the last of them empty."""
    score = _normal(g, (N, E)) + 0.3 * _normal(g, (E,))
    topk = torch.sort(score, dim=1, descending=True).indices[:, :K].contiguous()
    order = torch.sort(topk.reshape(-1), stable=True).indices            # buffer position -> slot
    cu = torch.zeros(rows + 1, dtype=torch.int64, device="cuda")
    cu[1:] = torch.cumsum(torch.bincount(topk.reshape(-1), minlength=rows), 0)
    return order.int(), cu.int(), torch.softmax(torch.gather(score, 1, topk), 1)


def _rows8(v):
    """Whole values (as float64) and scales (float32) of rows v: the division in 64 bits, so that
    values next to a border between two whole numbers fall on the right side."""
    scale = (v.abs().amax(1).double() / 127.0).float().clamp_min(LEAST)
    return torch.round(v.double() / scale.double().unsqueeze(1)), scale


def _pack(q):
    """One weight [H, W] of whole values in the order the product reads it: blocks of 16 columns
    by 64 k, H padded to whole 128s with zeros, 16 k of a column together."""
    H, W = q.shape
    KB, NB = 2 * -(-H // 128), -(-W // 16)
    pad = torch.zeros((KB * 64, NB * 16), dtype=torch.int8, device=q.device)
    pad[:H, :W] = q
    return pad.view(KB, 4, 16, NB, 16).permute(3, 0, 1, 4, 2).reshape(NB, KB, 64, 16)


def prepare(case, seed):
    c, op, N, K, E, H = case, case["op"], case["N"], case["K"], case["E"], case["H"]
    W, NK, dt = _wide(case), N * K, _dtype(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    st = {"case": c}
    grad = op == "grad"
    KB, NB = 2 * -(-H // 128), -(-W // 16)
    # the weights: [H, W] packed, for the gradient [W, H] packed; scales of the W columns
    # (a training layer has as many rows again for replicas; one rank leaves them empty)
    rows = 2 * E if grad else E
    shape = (rows, -(-H // 16), 2 * -(-W // 128), 64, 16) if grad else (rows, NB, KB, 64, 16)
    st["wq"] = torch.zeros(shape, dtype=torch.int8, device="cuda")
    st["ws"] = torch.zeros((rows, NB * 16), dtype=torch.float32, device="cuda")
    for e in range(E):
        w = _normal(g, (W, H), H ** -0.5) * torch.exp(0.3 * _normal(g, (W, 1)))
        q, st["ws"][e, :W] = _rows8(w)
        st["wq"][e] = _pack(q if grad else q.t())
    if not op.startswith("dense"):
        st["src_index"], st["cu"], gates = _plan(g, N, E, K, rows)
        st["gates"] = gates.contiguous()
        st["bounds"] = st["cu"].tolist()
    # activations: channels of different sizes, as a model's are
    rows, width = (N if c["gather"] else NK, W) if grad else (N, H)
    st["x"] = (_normal(g, (rows, width)) * torch.exp(0.5 * _normal(g, (width,)))).to(dt)
    if op == "dense":
        st["add"] = _normal(g, (N, W))
    if not own:
        return st
    # the shapes, the workspace and the buffers that a layer keeps
    from redundant_expert_balancing_amd import _lib as L, int8
    st["L"] = L
    f32 = dict(dtype=torch.float32, device="cuda")
    mode, B = (L.TRAIN, E) if grad else (L.INFER, 0)
    ty = L.FP32 if c["dtype"] == "fp32" else L.BF16
    sh = st["shape"] = L.Shape(1, N, E, K, B, H, c["Hp"], mode, ty)
    st["back"] = L.Shape(1, N, E, K, B, W, H, mode, ty)
    st["xq"], st["xs"] = int8.buffers(NK if grad else N, W if grad else H)
    if not op.startswith("dense"):
        up = L.Shape(1, N, E, K, B, H, W, mode, ty)
        st["work"] = torch.empty((L.moonep_workspace_bytes(up) // 4,), dtype=torch.int32, device="cuda")
        L.moonep_workspace_init(up, st["work"])
    if op in ("grouped", "dense"):
        st["c"] = torch.empty((NK, W), **f32)
    elif grad:
        st["c"] = torch.empty((NK, H), **f32)
    else:
        st["act"] = torch.empty((NK, c["Hp"]), dtype=dt, device="cuda")
        st["h"] = torch.empty((NK, W), dtype=dt, device="cuda") if c["saved"] else None
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    c, L, sh = st["case"], st["L"], st["shape"]
    op, N = c["op"], c["N"]
    xq, xs = st["xq"], st["xs"]
    if op == "grad":
        L.moonep_int_quantize_grad(sh, st["x"], st["src_index"] if c["gather"] else None,
                                  st["gates"] if c["gather"] else None, st["ws"], st["cu"], xq, xs)
        L.moonep_int_grouped_gemm(st["back"], xq, xs, None, st["wq"], None, st["cu"], st["c"],
                                 st["work"])
        return st["c"]
    L.moonep_int_quantize(sh, N, c["H"], st["x"], xq, xs)
    if op == "grouped":
        L.moonep_int_grouped_gemm(sh, xq, xs, st["src_index"], st["wq"], st["ws"], st["cu"], st["c"],
                                 st["work"])
        return st["c"]
    if op == "dense":
        L.moonep_int_gemm(sh, N, xq, xs, st["wq"], st["ws"], st["add"], st["c"])
        return st["c"]
    if op == "swiglu":
        L.moonep_int_grouped_gemm_swiglu(sh, xq, xs, st["src_index"], st["wq"], st["ws"], st["cu"],
                                        st["act"], st["h"], st["work"])
    else:
        L.moonep_int_gemm_swiglu(sh, N, xq, xs, st["wq"], st["ws"], st["act"], st["h"])
    return (st["act"], st["h"]) if c["saved"] else st["act"]


def _weight(q, H, W):
    """One packed weight as float32 [H, W]."""
    NB, KB = q.shape[:2]
    return q.view(NB, KB, 4, 16, 16).permute(1, 2, 4, 0, 3).reshape(KB * 64, NB * 16)[:H, :W].float()


def _run_plain(st):
    c = st["case"]
    op, K, H, W, dt = c["op"], c["K"], c["H"], _wide(st["case"]), _dtype(st["case"])
    x = st["x"].float()
    if op.startswith("dense"):
        q, s = _rows8(x)
        h = (q.float() @ _weight(st["wq"][0], H, W)) * s.unsqueeze(1) * st["ws"][0, :W]
        return h + st["add"] if op == "dense" else _swiglu_plain(h, dt, c["saved"])
    slot = st["src_index"].long()
    if op == "grad":
        out = torch.empty((slot.numel(), H), dtype=torch.float32, device="cuda")
        gate = st["gates"].reshape(-1)
        for e in range(c["E"]):
            lo, hi = st["bounds"][e], st["bounds"][e + 1]
            if hi > lo:
                rows = x[slot[lo:hi] // K] if c["gather"] else x[lo:hi]
                q, s = _rows8(rows * st["ws"][e, :W])
                if c["gather"]:
                    s = s * gate[slot[lo:hi]]
                out[lo:hi] = (q.float() @ _weight(st["wq"][e], W, H)) * s.unsqueeze(1)
        return out
    q, s = _rows8(x)
    q = q.float()
    h = torch.empty((slot.numel(), W), dtype=torch.float32, device="cuda")
    for e in range(c["E"]):
        lo, hi = st["bounds"][e], st["bounds"][e + 1]
        if hi > lo:
            at = slot[lo:hi] // K
            h[lo:hi] = (q[at] @ _weight(st["wq"][e], H, W)) * s[at].unsqueeze(1) * st["ws"][e, :W]
    return h if op == "grouped" else _swiglu_plain(h, dt, c["saved"])


def _swiglu_plain(h, dt, saved):
    v = h.view(h.shape[0], -1, 2, BLOCK)
    gate, up = v[:, :, 0], v[:, :, 1]
    act = (gate / (1.0 + torch.exp(-gate)) * up).reshape(h.shape[0], -1).to(dt)
    return (act, h.to(dt)) if saved else act


# ------------------------------------------------------------------ results in 64 bits
def exact(case, seed):
    c, op, K, H, W = case, case["op"], case["K"], case["H"], _wide(case)
    st = _inputs(case, seed)
    x, E = st["x"].double(), c["E"]
    NK = c["N"] * K
    out = torch.empty((NK, H if op == "grad" else W), dtype=torch.float64, device="cuda")
    token = (torch.arange(NK, device="cuda") if op.startswith("dense")
             else torch.div(st["src_index"].long(), K, rounding_mode="floor"))
    ends = [0, NK] if op.startswith("dense") else st["bounds"]
    for e in range(E):
        for lo in range(ends[e], ends[e + 1], 65536):
            at = slice(lo, min(lo + 65536, ends[e + 1]))
            if op == "grad":
                rows = x[token[at]] if c["gather"] else x[at]
                # the scaled gradient is held in 32 bits before it is rounded to 8
                rows = (rows * st["ws"][e, :W].double()).float().double()
                v = torch.matmul(_held(rows), _weight_exact(st["wq"][e], W, H))
                if c["gather"]:
                    v *= st["gates"].double().reshape(-1)[st["src_index"].long()[at]].unsqueeze(1)
                out[at] = v
            else:
                w = _weight_exact(st["wq"][e], H, W) * st["ws"][e, :W].double()
                out[at] = torch.matmul(_held(x[token[at]]), w)
    if op == "grouped":
        return out
    if op == "dense":
        return out + st["add"].double()
    if op == "grad":
        return out
    col = torch.arange(c["Hp"], device="cuda")
    at = 2 * BLOCK * torch.div(col, BLOCK, rounding_mode="floor") + col % BLOCK
    act = torch.empty((NK, c["Hp"]), dtype=torch.float64, device="cuda")
    for lo in range(0, NK, 16384):
        gate = out[lo:lo + 16384, at]
        act[lo:lo + 16384] = gate * torch.sigmoid(gate) * out[lo:lo + 16384, at + BLOCK]
    return (act, out) if c["saved"] else act


def _inputs(case, seed):
    """The inputs alone, whichever side is measured."""
    global own
    kept, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = kept


def _held(v):
    """The values that rows v stand for once they are held in 8 bits with a 32-bit scale."""
    step = (v.abs().max(1, keepdim=True).values / 127).to(torch.float32).double()
    step = torch.where(step < LEAST, LEAST, step)
    whole = torch.floor(v / step)
    rest = v / step - whole
    up = (rest > 0.5) | ((rest == 0.5) & (whole % 2 != 0))
    return (whole + up) * step


def _weight_exact(q, H, W):
    """[H, W] in float64; (k, n) is byte k % 16 of lane 16 * (k / 16 % 4) + n % 16 of block
    (n / 16, k / 64)."""
    n = torch.arange(W, device="cuda").unsqueeze(0)
    k = torch.arange(H, device="cuda").unsqueeze(1)
    return q[n // 16, k // 64, 16 * ((k // 16) % 4) + n % 16, k % 16].double()
