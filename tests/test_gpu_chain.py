"""Router, experts and gradients run together, as a training step and a serving step use them."""
import numpy as np
import pytest
import torch

from oracle import ffn as FF
from oracle import formats as F
from oracle import route as RT
from redundant_expert_balancing_amd.ffn import MoEFFN
from redundant_expert_balancing_amd.mx import MXFFN
from redundant_expert_balancing_amd.router import MoERouter
from redundant_expert_balancing_amd.synth import make_dense

from gpu_helpers import say, small_cfg

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
KW = dict(score="sigmoid", groups=4, top_groups=2, group_top=2, scale=1.5)


def test_training_step_on_checkpoints():
    """logits -> route -> FFN on checkpoints -> dgates -> dlogits, with padding tokens (every
    logit -inf) behind the batch; two layers that share their slot buffers; eager and replayed."""
    cfg = small_cfg(name="chain", R=4, S=30, E=16, K=3, H=64, Hp=128, dtype="fp32")
    say("chain training")
    N, E, K, Hp = cfg.N, cfg.E, cfg.K, cfg.Hp
    rng = np.random.default_rng(2)
    logits = torch.from_numpy(rng.standard_normal((N, E)).astype(np.float32)).cuda().bfloat16()
    pad = 7
    logits[N - pad:] = float("-inf")
    bias = torch.from_numpy(0.1 * rng.standard_normal(E).astype(np.float32)).cuda()
    d = [make_dense(cfg, "cuda", s, which=("x", "W1", "W2", "dyH"), w_rows=cfg.E + cfg.R * cfg.B)
         for s in (0, 1)]
    rt = [MoERouter(cfg, dtype="bf16", backward=True, **KW) for _ in d]
    l0 = MoEFFN(cfg, backward=True, w1_all=d[0]["W1"], w2_all=d[0]["W2"], checkpoint=True)
    l1 = MoEFFN(cfg, backward=True, w1_all=d[1]["W1"], w2_all=d[1]["W2"], checkpoint=True, scratch=l0)
    layers = [l0, l1]

    def run():
        for r, l, t in zip(rt, layers, d):
            l.forward(*_pair(r.forward(logits, bias), t["x"]))
        for r, l, t in list(zip(rt, layers, d))[::-1]:
            l.backward(t["dyH"], r.gates)
            r.backward(logits, l.gate_grad(t["dyH"]), bias)

    def _pair(choice, x):
        return choice[0], x, choice[1]

    def outputs():
        return [t for r, l in zip(rt, layers)
                for t in (r.topk_idx, r.gates, r.dlogits, l.y, l.dx, l.dgates)]

    run()
    torch.cuda.synchronize()
    lh, bh = logits.double().cpu().numpy(), bias.double().cpu().numpy()
    want_ids, want_g = RT.route(lh, bh, K, **KW)
    gc, uc = FF.gate_up_columns(Hp)
    for r, l, t in zip(rt, layers, d):
        assert np.array_equal(r.topk_idx.cpu().numpy(), want_ids)
        g = r.gates.double().cpu().numpy()
        assert (g[N - pad:] == 0).all() and not l.y[N - pad:].any() and not l.dx[N - pad:].any()
        sm = l.slot_map.cpu().numpy()
        hv = F.checkpoint_values(l.hq.cpu().numpy(), l.hscales.cpu().numpy()[:, :2 * Hp // 32])[sm]
        dy, W2 = t["dyH"].double().cpu().numpy(), t["W2"].double().cpu().numpy()
        dg = np.zeros((N, K))
        for n in range(N):
            for k in range(K):
                gv, uv = hv[n * K + k, gc], hv[n * K + k, uc]
                dg[n, k] = (gv * FF.sigmoid(gv) * uv) @ (dy[n] @ W2[want_ids[n, k]].T)
        got = l.dgates.double().cpu().numpy()
        assert np.abs(got - dg).max() <= 1e-5 * np.sqrt((dg ** 2).mean())   # the fp32 layer's bar
        ref = RT.route_backward(lh, bh, want_ids, g, got, score="sigmoid", scale=KW["scale"])
        terms = (g * np.abs(got)).sum(1, keepdims=True) * (1 + 1 / KW["scale"]) + 1e-30
        # as in the router's own test: float32 terms, then one rounding to bfloat16
        bound = (2 * 200 + E + 2 * K + 16) * U * terms + np.abs(ref) * 2.0 ** -8 * (1 + 2.0 ** -7)
        dl = r.dlogits.double().cpu().numpy()
        assert (np.abs(dl - ref) <= bound).all() and not dl[N - pad:].any()
    want = [t.clone() for t in outputs()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for rep in range(3):
        for t in outputs():
            t.fill_(0)
        _ = torch.randn(4096, device="cuda").sum().item()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outputs())), rep


@pytest.mark.parametrize("S", [1, 3])
def test_serving_step_on_4_bit_experts(S):
    """A step of S tokens: logits -> route -> 4-bit FFN, replayed for new tokens, against the
    formula on the values the 4-bit operands stand for."""
    cfg = small_cfg(name="chain_mx", R=1, S=S, E=16, K=4, B=0, H=192, Hp=64, mode="infer")
    say("chain serving", S)
    d = make_dense(cfg, "cuda", 0, which=("x", "W1", "W2"))
    rt, l = MoERouter(cfg, **KW), MXFFN(cfg)
    l.quantise_weights(d["W1"], d["W2"])
    logits, x = torch.zeros((cfg.N, cfg.E), device="cuda"), torch.zeros_like(d["x"])

    def step():
        ids, gates = rt.forward(logits)
        l.forward(ids, x, gates)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    rng = np.random.default_rng(S)
    w1 = [F.mx_values(*F.mx(w.T)).T for w in d["W1"].double().cpu().numpy()]
    w2 = [F.mx_values(*F.mx(w.T)).T for w in d["W2"].double().cpu().numpy()]
    for rep in range(4):
        logits.copy_(torch.from_numpy(rng.standard_normal((cfg.N, cfg.E)).astype(np.float32)))
        x.copy_(torch.from_numpy(rng.standard_normal((cfg.N, cfg.H)).astype(np.float32)))
        l.y.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        ids, gates = RT.route(logits.double().cpu().numpy(), None, cfg.K, **KW)
        assert np.array_equal(rt.topk_idx.cpu().numpy(), ids)
        xv = F.mx_values(*F.mx(x.double().cpu().numpy()))
        act = l.act.double().cpu().numpy()
        av, sm = F.mx_values(*F.mx(act)), l.slot_map.cpu().numpy()
        ref = np.zeros((cfg.N, cfg.H))
        for t in range(cfg.N):
            for k in range(cfg.K):
                e, pos = ids[t, k], sm[t * cfg.K + k]
                a = FF.swiglu((xv[t] @ w1[e])[None], "bf16")[0]
                # one bfloat16 step where the float32 and float64 sums straddle a border
                assert (np.abs(act[pos] - a) <= 2.0 ** -7 * np.abs(a) + 1e-5).all()
                ref[t] += gates[t, k] * (av[pos] @ w2[e])
        err = np.abs(l.y.double().cpu().numpy() - ref).max() / np.sqrt((ref ** 2).mean())
        assert err <= 1e-5, (rep, err)
