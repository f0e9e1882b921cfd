"""4-bit experts on the GPU: stored bytes equal the oracle's, the grouped GEMM within the
float32 accumulation of the exact products, the layers on them."""
import numpy as np
import pytest
import torch

from oracle import ffn as FF
from oracle import formats as F
from oracle import plan as P
from redundant_expert_balancing_amd import _lib as L
from redundant_expert_balancing_amd import mx
from redundant_expert_balancing_amd.mx import MXFFN, MXProjection
from redundant_expert_balancing_amd.synth import make_dense, make_routing

from gpu_helpers import say, small_cfg

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _dt(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _shape(H, Hp, dtype="bf16", S=8, E=4, K=1):
    return L.Shape(1, S, E, K, 0, H, Hp, L.INFER, L.BF16 if dtype == "bf16" else L.FP32)


def _wide(rng, shape):
    x = rng.standard_normal(shape) * 2.0 ** rng.integers(-3, 4, shape)
    x[rng.random(shape) < 0.05] = 0.0
    x.reshape(-1)[:8] = [0.0, 6.0, -6.0, 5.0, 2.5, -0.25, 0.75, 3.5]
    return x.astype(np.float32)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,width", [(1, 32), (3, 64), (7, 96), (33, 128), (5, 544), (17, 1408), (2, 4096)])
def test_quantise_rows(dtype, rows, width):
    say("mx rows", dtype, rows, width)
    rng = np.random.default_rng(width)
    x = torch.from_numpy(_wide(rng, (rows, width))).cuda().to(_dt(dtype))
    if rows > 2:
        x[2, width - 1] = float("nan")
        x[1] = 0
    q, s = mx.buffers(rows, width)
    q.fill_(0xAA), s.fill_(0xAA)
    L.moonep_mx_quantize(_shape(64, 64, dtype), rows, width, x, q, s)
    torch.cuda.synchronize()
    codes, sb = F.mx(x.double().cpu().numpy())
    want_q, want_s = F.mx_pack_rows(codes, sb)
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(q.cpu().numpy(), want_q)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,Hp", [(32, 16), (64, 64), (160, 48), (1408, 64), (512, 192)])
def test_quantise_weights(dtype, H, Hp):
    say("mx weights", dtype, H, Hp)
    E = 3
    rng = np.random.default_rng(H)
    w = torch.from_numpy(_wide(rng, (E, H, Hp))).cuda().to(_dt(dtype))
    wq, ws = mx.weight_buffers(E, H, Hp)
    wq.fill_(0xAA), ws.fill_(0xAA)
    L.moonep_mx_quantize_weight(_shape(H, Hp, dtype, E=E), w, wq, ws)
    torch.cuda.synchronize()
    for e in range(E):
        codes, sb = F.mx(w[e].double().cpu().numpy().T)
        q, s = F.mx_pack_weight(codes, sb)
        assert np.array_equal(ws[e].cpu().numpy(), s)
        assert np.array_equal(wq[e].cpu().numpy(), q)


def _layer(cfg, alpha, seed=0):
    r = make_routing(cfg, 3.0, seed=seed, alpha=alpha)
    d = make_dense(cfg, "cuda", seed, which=("x", "W"))
    l = MXProjection(cfg)
    l.wq.fill_(0xFF), l.wscales.fill_(0xFF)       # unused slots stay NaN
    l.quantise_weights(d["W"])
    topk, gates = torch.from_numpy(r.topk_idx).cuda(), torch.from_numpy(r.gates).cuda()
    l.out.fill_(float("nan")), l.y.fill_(float("nan"))
    return r, d, l, topk, gates


def _check_layer(cfg, alpha, experts=None, seed=0):
    say("mx layer", cfg)
    r, d, l, topk, gates = _layer(cfg, alpha, seed)
    y = l.forward(topk, d["x"], gates)
    torch.cuda.synchronize()
    pl = P.plan(r.topk_idx, cfg.R, cfg.S, cfg.E, cfg.K, cfg.B, cfg.mode)
    assert np.array_equal(l.slot_map.cpu().numpy()[:cfg.N * cfg.K], pl.slot_map)
    xv = torch.from_numpy(F.mx_values(*F.mx(d["x"].double().cpu().numpy())))
    out = l.out.double().cpu()[torch.from_numpy(pl.slot_map).long()]
    for e in range(cfg.E) if experts is None else experts:
        tok, kk = np.nonzero(r.topk_idx == e)
        if not len(tok):
            continue
        wv = torch.from_numpy(F.mx_values(*F.mx(d["W"][e].double().cpu().numpy().T)))
        want = xv[tok] @ wv.T
        mag = xv[tok].abs() @ wv.T.abs()
        got = out[tok * cfg.K + kk]
        # products of two e2m1 values and power-of-two scales are exact; a float32 sum of H
        # of them in any order is off by at most H roundings of the magnitude sum
        assert bool(((got - want).abs() <= cfg.H * U * mag).all()), e
    assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(l.out).all())
    g = torch.from_numpy(r.gates).double()
    yref = (out.view(cfg.N, cfg.K, -1) * g[..., None]).sum(1)
    mag = (out.view(cfg.N, cfg.K, -1) * g[..., None]).abs().sum(1)
    assert bool(((y.double().cpu() - yref).abs() <= (cfg.K + 1) * U * mag + 1e-30).all())


@pytest.mark.parametrize("kw", [
    dict(R=1, S=1, E=4, K=1, B=0, H=64, Hp=64),                  # one token, one expert
    dict(R=1, S=1, E=16, K=8, B=0, H=512, Hp=128),               # one token
    dict(R=2, S=5, E=16, K=3, B=2, H=192, Hp=320),               # ragged k chunk, 5 column tiles
    dict(R=4, S=37, E=16, K=2, B=4, H=128, Hp=64),
    dict(R=4, S=64, E=8, K=2, B=1, H=1408, Hp=192),              # overflow rows
    dict(R=1, S=700, E=4, K=2, B=0, H=576, Hp=512),              # segments beyond a tile
    dict(R=2, S=512, E=8, K=4, B=4, H=320, Hp=576),
])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_layer_against_the_oracle(kw, dtype):
    _check_layer(small_cfg(name="mx", dtype=dtype, mode="infer", **kw), 2.0)


def test_training_plan_and_every_slot():
    _check_layer(small_cfg(name="mx_train", R=4, S=96, E=16, K=4, H=256, Hp=128), 2.5)


def test_long_segments_and_wide_layers():
    """More tiles than one round of the card, sampled experts."""
    _check_layer(small_cfg(name="mx_large", R=4, S=4096, E=32, K=4, B=8, H=1024, Hp=1088,
                           mode="infer"), 1.0, experts=[0, 3, 11, 31])


def test_rows_in_place_and_bad_positions():
    """src_index NULL reads one row per position; positions outside the plan give zeros."""
    say("mx in place")
    S, E, H, Hp = 70, 4, 192, 128
    sh = _shape(H, Hp, S=S, E=E)
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((S, H)).astype(np.float32)).cuda().bfloat16()
    w = torch.from_numpy(rng.standard_normal((E, H, Hp)).astype(np.float32)).cuda().bfloat16()
    xq, xs = mx.buffers(S, H)
    wq, wsc = mx.weight_buffers(E, H, Hp)
    L.moonep_mx_quantize(sh, S, H, x, xq, xs)
    L.moonep_mx_quantize_weight(sh, w, wq, wsc)
    cu = torch.tensor([[0, 3, 3, 68, 70]], dtype=torch.int32, device="cuda")
    ws = torch.empty(L.moonep_workspace_bytes(sh) // 4, dtype=torch.int32, device="cuda")
    L.moonep_workspace_init(sh, ws)
    a, b, c = (torch.full((S, Hp), float("nan"), device="cuda") for _ in range(3))
    ident = torch.arange(S, dtype=torch.int32, device="cuda")
    L.moonep_mx_grouped_gemm(sh, xq, xs, None, wq, wsc, cu, a, ws)
    L.moonep_mx_grouped_gemm(sh, xq, xs, ident, wq, wsc, cu, b, ws)
    broken = ident.clone()
    broken[5], broken[69] = -1, S
    L.moonep_mx_grouped_gemm(sh, xq, xs, broken, wq, wsc, cu, c, ws)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and bool(torch.isfinite(a).all())
    assert not c[5].any() and not c[69].any()
    keep = [i for i in range(S) if i not in (5, 69)]
    assert torch.equal(c[keep], a[keep])
    # rows behind the last segment are left as they were
    part = torch.tensor([[0, 2, 2, 40, 41]], dtype=torch.int32, device="cuda")
    c.fill_(7.0)
    L.moonep_mx_grouped_gemm(sh, xq, xs, ident, wq, wsc, part, c, ws)
    torch.cuda.synchronize()
    assert bool((c[41:] == 7.0).all()) and torch.equal(c[:2], a[:2])
    # an empty plan
    L.moonep_mx_grouped_gemm(sh, xq, xs, ident, wq, wsc, torch.zeros_like(part), c, ws)
    torch.cuda.synchronize()
    assert bool((c[41:] == 7.0).all())


def test_a_nan_token_stays_in_its_rows():
    say("mx nan token")
    cfg = small_cfg(name="mx_nan", R=2, S=40, E=8, K=2, B=2, H=256, Hp=128, mode="infer")
    r, d, l, topk, gates = _layer(cfg, 2.0)
    d["x"][7, 100] = float("nan")
    y = l.forward(topk, d["x"], gates)
    torch.cuda.synchronize()
    bad = torch.isnan(y).any(1).cpu()
    assert bool(torch.isnan(y[7]).all()) and int(bad.sum()) == 1


def test_ffn_against_the_oracle():
    cfg = small_cfg(name="mx_ffn", R=4, S=30, E=8, K=2, B=2, H=128, Hp=192, mode="infer")
    say("mx ffn")
    r = make_routing(cfg, 3.0, alpha=2.0)
    d = make_dense(cfg, "cuda", 0, which=("x", "W1", "W2"))
    l = MXFFN(cfg)
    l.quantise_weights(d["W1"], d["W2"])
    topk, gates = torch.from_numpy(r.topk_idx).cuda(), torch.from_numpy(r.gates).cuda()
    y = l.forward(topk, d["x"], gates)
    torch.cuda.synchronize()
    xv = F.mx_values(*F.mx(d["x"].double().cpu().numpy()))
    act = l.act.double().cpu().numpy()
    av = F.mx_values(*F.mx(act))
    sm = l.slot_map.cpu().numpy()
    ref = np.zeros((cfg.N, cfg.H))
    for e in range(cfg.E):
        w1 = F.mx_values(*F.mx(d["W1"][e].double().cpu().numpy().T)).T
        w2 = F.mx_values(*F.mx(d["W2"][e].double().cpu().numpy().T)).T
        for t, k in zip(*np.nonzero(r.topk_idx == e)):
            pos = sm[t * cfg.K + k]
            a = FF.swiglu((xv[t] @ w1)[None], "bf16")[0]
            # one bfloat16 step where the float32 and float64 sums straddle a border
            assert (np.abs(act[pos] - a) <= 2.0 ** -7 * np.abs(a) + 1e-5).all()
            ref[t] += r.gates[t, k] * (av[pos] @ w2)
    err = np.abs(y.double().cpu().numpy() - ref).max() / np.sqrt((ref ** 2).mean())
    assert err <= 1e-5, err


def test_graph_replays_match_eager():
    cfg = small_cfg(name="mx_graph", R=4, S=64, E=16, K=4, B=2, H=256, Hp=192, mode="infer")
    say("mx graph")
    r, d, l, topk, gates = _layer(cfg, 2.0)
    want = l.forward(topk, d["x"], gates).clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        l.forward(topk, d["x"], gates)
    for rep in range(3):
        l.y.fill_(float("nan")), l.out.fill_(float("nan"))
        _ = torch.randn(4096, device="cuda").sum().item()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(l.y, want), rep
