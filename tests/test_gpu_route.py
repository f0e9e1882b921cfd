"""Router and gates' gradient on the GPU against the float64 oracle: choices equal, gates
and gradients within their float32 error bounds."""
import dataclasses
import itertools

import numpy as np
import pytest
import torch

from oracle import moe as M
from oracle import route as RT
from redundant_expert_balancing_amd import _lib as L
from redundant_expert_balancing_amd.layer import MoEProjection
from redundant_expert_balancing_amd.router import MoERouter
from redundant_expert_balancing_amd.synth import LayerConfig, make_dense

from gpu_helpers import say, small_cfg

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def cfg_of(N, E, K, mode="train"):
    return LayerConfig("route", 1, N, E, K, E, 64, 64, "bf16", mode, (1.0,))


def to(logits, dtype):
    return torch.from_numpy(np.asarray(logits, np.float32)).cuda().to(
        torch.bfloat16 if dtype == "bf16" else torch.float32)


def check(cfg, logits, bias, dtype="fp32", **kw):
    """One route and one backward against the oracle."""
    rt = MoERouter(cfg, dtype=dtype, backward=True, **kw)
    t = to(logits, dtype)
    b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
    rt.topk_idx.fill_(-7)
    rt.gates.fill_(-7.0)
    ids, gates = rt.forward(t, b)
    torch.cuda.synchronize()
    lh = t.double().cpu().numpy()
    bh = None if b is None else b.double().cpu().numpy()
    want_ids, want = RT.route(lh, bh, cfg.K, **kw)
    got = gates.double().cpu().numpy()
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    # exp of a rounded argument x: relative error (|x| + 2) u; sums of at most E positive
    # terms add E u at most, two divisions, a product and the sigmoid's own sum 8 u
    with np.errstate(invalid="ignore"):
        x = np.nan_to_num(np.abs(np.where(np.isfinite(lh), lh, 0)).clip(max=200).max(), nan=0)
    tol = (2 * x + cfg.E + 16) * U
    ok = ~np.isnan(want)
    assert (np.abs(got - want)[ok] <= tol * np.abs(want)[ok] + 1e-37).all()
    if cfg.N == 0:
        return
    rng = np.random.default_rng(5)
    dg = rng.standard_normal((cfg.N, cfg.K)).astype(np.float32)
    rt.dlogits.fill_(float("nan"))
    d = rt.backward(t, torch.from_numpy(dg).cuda(), b)
    torch.cuda.synchronize()
    bk = dict(score=kw.get("score", "softmax"), renorm=kw.get("renorm", True),
              scale=kw.get("scale", 1.0))
    ref = RT.route_backward(lh, bh, want_ids, got, dg, **bk)
    d = d.double().cpu().numpy()
    rows = ~np.isnan(got).any(1)
    # terms summed: |g| (|dg| + sum |q dg|) at the chosen, |p| sum |g dg| everywhere else
    ga = np.abs(np.nan_to_num(got))
    terms = (ga * np.abs(dg)).sum(1, keepdims=True) * (1 + 1 / bk["scale"]) + 1e-30
    bound = (2 * x + cfg.E + 2 * cfg.K + 16) * U * terms
    if dtype == "bf16":
        bound = bound + np.abs(ref) * 2.0 ** -8 * (1 + 2.0 ** -7)
    assert (np.abs(d - ref)[rows] <= bound[rows]).all()
    return ids, gates


GROUPS = [dict(), dict(groups=4, top_groups=2, group_top=2), dict(groups=4, top_groups=3, group_top=1)]


@pytest.mark.parametrize("score,renorm,dtype", list(itertools.product(
    ["softmax", "sigmoid"], [True, False], ["fp32", "bf16"])))
@pytest.mark.parametrize("bias", [False, True])
def test_choice_gates_and_gradient(score, renorm, dtype, bias):
    say("route", score, renorm, dtype, bias)
    for N, E, K in ((1, 8, 1), (3, 64, 8), (67, 60, 7), (33, 384, 8), (5, 1024, 32), (130, 100, 3),
                    (9, 264, 6), (1, 256, 8)):
        for g in GROUPS:
            if K > E // 4 * g.get("top_groups", 4):
                continue
            rng = np.random.default_rng(N * E + K)
            b = 0.05 * rng.standard_normal(E) if bias else None
            check(cfg_of(N, E, K), rng.standard_normal((N, E)), b, dtype, score=score,
                  renorm=renorm, scale=2.5, **g)


@pytest.mark.parametrize("E", [1, 2, 63, 65, 97])
def test_odd_expert_counts(E):
    say("route odd", E)
    rng = np.random.default_rng(E)
    for dtype in ("fp32", "bf16"):
        for score in ("softmax", "sigmoid"):
            check(cfg_of(37, E, min(E, 5)), rng.standard_normal((37, E)), None, dtype, score=score,
                  renorm=False)


@pytest.mark.parametrize("E,groups", [(64, 2), (64, 8), (64, 16), (128, 8), (256, 8), (384, 8),
                                      (192, 16), (320, 4), (448, 2), (512, 16)])
def test_groups_of_whole_lanes(E, groups):
    """Group counts of the packed form, with both group scores, plain and biased."""
    say("route groups", E, groups)
    rng = np.random.default_rng(E + groups)
    for top in {max(1, groups // 2), groups}:
        for group_top in (1, 2):
            for score in ("softmax", "sigmoid"):
                for bias in (None, 0.05 * rng.standard_normal(E)):
                    K = min(8, top * (E // groups))
                    check(cfg_of(21, E, K), rng.standard_normal((21, E)), bias, score=score,
                          groups=groups, top_groups=top, group_top=group_top)


@pytest.mark.parametrize("E,groups", [(60, 4), (60, 3), (376, 8), (75, 5), (45, 15), (112, 16),
                                      (200, 2), (10, 5), (16, 16), (48, 3), (512, 8), (480, 15),
                                      (340, 17), (1020, 4), (18, 2), (1024, 8), (720, 3), (600, 1)])
def test_groups_that_do_not_fill_their_lanes(E, groups):
    """Group sizes and counts that leave places empty behind every group, or whole lanes; rows
    with fewer than K experts left among them, near ties, masks and NaN."""
    say("route odd groups", E, groups)
    rng = np.random.default_rng(E * groups)
    per, N = E // groups, 27
    l = rng.standard_normal((N, E))
    l[0] = -np.inf
    l[1, 1:] = -np.inf
    l[2, : E // 2] = -np.inf
    l[3, per:] = -np.inf                       # one group left
    l[4] = float(torch.finfo(torch.float32).min)
    l[5, E - 1] = np.nan
    l[6, E - 1] = 1e30
    l[7] = 1.5 + 2.0 ** -22 * rng.integers(0, 3, E)
    l[8] = 1.5
    l[9] *= 1e4
    off = 0.05 * rng.standard_normal(E)
    off[-per:] = -np.inf                       # the last group switched off
    off[0] = -np.inf
    for top in {1, max(1, groups // 2), groups}:
        for group_top in {1, min(2, per)}:
            for score in ("softmax", "sigmoid"):
                for bias in (None, 0.05 * rng.standard_normal(E), off):
                    for K in {min(8, top * per), min(13, top * per)}:
                        check(cfg_of(N, E, K), l, bias, score=score, groups=groups,
                              top_groups=top, group_top=group_top, renorm=bias is not None)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K", [(64, 8), (384, 8), (384, 5), (100, 1), (384, 16), (256, 10),
                                 (1000, 8), (1024, 12)])
def test_last_choice_next_to_its_neighbour(score, E, K):
    """The K-th best and the next differ by one float32 step and have neighbouring ids, all
    others are far from each other: the higher id is right where it is the larger."""
    say("route last choice", score, E, K)
    rng = np.random.default_rng(E + K)
    N = 61
    l = rng.uniform(-3.0, -1.0, (N, E)).astype(np.float32)
    for g in range(N):
        a = 2 * int(rng.integers(0, E // 2))
        others = np.setdiff1d(np.arange(E), [a, a + 1])
        l[g, rng.permutation(others)[:K - 1]] = 2.0 + 0.125 * np.arange(K - 1)
        l[g, a] = 1.0
        l[g, a + 1] = np.nextafter(np.float32(1.0), np.float32(2.0))
        if g % 3 == 0:
            l[g, [a, a + 1]] = l[g, [a + 1, a]]
    for bias in (None, np.zeros(E, np.float32)):
        check(cfg_of(N, E, K), l, bias, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K", [(128, 16), (384, 12), (384, 9), (1024, 16), (96, 10)])
def test_choices_that_lie_together(score, E, K):
    """All of the K best among consecutive ids, rows with fewer than K experts left, and
    ordinary rows between them."""
    say("route together", score, E, K)
    rng = np.random.default_rng(E * K)
    N = 31
    l = rng.standard_normal((N, E)).astype(np.float32)
    for g in range(0, N, 2):
        at = int(rng.integers(0, E - K + 1))
        l[g, at:at + K] += 20.0
    l[1] = -np.inf
    l[3, 5:] = -np.inf
    l[5] = 0.5
    for renorm in (True, False):
        for bias in (None, 0.05 * rng.standard_normal(E)):
            check(cfg_of(N, E, K), l, bias, score=score, renorm=renorm)
            check(cfg_of(N, E, K), l, bias, "bf16", score=score, renorm=renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [64, 384])
def test_near_ties_are_settled_in_64_bits(score, E):
    """Biased scores and group scores that float32 cannot order: pairs, runs of a dozen (the
    refined list) and of forty (beyond it), tokens of both kinds side by side."""
    say("route near ties", score, E)
    rng = np.random.default_rng(E)
    N = 23
    for run in (2, 12, 40):
        l = rng.standard_normal((N, E)).astype(np.float32)
        for g in range(N):
            if g % 3 == 2:
                continue                       # an ordinary token between them
            at = rng.permutation(E)[:run]
            l[g, at] = 3.0 + 2.0 ** -22 * rng.integers(0, 3, run)
        b = np.zeros(E, np.float32)
        b[::3] = 2.0 ** -25                    # equal logits, biases below float32's step at 1
        for g in (dict(), dict(groups=8, top_groups=3, group_top=2), dict(groups=4, top_groups=2)):
            check(cfg_of(N, E, 8), l, b, score=score, **g)
            check(cfg_of(N, E, 5), l, None, score=score, **g)
    # groups whose best pairs differ by a step or not at all
    l = np.tile(rng.standard_normal(E // 8).astype(np.float32), (N, 8))
    for g in range(N):
        l[g, rng.integers(0, E)] += np.float32(2.0 ** -20)
    for group_top in (1, 2):
        for b in (None, np.full(E, 0.125, np.float32)):
            check(cfg_of(N, E, 6), l, b, score=score, groups=8, top_groups=3, group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_wide_ranges_and_masks_with_groups(score):
    """Rows whose keys span more than the packed range resolves, and masked rows, with the
    groups of the packed form."""
    say("route wide", score)
    rng = np.random.default_rng(8)
    E, N = 128, 24
    l = rng.standard_normal((N, E))
    lowest = float(torch.finfo(torch.float32).min)
    l[0] *= 1e4
    l[1] *= 1e30
    l[2, 3:] = lowest
    l[3] = lowest
    l[4, :120] = -np.inf
    l[5] = -np.inf
    l[6, 64:] = np.nan
    l[7, 9] = np.inf
    l[8, ::2] -= 200.0
    l[9, 5:] -= 1000.0
    l[10, :4] = 50.0
    off = 0.1 * rng.standard_normal(E)
    off[32:64] = -np.inf                       # a whole group switched off
    off[70] = -np.inf
    for renorm in (True, False):
        for g in (dict(), dict(groups=4, top_groups=2, group_top=2), dict(groups=4, top_groups=3)):
            for bias in (None, off):
                for K in (8, 3):
                    check(cfg_of(N, E, K), l, bias, score=score, renorm=renorm, **g)


def test_more_tokens_than_one_launch():
    """2^26 + 5 tokens: the rows behind the first launch are those of a call on them alone."""
    N, E, K = (1 << 26) + 5, 4, 1
    say("route many tokens", N)
    tail = 9
    l = torch.empty((N, E), dtype=torch.bfloat16, device="cuda")
    l.normal_(generator=torch.Generator(device="cuda").manual_seed(0))
    big = MoERouter(cfg_of(N, E, K), score="sigmoid", dtype="bf16", renorm=False, backward=True)
    small = MoERouter(cfg_of(tail, E, K), score="sigmoid", dtype="bf16", renorm=False, backward=True)
    dg = torch.ones((N, K), device="cuda")
    big.forward(l)
    big.backward(l, dg)
    part = l[N - tail:].clone()
    small.forward(part)
    small.backward(part, dg[:tail].contiguous())
    torch.cuda.synchronize()
    for name in ("topk_idx", "gates", "dlogits"):
        assert torch.equal(getattr(big, name)[N - tail:], getattr(small, name)), name
    assert torch.equal(big.topk_idx.long(), l.argmax(1, keepdim=True)) or bool(
        (l.gather(1, big.topk_idx.long()) == l.amax(1, keepdim=True)).all())


def test_empty_layer():
    say("route empty")
    rt = MoERouter(cfg_of(0, 16, 2), backward=True)
    t = torch.zeros((1, 16), device="cuda")
    rt.gates.fill_(7.0)
    rt.forward(t)
    rt.backward(t, torch.zeros((1, 2), device="cuda"))
    torch.cuda.synchronize()
    assert bool((rt.gates == 7.0).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", GROUPS)
def test_ties_go_to_the_lower_id(score, groups):
    """Few distinct logits: equal scores everywhere, with and without an all-zero bias."""
    say("route ties", score, groups)
    rng = np.random.default_rng(3)
    l = rng.integers(-1, 2, (65, 64)).astype(float)
    for b in (None, np.zeros(64)):
        for renorm in (True, False):
            check(cfg_of(65, 64, 6), l, b, "bf16", score=score, renorm=renorm, **groups)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_values_next_to_a_border(score):
    """Biased scores that differ by far less than float32 resolves keep their order: logits
    one float32 step apart, and biases that almost cancel the difference of two scores."""
    say("route border", score)
    rng = np.random.default_rng(4)
    N, E = 64, 32
    base = np.float32(1.5)
    l = np.full((N, E), base)
    for g in range(N):
        l[g] = base + np.float32(2.0 ** -23) * rng.integers(0, 4, E).astype(np.float32)
    check(cfg_of(N, E, 8), l, np.full(E, 0.25), score=score)
    check(cfg_of(N, E, 8), l, None, score=score)
    l = rng.standard_normal((N, E)).astype(np.float32)
    s = 1 / (1 + np.exp(-l[0].astype(np.float64)))
    if score == "softmax":
        s = np.exp(l[0].astype(np.float64)) / np.exp(l[0].astype(np.float64)).sum()
    check(cfg_of(N, E, 8), np.repeat(l[:1], N, 0), (1.0 - s).astype(np.float32), score=score)
    check(cfg_of(N, E, 8), np.repeat(l[:1], N, 0), (1.0 - s).astype(np.float32), score=score,
          groups=4, top_groups=2, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_masks_infinities_and_nan(score, dtype):
    say("route masks", score, dtype)
    rng = np.random.default_rng(6)
    E, K = 48, 4
    lowest = float(torch.finfo(torch.bfloat16).min)
    l = rng.standard_normal((40, E))
    l[0] = -np.inf                       # nothing left
    l[1, 2:] = -np.inf                   # fewer than K left
    l[2] = lowest                        # masks of the type's lowest value
    l[3, 1:] = lowest
    l[4, :] = -1000.0
    l[5, 7] = np.nan
    l[6, 3] = np.inf
    l[7, :3] = np.inf
    l[8, 0] = 1000.0
    l[9] = -90.0 + rng.standard_normal(E)
    l[10, ::2] = -np.inf
    b = 0.1 * rng.standard_normal(E)
    off = b.copy()
    off[5] = off[11] = -np.inf           # switched off ...
    l[11, 5] = np.nan                    # ... whatever their logits hold
    l[12, 11] = np.inf
    high = b.copy()
    high[9] = np.inf
    for renorm in (True, False):
        for g in GROUPS:
            for bias in (None, off, high):
                check(cfg_of(40, E, K), l, bias, dtype, score=score, renorm=renorm, **g)
    most = np.full(E, -np.inf)
    most[[3, 40]] = 0.0
    check(cfg_of(40, E, K), l, most, dtype, score=score)
    bad = b.copy()
    bad[4] = np.nan
    check(cfg_of(40, E, K), l, bad, dtype, score=score)


def test_backward_skips_bad_ids_and_adds_repeated_ones():
    say("route backward ids")
    cfg = cfg_of(2, 8, 3)
    rt = MoERouter(cfg, score="sigmoid", renorm=False, backward=True)
    l = torch.zeros((2, 8), device="cuda")
    rt.topk_idx.copy_(torch.tensor([[1, 1, 9], [-1, 2, 3]], dtype=torch.int32))
    rt.gates.fill_(0.5)
    d = rt.backward(l, torch.ones((2, 3), device="cuda"))
    torch.cuda.synchronize()
    want = torch.zeros((2, 8))
    want[0, 1], want[1, 2], want[1, 3] = 0.5, 0.25, 0.25
    assert torch.equal(d.cpu(), want)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_lone_choice_has_no_gradient(score):
    """K = 1 with renormalised gates: the gate is the scale whatever the logits are."""
    say("route lone choice", score)
    cfg = cfg_of(50, 12, 1)
    rng = np.random.default_rng(9)
    for scale in (1.0, 2.5, 0.3):
        rt = MoERouter(cfg, score=score, scale=scale, backward=True)
        l = torch.from_numpy(rng.standard_normal((50, 12)).astype(np.float32)).cuda()
        _, gates = rt.forward(l)
        d = rt.backward(l, torch.from_numpy(rng.standard_normal((50, 1)).astype(np.float32)).cuda())
        torch.cuda.synchronize()
        assert bool((gates == np.float32(scale)).all()) and not d.any()


@pytest.mark.parametrize("dtype,width,K", [("fp32", 64, 1), ("fp32", 76, 3), ("bf16", 8, 2),
                                           ("bf16", 1408, 8), ("fp32", 1028, 9), ("bf16", 7168, 8),
                                           ("bf16", 264, 32)])
def test_gate_grad(dtype, width, K):
    say("gate grad", dtype, width, K)
    N, E = 53, 64
    other = 64
    sh = L.Shape(1, N, E, K, E, width, other, L.TRAIN, L.BF16 if dtype == "bf16" else L.FP32)
    rng = np.random.default_rng(width)
    src = torch.from_numpy(rng.standard_normal((N * K, width)).astype(np.float32)).cuda()
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    dy = torch.from_numpy(rng.standard_normal((N, width)).astype(np.float32)).cuda().to(dt)
    perm = rng.permutation(N * K).astype(np.int32)
    perm[3], perm[N * K - 1] = -1, N * K + 5          # slots without a row
    out = torch.full((N, K), float("nan"), device="cuda")
    src[torch.from_numpy(np.setdiff1d(np.arange(N * K), perm)).cuda()] = float("nan")
    L.moonep_gate_grad(sh, width, src, torch.from_numpy(perm).cuda(), dy, out)
    torch.cuda.synchronize()
    ok = (perm >= 0) & (perm < N * K)
    a = src.double().cpu().numpy()[np.where(ok, perm, 0)]
    b = np.repeat(dy.double().cpu().numpy(), K, 0)
    want = np.where(ok, (a * b).sum(1), 0.0)
    mag = np.where(ok, (np.abs(a) * np.abs(b)).sum(1), 0.0)
    got = out.double().cpu().numpy().reshape(-1)
    assert (got[~ok] == 0).all()
    # a sum of `width` products in any order: at most width roundings of the magnitude sum
    assert (np.abs(got - want) <= width * U * mag)[ok].all()


def test_router_and_layer_together():
    """logits -> route -> plan .. combine, then dy -> gates' gradient -> dlogits, against the
    dense oracle's differences through the gates."""
    cfg = small_cfg(name="route_layer", R=4, S=24, E=16, K=3, H=64, Hp=64, dtype="fp32")
    say("router and layer", cfg.name)
    d = make_dense(cfg, "cuda", 0, which=("x", "W", "dy"), w_rows=cfg.E + cfg.R * cfg.B)
    rng = np.random.default_rng(0)
    logits = torch.from_numpy(rng.standard_normal((cfg.N, cfg.E)).astype(np.float32)).cuda()
    rt = MoERouter(cfg, score="sigmoid", backward=True, scale=1.5, groups=4, top_groups=2, group_top=2)
    layer = MoEProjection(cfg, backward=True, w_all=d["W"])
    ids, gates = rt.forward(logits)
    y = layer.forward(ids, d["x"], gates)
    dl = rt.backward(logits, layer.gate_grad(d["dy"]))
    torch.cuda.synchronize()
    kw = dict(score="sigmoid", scale=1.5, groups=4, top_groups=2, group_top=2)
    lh = logits.double().cpu().numpy()
    want_ids, want_g = RT.route(lh, None, cfg.K, **kw)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    W = d["W"][:cfg.E].cpu().numpy()
    x, dy = d["x"].cpu().numpy(), d["dy"].cpu().numpy()
    outs = M.dense_expert_outputs(x, W, want_ids).reshape(cfg.N, cfg.K, cfg.Hp)
    ref = (outs * want_g[..., None]).sum(1)
    assert np.abs(y.cpu().numpy() - ref).max() <= 1e-5 * np.sqrt((ref ** 2).mean())
    # the loss <y, dy> as a function of the logits, by central differences
    dgates = (outs * dy[:, None, :].astype(np.float64)).sum(-1)
    got = dl.double().cpu().numpy()
    h = 1e-5
    for g in range(0, cfg.N, 7):
        for e in range(cfg.E):
            f = []
            for s in (1, -1):
                row = lh[g:g + 1].copy()
                row[0, e] += s * h
                i, v = RT.route(row, None, cfg.K, **kw)
                assert np.array_equal(i[0], want_ids[g])
                f.append((v * dgates[g]).sum())
            diff = (f[0] - f[1]) / (2 * h)
            scale = np.abs(dgates[g]).max()
            assert abs(got[g, e] - diff) <= 1e-5 * scale + 1e-6


def test_router_graph_capture_and_stream():
    """Route, gates' gradient and backward captured in one graph and replayed after eager
    work; and issued on a side stream."""
    cfg = small_cfg(name="route_graph", R=2, S=40, E=32, K=4, H=64, Hp=128)
    say("route graph")
    g0 = torch.Generator(device="cuda").manual_seed(0)
    logits = torch.randn((cfg.N, cfg.E), generator=g0, device="cuda")
    d = make_dense(cfg, "cuda", 0, which=("x", "W", "dy"), w_rows=cfg.E + cfg.R * cfg.B)
    rt = MoERouter(cfg, score="sigmoid", backward=True)
    layer = MoEProjection(cfg, backward=True, w_all=d["W"])

    def run():
        ids, gates = rt.forward(logits)
        layer.forward(ids, d["x"], gates)
        rt.backward(logits, layer.gate_grad(d["dy"]))

    run()
    torch.cuda.synchronize()
    want = [t.clone() for t in (rt.topk_idx, rt.gates, rt.dlogits, layer.dgates)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (rt.topk_idx, rt.gates, rt.dlogits, layer.dgates)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for rep in range(3):
        for t in (rt.topk_idx, rt.gates, rt.dlogits, layer.dgates):
            t.fill_(0)
        _ = torch.randn(4096, device="cuda").sum().item()
        g.replay()
        torch.cuda.synchronize()
        got = (rt.topk_idx, rt.gates, rt.dlogits, layer.dgates)
        assert all(torch.equal(a, b) for a, b in zip(want, got)), rep


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_keys_that_hardly_differ(score, dtype):
    """Keys whose spread is too small for the packed range: scores of very low logits with a
    bias of zeros, logits that differ by subnormals, and ordinary and masked rows between."""
    say("route tiny spread", score, dtype)
    rng = np.random.default_rng(12)
    E, N = 64, 32
    l = rng.standard_normal((N, E))
    for g, at in enumerate((-22.0, -25.0, -40.0, -60.0, -75.0, -80.0, -86.0)):
        l[g] += at
    l[8:12] = 0.0
    l[8, 37] = 1e-35
    l[9] = rng.integers(0, 4, E) * 1e-35
    l[10] = rng.integers(0, 5, E) * 2.0 ** -133         # subnormal in both types
    l[11] = rng.integers(-3, 3, E) * 1e-33
    l[12] = 1e-3 + 2.0 ** -30 * rng.integers(0, 4, E)
    l[13] = -80.0 + rng.standard_normal(E)
    l[13, 5:] = -np.inf
    l[14] = -np.inf
    l[15, 9:] = -80.0
    same = np.full(E, 1e-35)
    for renorm in (True, False):
        for g in (dict(), dict(groups=4, top_groups=2, group_top=2), dict(groups=8, top_groups=5)):
            for bias in (None, np.zeros(E), same):
                for K in (8, 12):
                    check(cfg_of(N, E, K), l, bias, dtype, score=score, renorm=renorm, **g)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_of_the_lowest_value(score):
    """Experts put last by a bias of float32's lowest value, which masks nothing: near ties
    among the others, and rows that need some of them."""
    say("route lowest bias", score)
    rng = np.random.default_rng(13)
    E, N = 64, 33
    l = rng.standard_normal((N, E)).astype(np.float32)
    l[::3] = 1.5 + 2.0 ** -23 * rng.integers(0, 4, (len(l[::3]), E))
    for left in (40, 20, 6):
        b = np.full(E, np.finfo(np.float32).min)
        b[rng.permutation(E)[:left]] = 0.0
        for g in (dict(), dict(groups=8, top_groups=5, group_top=2), dict(groups=4, top_groups=3)):
            for K in (8, 12):
                check(cfg_of(N, E, K), l, b, score=score, **g)


def test_last_choice_at_the_end_of_the_packed_range():
    """Biases of about -64 on all but one expert put the last choice 64 below the best, where
    the packed range ends; its rivals' scores differ by less than a float32 sum resolves."""
    say("route range end")
    rng = np.random.default_rng(14)
    E, N, K = 64, 1024, 2
    step = 2.0 ** -18                          # of float32 numbers in [-64, -32)
    b = -64.0 + step * rng.integers(0, 50000, E)
    b[0] = 0.0
    # sums just below the middle of two float32 numbers, 8 .. 23 steps below hi - 64 = -63.5
    key = -63.5 - step * (8.5 + np.arange(N)[:, None] % 16) + 2e-8 * (rng.standard_normal((N, E)) - 3.0)
    s = key - b
    s[:, 0] = 0.5
    check(cfg_of(N, E, K), np.log(s / (1.0 - s)), b, score="sigmoid")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_group_scores_beyond_float32(score):
    """Two biases of float32's lowest (or highest) value add up to more than float32 holds: such
    a group still comes before one whose experts are all switched off, and ties to the lower."""
    say("route group sums", score)
    rng = np.random.default_rng(15)
    E, N, per = 16, 13, 4
    l = rng.standard_normal((N, E))
    low, high = float(np.finfo(np.float32).min), float(np.finfo(np.float32).max)
    for groups in ((-np.inf, low, 0.0, 0.0), (-np.inf, 0.0, low, low), (low, -np.inf, low, 0.0),
                   (low, low, -np.inf, low), (0.75 * high, high, 0.0, high), (low, 0.6 * low, 0.0, -np.inf),
                   (-np.inf, -np.inf, low, -np.inf)):
        b = np.repeat(np.array(groups), per)
        for top, K in ((3, 10), (2, 6), (1, 3)):
            check(cfg_of(N, E, K), l, b, score=score, groups=4, top_groups=top, group_top=2)
