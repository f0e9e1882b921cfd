"""8-bit integer experts on the GPU: stored bytes equal the oracle's, products within the three
float32 roundings behind their exact sums, the layers on them, and their gradients.

U = 2^-24 is half a step of float32, relative to the value. A result is (sum * row scale) *
column scale: the sum's conversion and two products, each off by at most U, so within 3.01 U of
the exact value (1 + U)^3; one more with an addition, which is relative to the sum of both.
"""
import numpy as np
import pytest
import torch

from oracle import ffn as FF
from oracle import int8 as I
from oracle import plan as P
from redundant_expert_balancing_amd import _lib as L
from redundant_expert_balancing_amd import int8
from redundant_expert_balancing_amd.int8 import IntFFN, IntProjection
from redundant_expert_balancing_amd.synth import make_dense, make_routing

from gpu_helpers import say, small_cfg

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TINY = 1e-37                     # products of subnormal scales
NAN = float("nan")


def _dt(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _shape(H, Hp, dtype="bf16", S=8, E=4, K=1, mode=L.INFER, R=1):
    return L.Shape(R, S, E, K, E // R if mode == L.TRAIN else 0, H, Hp, mode,
                   L.BF16 if dtype == "bf16" else L.FP32)


def _wide(rng, shape):
    x = rng.standard_normal(shape) * 2.0 ** rng.integers(-3, 4, shape)
    x[rng.random(shape) < 0.05] = 0.0
    return x.astype(np.float32)


def _cuda(a, dtype="fp32"):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(_dt(dtype))


def _np(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,width", [(1, 8), (3, 64), (7, 96), (33, 128), (5, 544), (6, 1000), (17, 1408),
                                        (2, 4096), (9, 7168), (3, 16392), (2, 131072)])
def test_quantise_rows(dtype, rows, width):
    say("int rows", dtype, rows, width)
    rng = np.random.default_rng(width)
    x = _cuda(_wide(rng, (rows, width)), dtype)
    x[0, :8] = torch.tensor([127.0, 0.5, 1.5, -2.5, 3.5, 63.5, -126.5, 0.0])     # ties, if 127 is the largest
    if rows > 4:
        x[1] = 0
        x[2, width - 1], x[3, 0] = float("nan"), float("inf")
        x[4] *= 2.0 ** -125
    q, s = int8.buffers(rows, width)
    q.fill_(-86), s.fill_(NAN)
    L.moonep_int_quantize(_shape(64, 64, dtype), rows, width, x, q, s)
    torch.cuda.synchronize()
    want_q, want_s = I.rows(_np(x))
    assert np.array_equal(s.cpu().numpy(), want_s.astype(np.float32), equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), I.pack_rows(want_q))


def test_many_rows():
    """More rows than one launch has wavefronts."""
    say("int many rows")
    x = torch.randn((300001, 8), device="cuda", generator=torch.Generator("cuda").manual_seed(0))
    q, s = int8.buffers(300001, 8)
    L.moonep_int_quantize(_shape(64, 64, "fp32"), 300001, 8, x, q, s)
    torch.cuda.synchronize()
    want_q, want_s = I.rows(_np(x))
    assert np.array_equal(s.cpu().numpy(), want_s.astype(np.float32))
    assert np.array_equal(q.cpu().numpy()[:, :8], want_q) and not q[:, 8:].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,Hp", [(8, 8), (64, 64), (160, 48), (1408, 72), (520, 200)])
def test_weights_there_and_back(dtype, H, Hp):
    say("int weights", dtype, H, Hp)
    E = 3
    rng = np.random.default_rng(H)
    w = _cuda(_wide(rng, (E, H, Hp)), dtype)
    w[1, :, 3] = 0
    w[2, H - 1, Hp - 1] = float("inf")
    sh = _shape(H, Hp, dtype, E=E)
    wq, ws = int8.weight_buffers(E, H, Hp)
    wt, _ = int8.weight_buffers(E, Hp, H)
    wq.fill_(-86), ws.fill_(NAN), wt.fill_(-86)
    L.moonep_int_quantize_weight(sh, w, wq, ws)
    L.moonep_int_transpose_weight(sh, wq, wt)
    torch.cuda.synchronize()
    for e in range(E):
        q, s = I.weight(_np(w[e]))
        assert np.array_equal(ws[e].cpu().numpy(), I.pack_scales(s), equal_nan=True)
        assert np.array_equal(wq[e].cpu().numpy(), I.pack_weight(q))
        assert np.array_equal(wt[e].cpu().numpy(), I.pack_weight(q.T))


def test_binding_refusals():
    """What must not reach a kernel as an address is refused before the call."""
    say("int refusals")
    sh = _shape(128, 64, S=4, E=1)
    x = torch.zeros((4, 128), device="cuda", dtype=torch.bfloat16)
    q, s = int8.buffers(4, 128)
    call = lambda **k: L.moonep_int_quantize(sh, *[{**dict(rows=4, width=128, src=x, q=q, scales=s), **k}[n]      # noqa: E731
                                                   for n in ("rows", "width", "src", "q", "scales")])
    call()
    for k, why in ((dict(src=x.float()), "dtype"), (dict(src=x.cpu()), "GPU tensor"),
                   (dict(src=x.t()), "contiguous"), (dict(rows=5), "bytes"), (dict(q=None), "required"),
                   (dict(q=q[:, :64].contiguous()), "bytes"), (dict(scales=s.double()), "dtype")):
        with pytest.raises(ValueError, match=why):
            call(**k)
    for k in (dict(rows=-1), dict(width=120 + 4), dict(width=1 << 40, src=None)):
        with pytest.raises((ValueError, L.MoonepError)):
            call(**k)
    with pytest.raises(TypeError):
        L.moonep_int_quantize(object(), 4, 128, x, q, s)
    with pytest.raises(ValueError):
        L.moonep_int_quantize(sh, "four", 128, x, q, s)
    with pytest.raises(TypeError):
        L.moonep_int_quantize(sh, 4, None, x, q, s)
    c = torch.zeros((4, 64), device="cuda")
    wq, ws = int8.weight_buffers(1, 128, 64)
    wq.zero_(), ws.zero_()
    L.moonep_int_gemm(sh, 4, q, s, wq, None, None, c)
    with pytest.raises(ValueError, match="wq"):
        L.moonep_int_gemm(sh, 4, q, s, wq[:, :2].contiguous(), None, None, c)
    with pytest.raises(ValueError, match="add"):
        L.moonep_int_gemm(sh, 4, q, s, wq, None, c[:3], c)
    with pytest.raises(L.MoonepError) as e:
        L.moonep_int_quantize_grad(sh, x[:, :64].contiguous(), None, None, ws, None, q, s)
    assert e.value.status == L.EMODE
    torch.cuda.synchronize()


def _layer(cfg, alpha, seed=0):
    r = make_routing(cfg, 3.0, seed=seed, alpha=alpha)
    d = make_dense(cfg, "cuda", seed, which=("x", "W"))
    l = IntProjection(cfg)
    l.wq.fill_(-1), l.wscales.fill_(NAN)          # unused slots stay NaN
    l.quantise_weights(d["W"])
    topk, gates = torch.from_numpy(r.topk_idx).cuda(), torch.from_numpy(r.gates).cuda()
    l.out.fill_(NAN), l.y.fill_(NAN)
    return r, d, l, topk, gates


def _check_layer(cfg, alpha, experts=None, seed=0):
    say("int layer", cfg)
    r, d, l, topk, gates = _layer(cfg, alpha, seed)
    y = l.forward(topk, d["x"], gates)
    torch.cuda.synchronize()
    pl = P.plan(r.topk_idx, cfg.R, cfg.S, cfg.E, cfg.K, cfg.B, cfg.mode)
    assert np.array_equal(l.slot_map.cpu().numpy()[:cfg.N * cfg.K], pl.slot_map)
    qx, sx = I.rows(_np(d["x"]))
    out = _np(l.out)[pl.slot_map]
    for e in range(cfg.E) if experts is None else experts:
        tok, kk = np.nonzero(r.topk_idx == e)
        if not len(tok):
            continue
        want = I.product(qx[tok], sx[tok], *I.weight(_np(d["W"][e])))
        assert (np.abs(out[tok * cfg.K + kk] - want) <= 3.01 * U * np.abs(want) + TINY).all(), e
    assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(l.out).all())
    parts = out.reshape(cfg.N, cfg.K, -1) * r.gates.astype(np.float64)[..., None]
    assert (np.abs(_np(y) - parts.sum(1)) <= (cfg.K + 1) * U * np.abs(parts).sum(1) + 1e-30).all()


@pytest.mark.parametrize("kw", [
    dict(R=1, S=1, E=4, K=1, B=0, H=64, Hp=64),                  # one token, one expert
    dict(R=1, S=1, E=16, K=8, B=0, H=512, Hp=128),               # one token
    dict(R=1, S=3, E=4, K=2, B=0, H=8, Hp=8),                    # the smallest rows
    dict(R=2, S=5, E=16, K=3, B=2, H=192, Hp=328),               # columns that end inside a block
    dict(R=4, S=37, E=16, K=2, B=4, H=136, Hp=72),
    dict(R=4, S=64, E=8, K=2, B=1, H=1408, Hp=192),              # overflow rows
    dict(R=1, S=700, E=4, K=2, B=0, H=584, Hp=520),              # segments beyond a tile
    dict(R=2, S=512, E=8, K=4, B=4, H=320, Hp=600),
    dict(R=2, S=2048, E=8, K=2, B=2, H=200, Hp=520),             # 128-row tiles
    dict(R=8, S=600, E=16, K=2, B=2, H=1032, Hp=1096),           # 256-row tiles
])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_layer_against_the_oracle(kw, dtype):
    _check_layer(small_cfg(name="int", dtype=dtype, mode="infer", **kw), 2.0)


def test_training_plan_and_every_slot():
    _check_layer(small_cfg(name="int_train", R=4, S=96, E=16, K=4, H=256, Hp=128), 2.5)


def test_long_segments_and_wide_layers():
    """More tiles than one round of the card, sampled experts."""
    _check_layer(small_cfg(name="int_large", R=4, S=4096, E=32, K=4, B=8, H=1024, Hp=1096,
                           mode="infer"), 1.0, experts=[0, 3, 11, 31])


def test_empty_layer():
    say("int empty")
    cfg = small_cfg(name="int_empty", R=2, S=0, E=8, K=2, B=2, H=128, Hp=64, mode="infer")
    l = IntFFN(cfg, shared=64)
    z = lambda *s, **k: torch.zeros(s, device="cuda", **k)      # noqa: E731
    l.forward(z(1, 2, dtype=torch.int32), z(1, 128, dtype=torch.bfloat16), z(1, 2))
    torch.cuda.synchronize()


def _operands(H, W, rows, E=1, dtype="bf16", seed=0):
    """Rounded rows and weights on the GPU and the oracle's, from one generator."""
    rng = np.random.default_rng(seed)
    x = _cuda(_wide(rng, (rows, H)), dtype)
    w = _cuda(_wide(rng, (E, H, W)), dtype)
    sh = _shape(H, W, dtype, S=rows, E=E)
    xq, xs = int8.buffers(rows, H)
    wq, ws = int8.weight_buffers(E, H, W)
    L.moonep_int_quantize(sh, rows, H, x, xq, xs)
    L.moonep_int_quantize_weight(sh, w, wq, ws)
    return sh, x, w, xq, xs, wq, ws


def _workspace(sh):
    ws = torch.empty(L.moonep_workspace_bytes(sh) // 4, dtype=torch.int32, device="cuda")
    L.moonep_workspace_init(sh, ws)
    return ws


@pytest.mark.parametrize("S,cu,part", [
    (70, [0, 3, 3, 68, 70], [0, 2, 2, 40, 41]),
    (3000, [0, 900, 900, 2999, 3000], [0, 700, 700, 1800, 1801]),       # segments of many rows
])
def test_rows_in_place_and_bad_positions(S, cu, part):
    """src_index NULL reads one row per position; positions outside the plan give zeros."""
    say("int in place", S)
    E, H, Hp = 4, 192, 8 * 600
    sh, x, w, xq, xs, wq, wsc = _operands(H, Hp, S, E)
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, part = torch.tensor([cu], **i32), torch.tensor([part], **i32)
    ws = _workspace(sh)
    a, b, c = (torch.full((S, Hp), NAN, device="cuda") for _ in range(3))
    ident = torch.arange(S, **i32)
    L.moonep_int_grouped_gemm(sh, xq, xs, None, wq, wsc, cu, a, ws)
    L.moonep_int_grouped_gemm(sh, xq, xs, ident, wq, wsc, cu, b, ws)
    broken = ident.clone()
    broken[5], broken[S - 1] = -1, S
    L.moonep_int_grouped_gemm(sh, xq, xs, broken, wq, wsc, cu, c, ws)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and bool(torch.isfinite(a).all())
    assert not c[5].any() and not c[S - 1].any()
    keep = [i for i in range(S) if i not in (5, S - 1)]
    assert torch.equal(c[keep], a[keep])
    # rows behind the last segment are left as they were
    end = int(part[0, -1])
    c.fill_(7.0)
    L.moonep_int_grouped_gemm(sh, xq, xs, ident, wq, wsc, part, c, ws)
    torch.cuda.synchronize()
    assert bool((c[end:] == 7.0).all()) and torch.equal(c[:2], a[:2])
    # an empty plan
    L.moonep_int_grouped_gemm(sh, xq, xs, ident, wq, wsc, torch.zeros_like(part), c, ws)
    torch.cuda.synchronize()
    assert bool((c[end:] == 7.0).all())
    # without column scales: all 1
    L.moonep_int_grouped_gemm(sh, xq, xs, None, wq, None, cu, c, ws)
    torch.cuda.synchronize()
    q, s = I.rows(_np(x[:2]))
    want = (q @ I.weight(_np(w[0]))[0]) * s[:, None]
    assert (np.abs(_np(c[:2]) - want) <= 2.01 * U * np.abs(want)).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,H,Hp", [(1, 64, 64), (1, 2048, 328), (5, 8, 8), (16, 200, 600), (17, 128, 64),
                                       (40, 136, 1000), (65, 1408, 80), (300, 72, 520),
                                       (1000, 256, 264), (4100, 512, 2048), (5000, 64, 8200), (9000, 200, 2600),
                                       (1100, 328, 2056), (33, 128, 16)])
def test_dense_product(rows, H, Hp, dtype):
    say("int dense", rows, H, Hp, dtype)
    sh, x, w, xq, xs, wq, ws = _operands(H, Hp, rows, dtype=dtype, seed=rows)
    add = torch.randn((rows, Hp), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    c, d = (torch.full((rows + 1, Hp), NAN, device="cuda") for _ in range(2))
    L.moonep_int_gemm(sh, rows, xq, xs, wq, ws, None, c)
    d[:rows] = add
    L.moonep_int_gemm(sh, rows, xq, xs, wq, ws, d, d)           # in place
    torch.cuda.synchronize()
    want = I.product(*I.rows(_np(x)), *I.weight(_np(w[0])))
    assert (np.abs(_np(c[:rows]) - want) <= 3.01 * U * np.abs(want) + TINY).all()
    assert torch.equal(d[:rows], c[:rows] + add)                # one float32 addition
    assert bool(torch.isnan(c[rows:]).all()) and bool(torch.isnan(d[rows:]).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,H,Hp,E", [(1, 64, 32, 1), (16, 200, 96, 1), (37, 136, 352, 4), (300, 72, 160, 3),
                                         (900, 256, 128, 2), (5000, 320, 416, 4), (20000, 136, 416, 4), (6000, 72, 992, 1)])
def test_swiglu_against_the_two_steps(rows, H, Hp, E, dtype):
    """The fused product against the product followed by moonep_swiglu, dense and grouped: the same
    pre-activation, the same activation in float32, and in bfloat16 one whose exponential and
    reciprocal are the hardware's, so that it may round to the neighbour: off by a step (2^-7 of
    the value) where the float32 values lie on two sides of a border. The reciprocal of
    1 + e^-gate above 2^126 is below 2^-126, the smallest normal number, and may come out as 0:
    off by |gate * up| * 2^-126."""
    say("int swiglu", rows, H, Hp, E, dtype)
    sh, x, w, xq, xs, wq, ws = _operands(H, 2 * Hp, rows, E, dtype, seed=rows)
    ffn = _shape(H, Hp, dtype, S=rows, E=E)
    cut = np.sort(np.random.default_rng(E).integers(0, rows + 1, E - 1)).tolist()
    cu = torch.tensor([[0] + cut + [rows]], dtype=torch.int32, device="cuda")
    work = _workspace(sh)
    h = torch.full((rows, 2 * Hp), NAN, device="cuda")
    new = lambda n: torch.full((rows + 1, n), NAN, device="cuda", dtype=_dt(dtype))     # noqa: E731
    a0, h0, a1, h1, a2 = new(Hp), new(2 * Hp), new(Hp), new(2 * Hp), new(Hp)
    L.moonep_int_grouped_gemm(sh, xq, xs, None, wq, ws, cu, h, work)
    L.moonep_swiglu(ffn, h, a0, h0)
    L.moonep_int_grouped_gemm_swiglu(ffn, xq, xs, None, wq, ws, cu, a1, h1, work)
    L.moonep_int_grouped_gemm_swiglu(ffn, xq, xs, None, wq, ws, cu, a2, None, work)
    torch.cuda.synchronize()
    def same(got, want):
        if dtype == "fp32":
            assert torch.equal(got[:rows], want[:rows])
        else:
            d, w = (got[:rows].double() - want[:rows].double()).abs(), want[:rows].double().abs()
            v = h.double().view(rows, -1, 2, 32)
            low = (v[:, :, 0] * v[:, :, 1]).abs().reshape(rows, -1) * 2.0 ** -126
            assert bool((d <= 2.0 ** -7 * w + low + TINY).all())

    same(a1, a0)
    assert torch.equal(a1[:rows], a2[:rows]) and torch.equal(h1[:rows], h0[:rows])
    for got in (a1, a2, h1):
        assert bool(torch.isnan(got[rows:]).all())
    # a row and a column whose scales are not numbers
    hurt, part = xs.clone(), ws.clone()
    hurt[rows // 2] = NAN
    part[:, 33] = NAN                 # an up column, of intermediate column 1
    L.moonep_int_grouped_gemm_swiglu(ffn, xq, hurt, None, wq, part, cu, a2, h1, work)
    torch.cuda.synchronize()
    want = torch.zeros((rows, Hp), dtype=torch.bool, device="cuda")
    want[rows // 2], want[:, 1] = True, True
    assert torch.equal(torch.isnan(a2[:rows]), want)
    assert torch.equal(torch.where(want, 0, a2[:rows]), torch.where(want, 0, a1[:rows]))
    L.moonep_int_grouped_gemm_swiglu(ffn, xq, xs, None, wq, ws, cu, a2, h1, work)
    if E > 1:
        return
    a1.fill_(NAN), h1.fill_(NAN)
    L.moonep_int_gemm_swiglu(ffn, rows, xq, xs, wq, ws, a1, h1)
    torch.cuda.synchronize()
    assert torch.equal(a1[:rows], a2[:rows]) and torch.equal(h1[:rows], h0[:rows])
    want = I.product(*I.rows(_np(x)), *I.weight(_np(w[0])))
    # half a step of the type, and the three float32 roundings before it
    half = 2.0 ** -8 if dtype == "bf16" else U
    assert (np.abs(_np(h1[:rows]) - want) <= (half * (1 + 2.0 ** -7) + 3.01 * U) * np.abs(want) + TINY).all()


def test_a_broken_token_or_channel_stays_in_its_place():
    say("int nan")
    cfg = small_cfg(name="int_nan", R=2, S=40, E=8, K=2, B=2, H=256, Hp=128, mode="infer")
    r, d, l, topk, gates = _layer(cfg, 2.0)
    d["x"][7, 100] = NAN
    d["x"][9, 3] = float("-inf")
    y = l.forward(topk, d["x"], gates)
    torch.cuda.synchronize()
    bad = torch.isnan(y).any(1).cpu()
    assert bool(torch.isnan(y[[7, 9]]).all()) and int(bad.sum()) == 2
    d["x"][7, 100] = d["x"][9, 3] = 0.0
    d["W"][3, 5, 17] = float("inf")
    l.quantise_weights(d["W"])
    y = l.forward(topk, d["x"], gates)
    torch.cuda.synchronize()
    hit = torch.from_numpy((r.topk_idx == 3).any(1))
    assert int(hit.sum()) > 0
    assert torch.equal(torch.isnan(y).cpu(), hit[:, None] & (torch.arange(128) == 17))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("R,S,E,K,Hp", [(1, 9, 4, 2, 8), (4, 37, 16, 3, 200), (2, 300, 8, 4, 1408), (1, 4, 2, 1, 8200)])
def test_gradient_rows(R, S, E, K, Hp, dtype):
    """Gathered with gates, and in place; behind the last row nothing is written."""
    say("int gradient rows", R, S, E, K, Hp, dtype)
    rng = np.random.default_rng(Hp)
    sh = _shape(64, Hp, dtype, S=S, E=E, K=K, mode=L.TRAIN, R=R)
    N, SK, EB = R * S, S * K, E + E // R
    NK = N * K
    cols = 16 * -(-Hp // 16)
    wsc = _cuda(rng.random((E + E, cols)) + 0.5)
    lens = rng.multinomial(SK - 3, np.ones(EB) / EB, size=R)
    lens[:, ::3] = 0                                                     # empty rows of the view
    cu = np.concatenate([np.zeros((R, 1), int), np.cumsum(lens, 1)], 1)
    src_index = rng.permutation(NK)
    src_index[2] = -1
    src_index[NK // 2] = NK
    gates = rng.random((N, K)).astype(np.float32)
    dy = _cuda(_wide(rng, (N, Hp)), dtype)
    dh = _cuda(_wide(rng, (NK, Hp)), dtype)
    dy[1, 0] = NAN
    i32 = dict(dtype=torch.int32, device="cuda")
    cu_t, src_t = torch.tensor(cu, **i32), torch.tensor(src_index, **i32)
    wrow = np.full(NK, -1)
    for q in range(R):
        for i in range(EB):
            wrow[q * SK + cu[q, i]:q * SK + cu[q, i + 1]] = i if i < E else E + q * (E // R) + i - E
    live = wrow >= 0
    W = _np(wsc)[:, :Hp][np.maximum(wrow, 0)]

    def check(q, s, dc, gate, there, live):
        want_q, want_s = I.grad_rows(dc, W if live is not None else np.broadcast_to(W0, dc.shape))
        want_s = np.where(there, (want_s.astype(np.float32) * gate).astype(np.float64), 0.0)
        want_q = np.where(there[:, None], want_q, 0)
        m = live if live is not None else np.ones(NK, bool)
        assert np.array_equal(s.cpu().numpy()[m], want_s[m].astype(np.float32), equal_nan=True)
        assert np.array_equal(q.cpu().numpy()[m], I.pack_rows(want_q)[m])
        assert (q.cpu().numpy()[~m] == -86).all() and np.isnan(s.cpu().numpy()[~m]).all()

    def buffers():
        q, s = int8.buffers(NK, Hp)
        q.fill_(-86), s.fill_(NAN)
        return q, s

    there = (src_index >= 0) & (src_index < NK)
    at = np.where(there, src_index, 0)
    q, s = buffers()
    L.moonep_int_quantize_grad(sh, dy, src_t, _cuda(gates), wsc, cu_t, q, s)
    torch.cuda.synchronize()
    check(q, s, _np(dy)[at // K], gates.reshape(-1)[at], there, live)
    q, s = buffers()
    L.moonep_int_quantize_grad(sh, dh, None, None, wsc, cu_t, q, s)
    torch.cuda.synchronize()
    check(q, s, _np(dh), np.float32(1), np.ones(NK, bool), live)
    q, s = buffers()                                                     # one weight for all
    W0 = _np(wsc)[0, :Hp]
    L.moonep_int_quantize_grad(sh, dh, None, None, wsc, None, q, s)
    torch.cuda.synchronize()
    check(q, s, _np(dh), np.float32(1), np.ones(NK, bool), None)


@pytest.mark.parametrize("Hp", [200, 8200])
def test_gradient_rows_ahead_of_the_first(Hp):
    """Positions ahead of a rank's first row are left as they were, the ones behind it are not."""
    say("int gradient rows ahead", Hp)
    R, S, E = 2, 12, 4
    sh = _shape(64, Hp, S=S, E=E, K=2, mode=L.TRAIN, R=R)
    g = torch.Generator("cuda").manual_seed(Hp)
    dh = torch.randn((R * S * 2, Hp), device="cuda", generator=g).bfloat16()
    wsc = torch.ones((2 * E, 16 * -(-Hp // 16)), device="cuda")
    cu = torch.tensor([[5, 5, 9, 9, 9, 20, 20], [0, 3, 7, 11, 15, 20, 24]], dtype=torch.int32, device="cuda")
    q, s = int8.buffers(R * S * 2, Hp)
    q0, s0 = int8.buffers(R * S * 2, Hp)
    q.fill_(-86), s.fill_(NAN)
    L.moonep_int_quantize(sh, R * S * 2, Hp, dh, q0, s0)      # scales of one: the same rows
    L.moonep_int_quantize_grad(sh, dh, None, None, wsc, cu, q, s)
    torch.cuda.synchronize()
    out = torch.zeros(R * S * 2, dtype=torch.bool, device="cuda")
    out[:5], out[20:24] = True, True
    assert torch.equal(q[~out], q0[~out]) and torch.equal(s[~out], s0[~out])
    assert bool((q[out] == -86).all()) and bool(torch.isnan(s[out]).all())


def _ffn(cfg, shared=0, backward=False, seed=0):
    r = make_routing(cfg, 3.0, alpha=2.0, seed=seed)
    d = make_dense(cfg, "cuda", seed, which=("x", "W1", "W2"))
    l = IntFFN(cfg, shared=shared, backward=backward)
    g = torch.Generator("cuda").manual_seed(seed + 1)
    s1 = s2 = None
    if shared:
        s1 = (torch.randn((cfg.H, 2 * shared), device="cuda", generator=g) * cfg.H ** -0.5).to(l.dtype)
        s2 = (torch.randn((shared, cfg.H), device="cuda", generator=g) * shared ** -0.5).to(l.dtype)
    l.quantise_weights(d["W1"], d["W2"], s1, s2)
    dy = torch.randn((cfg.N, cfg.H), device="cuda", generator=g).to(l.dtype)
    topk, gates = torch.from_numpy(r.topk_idx).cuda(), torch.from_numpy(r.gates).cuda()
    return r, d, l, topk, gates, s1, s2, dy


def _close(got, want, rel, base=0.0):
    assert (np.abs(got - want) <= rel * np.abs(want) + base).all(), np.abs(got - want).max()


def _check_ffn(cfg, shared, backward):
    """Each step against the oracle's on the values that the layer itself fed it."""
    say("int ffn", cfg, shared, backward)
    r, d, l, topk, gates, s1, s2, dy = _ffn(cfg, shared, backward)
    y = l.forward(topk, d["x"], gates)
    dx = l.backward(dy, gates) if backward else None
    torch.cuda.synchronize()
    half = 2.0 ** -8 if cfg.dtype == "bf16" else U
    N, K, H = cfg.N, cfg.K, cfg.H
    qx, sx = I.rows(_np(d["x"]))
    sm = l.slot_map.cpu().numpy()
    act, z = _np(l.act), _np(l.z)
    hs, da, dh, dxp = (_np(t) for t in (l.hs, l.da, l.dh, l.dxp)) if backward else (None,) * 4
    g64 = r.gates.astype(np.float64)

    def swiglu(h, got):
        # float32 roundings of h, exp and a quotient and product (under 10 U), and the type's
        gate, up = FF.gate_up_columns(h.shape[1] // 2)
        want = I.swiglu(h)
        slack = np.abs(h[:, gate] * h[:, up]) * 10 * U         # |d silu| <= 1.1
        assert (np.abs(got - want) <= (half * (1 + 2.0 ** -7) + 10 * U) * np.abs(want) + 2 * slack + TINY).all()

    for e in range(cfg.E):
        tok, kk = np.nonzero(r.topk_idx == e)
        if not len(tok):
            continue
        pos = sm[tok * K + kk]
        w1, sc1 = I.weight(_np(d["W1"][e]))
        w2, sc2 = I.weight(_np(d["W2"][e]))
        h = I.product(qx[tok], sx[tok], w1, sc1)
        swiglu(h, act[pos])
        want = I.product(*I.rows(act[pos]), w2, sc2)
        _close(z[pos], want, 3.01 * U, TINY)
        if backward:
            _close(hs[pos], h, half * (1 + 2.0 ** -7) + 3.01 * U, TINY)
            gq, gs = I.grad_rows(_np(dy)[tok], np.broadcast_to(sc2, (len(tok), H)), g64[tok, kk])
            # the sum's conversion, the scale's product with the gate and the result's
            _close(da[pos], (gq @ w2.T) * gs[:, None], 3.01 * U, TINY)
            gq, gs = I.grad_rows(dh[pos], np.broadcast_to(sc1, dh[pos].shape))
            _close(dxp[pos], (gq @ w1.T) * gs[:, None], 2.01 * U, TINY)
    parts = z[sm].reshape(N, K, H) * g64[..., None]
    want, mag = parts.sum(1), np.abs(parts).sum(1)
    if shared:
        sq1, ss1 = I.weight(_np(s1))
        sq2, ss2 = I.weight(_np(s2))
        h = I.product(qx, sx, sq1, ss1)
        swiglu(h, _np(l.s_act)[:N])
        more = I.product(*I.rows(_np(l.s_act)[:N]), sq2, ss2)
        want, mag = want + more, mag + np.abs(more)
    assert (np.abs(_np(y) - want) <= (K + 5) * U * mag + TINY).all()
    if not backward:
        return
    parts = dxp[sm].reshape(N, K, H)
    want, mag = parts.sum(1), np.abs(parts).sum(1)
    if shared:
        gq, gs = I.grad_rows(_np(dy), np.broadcast_to(ss2, (N, H)))
        _close(_np(l.s_da), (gq @ sq2.T) * gs[:, None], 2.01 * U, TINY)
        gq, gs = I.grad_rows(_np(l.s_dh), np.broadcast_to(ss1, (N, 2 * shared)))
        more = (gq @ sq1.T) * gs[:, None]
        want, mag = want + more, mag + np.abs(more)
    assert (np.abs(_np(dx) - want) <= (K + 5) * U * mag + TINY).all()
    dg = _np(l.gate_grad(dy))
    prod = z[sm].reshape(N, K, H) * _np(dy)[:, None]
    assert (np.abs(dg - prod.sum(2)) <= H * U * np.abs(prod).sum(2) + TINY).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kw,shared,backward", [
    (dict(R=4, S=30, E=8, K=2, B=2, H=128, Hp=192, mode="infer"), 0, False),
    (dict(R=2, S=1, E=8, K=3, B=1, H=136, Hp=32, mode="infer"), 96, False),
    (dict(R=4, S=24, E=8, K=2, H=128, Hp=96), 0, True),
    (dict(R=2, S=33, E=4, K=2, H=200, Hp=64), 160, True),
])
def test_ffn_against_the_oracle(kw, shared, backward, dtype):
    _check_ffn(small_cfg(name="int_ffn", dtype=dtype, **kw), shared, backward)


def test_input_gradient_against_differences():
    """The gradient of <dy, y> for x, with the rounding of x to 8 bits taken as the identity:
    central differences of the float64 layer on the rounded weights. What the layer rounds on the
    way (both gradients to 8 bits, half a scale per value of the reduction, and intermediates to
    float32) bounds the difference."""
    cfg = small_cfg(name="int_diff", R=2, S=6, E=4, K=2, H=64, Hp=32, dtype="fp32")
    say("int differences")
    r, d, l, topk, gates, s1, s2, dy = _ffn(cfg, 32, True)
    l.forward(topk, d["x"], gates)
    dx = _np(l.backward(dy, gates))
    torch.cuda.synchronize()
    xv = I.values(*I.rows(_np(d["x"])))
    W1, W2 = ([(lambda q, s: q * s)(*I.weight(_np(w[e]))) for e in range(cfg.E)] for w in (d["W1"], d["W2"]))
    S1, S2 = ((lambda q, s: q * s)(*I.weight(_np(w))) for w in (s1, s2))
    g64, up = r.gates.astype(np.float64), _np(dy)
    _, gate_c = None, FF.gate_up_columns(cfg.Hp)

    def loss(t, x):
        total = up[t] @ (I.swiglu((x @ S1)[None])[0] @ S2)
        for k in range(cfg.K):
            e = r.topk_idx[t, k]
            total += g64[t, k] * (up[t] @ (I.swiglu((x @ W1[e])[None])[0] @ W2[e]))
        return total

    def slack(t, x, w1, w2, gate):
        """Bound of what rounding dc W2^T and then dh W1^T to 8 bits can change in dx."""
        h = (x @ w1)[None]
        _, gs = I.grad_rows(up[t][None], np.ones((1, cfg.H)))
        sw2 = np.abs(w2).max(0) / 127                                    # column scales
        half2 = 0.5 * np.abs(up[t] * sw2).max() / 127                    # half a scale of dc * sw2
        eda = gate * half2 * (np.abs(w2) / np.maximum(sw2, 1e-300)).sum(1)
        da = gate * (up[t] @ w2.T)
        da_max = np.abs(da) + eda
        # dh is linear in da; |d silu| and |silu| of h
        gcol, ucol = gate_c
        f = np.zeros((2, 2 * cfg.Hp))
        f[0, gcol] = np.abs(h[0, ucol] * FF.silu_grad(h[0, gcol]))
        f[0, ucol] = np.abs(FF.silu(h[0, gcol]))
        edh, dh_max = np.zeros(2 * cfg.Hp), np.zeros(2 * cfg.Hp)
        for c in (gcol, ucol):
            edh[c], dh_max[c] = f[0, c] * eda, f[0, c] * da_max
        sw1 = np.abs(w1).max(0) / 127
        half1 = 0.5 * (dh_max * sw1).max() / 127
        return np.abs(w1) @ edh + half1 * (np.abs(w1) / np.maximum(sw1, 1e-300)).sum(1)

    step = 2.0 ** -12
    for t in (0, 5, 11):
        bound = slack(t, xv[t], S1, S2, 1.0)
        for k in range(cfg.K):
            e = r.topk_idx[t, k]
            bound = bound + slack(t, xv[t], W1[e], W2[e], g64[t, k])
        for j in (0, 13, 63):
            hi, lo = xv[t].copy(), xv[t].copy()
            hi[j] += step
            lo[j] -= step
            diff = (loss(t, hi) - loss(t, lo)) / (2 * step)
            # the third derivative's share of a central difference, and float32 on the way
            assert abs(dx[t, j] - diff) <= bound[j] * 1.001 + 1e-4 * np.abs(dx).max(), (t, j)


def test_training_step_with_the_router():
    """Logits to logits: route, 8-bit experts, the gates' gradient and the router's backward."""
    from redundant_expert_balancing_amd.router import MoERouter
    cfg = small_cfg(name="int_router", R=2, S=32, E=8, K=2, H=128, Hp=64)
    say("int router step")
    _, d, l, _, _, _, _, dy = _ffn(cfg, 64, True)
    router = MoERouter(cfg, backward=True)
    logits = torch.randn((cfg.N, cfg.E), device="cuda", generator=torch.Generator("cuda").manual_seed(3))

    def step():
        topk, gates = router.forward(logits)
        y = l.forward(topk, d["x"], gates)
        dx = l.backward(dy, gates)
        return y, dx, router.backward(logits, l.gate_grad(dy))

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    assert all(bool(torch.isfinite(t).all()) for t in want)
    dg = _np(l.dgates)
    g64 = _np(router.gates)
    q = g64 * (dg - (g64 * dg).sum(1, keepdims=True))            # softmax, renormalised
    full = np.zeros((cfg.N, cfg.E))
    np.put_along_axis(full, router.topk_idx.cpu().numpy().astype(int), q, 1)
    mag = np.abs(g64) * (np.abs(dg) + (g64 * np.abs(dg)).sum(1, keepdims=True))
    assert (np.abs(_np(want[2]) - full) <= 16 * U * mag.max(1, keepdims=True)).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for rep in range(3):
        for t in (*out, l.act, l.z, l.da, l.dh, l.dxp):
            t.fill_(NAN)
        _ = torch.randn(4096, device="cuda").sum().item()
        g.replay()
        torch.cuda.synchronize()
        for got, ref in zip(out, want):
            assert torch.equal(got, ref), rep


def test_large_forward_is_captured_and_runs_on_another_stream():
    """A layer of many tiles, eager, replayed, and on a stream that is not the current one."""
    cfg = small_cfg(name="int_graph", R=4, S=2048, E=16, K=4, B=2, H=256, Hp=520, mode="infer")
    say("int graph")
    r, d, l, topk, gates = _layer(cfg, 2.0)
    want = l.forward(topk, d["x"], gates).clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    l.y.fill_(NAN), l.out.fill_(NAN)
    torch.cuda.synchronize()
    l.forward(topk, d["x"], gates, stream=side)
    side.synchronize()
    assert torch.equal(l.y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        l.forward(topk, d["x"], gates)
    for rep in range(3):
        l.y.fill_(NAN), l.out.fill_(NAN)
        _ = torch.randn(4096, device="cuda").sum().item()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(l.y, want), rep


def test_a_rejected_routing_writes_nothing():
    cfg = small_cfg(name="int_reject", R=2, S=16, E=8, K=2, H=128, Hp=64)
    say("int rejected")
    r, d, l, topk, gates, _, _, dy = _ffn(cfg, 0, True)
    topk = topk.clone()
    topk[3, 1] = 99
    l.z.fill_(5.0), l.dxp.fill_(5.0)
    y = l.forward(topk, d["x"], gates)
    dx = l.backward(dy, gates)
    torch.cuda.synchronize()
    assert l.error_flags(clear=True) == L.ERR_ID_RANGE
    assert not y.any() and not dx.any()
    assert bool((l.z == 5.0).all()) and bool((l.dxp == 5.0).all())
