"""Every form of the 8-bit integer products on the calls that take it: gathered and in place, with
the SwiGLU in the epilogue and without, dense and grouped, a layer's backward pass, one expert
with nearly all rows, and token rows beyond 2 GiB.

Which form a call takes is computed here as int_product (csrc/int8.hip) chooses it for 256
compute units, so that a case cannot silently move to another form.
"""
import numpy as np
import pytest
import torch

from oracle import int8 as I
from redundant_expert_balancing_amd import _lib as L
from redundant_expert_balancing_amd import int8

from gpu_helpers import say, small_cfg

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TINY = 1e-37
NAN = float("nan")


def _form(NK, segs, H, W, dense=False):
    """Rows of the tiles, or 0 for the form for few rows; segs: E + R, 1 of a dense product."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    NB, KB = -(-W // 16), 2 * -(-H // 128)
    each = -(-NK // segs)
    if each <= (32 if dense else 8):
        return 0
    if segs * ((NB + 1) // 2) * -(-each // 64) <= 4 * cus and KB * -(-each // 16) <= 96:
        return 0

    def tiles(bt):
        return -(-(NK + bt // 2 * segs) // bt) * -(-W // bt)
    if NK >= 64 * segs and tiles(256) > cus // 2:
        return 256
    return 128 if tiles(128) > cus // 2 else 64


def _dt(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _shape(H, Hp, dtype, N, E, K):
    return L.Shape(1, N, E, K, 0, H, Hp, L.INFER, L.BF16 if dtype == "bf16" else L.FP32)


def _operands(H, W, N, E, K, dtype, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    spread = torch.exp2(torch.randint(-3, 3, (W,), device="cuda", generator=gen).float())
    x = torch.randn((N, H), device="cuda", generator=gen).to(_dt(dtype))
    w = (torch.randn((E, H, W), device="cuda", generator=gen) * H ** -0.5 * spread).to(_dt(dtype))
    sh = _shape(H, W, dtype, N, E, K)
    xq, xs = int8.buffers(N, H)
    wq, ws = int8.weight_buffers(E, H, W)
    L.moonep_int_quantize(sh, N, H, x, xq, xs)
    L.moonep_int_quantize_weight(sh, w, wq, ws)
    work = torch.empty(L.moonep_workspace_bytes(sh) // 4, dtype=torch.int32, device="cuda")
    L.moonep_workspace_init(sh, work)
    return sh, x, w, xq, xs, wq, ws, work


def _plan(NK, E, seed):
    """Positions of NK slots over E experts (one of them empty), the last two behind the last row, and
    a random order of slots with three bad entries."""
    rng = np.random.default_rng(seed)
    cut = np.sort(rng.integers(0, NK - 1, E - 2)).tolist() if E > 1 else []
    cu = [0] + cut + [NK - 2] * (2 if E > 1 else 1)
    src = rng.permutation(NK)
    src[[1, NK // 2, NK - 3]] = [-1, NK, -(2 ** 31)]
    i32 = dict(dtype=torch.int32, device="cuda")
    return cu, torch.tensor([cu], **i32), torch.from_numpy(src.astype(np.int64)).cuda().int()


def _same_act(got, want, h, dtype):
    """float32: the same bits. bfloat16: a step where the float32 values lie on two sides of a
    border (2^-7 of the value), and |gate * up| * 2^-126 where 1 / (1 + e^-gate) is below the
    normal numbers."""
    if dtype == "fp32":
        assert torch.equal(got, want)
        return
    v = h.double().view(h.shape[0], -1, 2, 32)
    low = (v[:, :, 0] * v[:, :, 1]).abs().reshape(h.shape[0], -1) * 2.0 ** -126
    d, w = (got.double() - want.double()).abs(), want.double().abs()
    assert bool((d <= 2.0 ** -7 * w + low + TINY).all())


GROUPED = [
    # N, K, E, H, H', form of the gate/up product [H, 2H']
    (13, 3, 7, 264, 96, 0),
    (50, 2, 4, 3200, 96, 64),            # 25 steps of 128: the two groups take 13 and 12
    (53, 3, 4, 4096, 160, 64),
    (170, 2, 16, 192, 1248, 128),
    (115, 3, 16, 1000, 1312, 128),
    (2400, 2, 4, 136, 800, 256),
    (3001, 3, 8, 72, 544, 256),          # one step
    (1700, 4, 16, 520, 480, 256),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,K,E,H,Hp,form", GROUPED)
def test_gathered_products(N, K, E, H, Hp, form, dtype):
    """The gate/up product with its SwiGLU, gathered by src_index with K slots a token, against the
    product and moonep_swiglu, and both against float64 on whole numbers."""
    NK, W = N * K, 2 * Hp
    assert _form(NK, E + 1, H, W) == form
    say("int gathered", N, K, E, H, Hp, dtype, "form", form)
    sh, x, w, xq, xs, wq, ws, work = _operands(H, W, N, E, K, dtype, N)
    ffn = _shape(H, Hp, dtype, N, E, K)
    cu, cu_t, src = _plan(NK, E, N)
    end = cu[-1]
    new = lambda n, dt=_dt(dtype): torch.full((NK, n), NAN, device="cuda", dtype=dt)     # noqa: E731
    c, a0, h0, a1, h1, a2 = new(W, torch.float32), new(Hp), new(W), new(Hp), new(W), new(Hp)
    L.moonep_int_grouped_gemm(sh, xq, xs, src, wq, ws, cu_t, c, work)
    L.moonep_swiglu(ffn, c, a0, h0)
    L.moonep_int_grouped_gemm_swiglu(ffn, xq, xs, src, wq, ws, cu_t, a1, h1, work)
    L.moonep_int_grouped_gemm_swiglu(ffn, xq, xs, src, wq, ws, cu_t, a2, None, work)
    torch.cuda.synchronize()
    assert torch.equal(h1[:end], h0[:end]) and torch.equal(a1[:end], a2[:end])
    _same_act(a1[:end], a0[:end], c[:end], dtype)
    for t in (c, a1, h1, a2):            # behind the last row
        assert bool(torch.isnan(t[end:]).all())
    qx, sx = (torch.from_numpy(a).cuda() for a in I.rows(x.double().cpu().numpy()))
    at = src[:end].long()
    there = (at >= 0) & (at < NK)
    tok = torch.where(there, at, 0) // K
    for e in range(E):
        lo, hi = cu[e], cu[e + 1]
        if lo == hi:
            continue
        qw, sw = (torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in I.weight(w[e].double().cpu().numpy()))
        want = (qx[tok[lo:hi]] @ qw) * sx[tok[lo:hi], None] * sw
        want = torch.where(there[lo:hi, None], want, 0.0)
        assert bool(((c[lo:hi].double() - want).abs() <= 3.01 * U * want.abs() + TINY).all()), e
    # rows in place: the same bits from a copy of each position's row
    pos_q, pos_s = xq[tok], xs[tok]
    pos_q[~there] = 0
    more = torch.zeros((2, xq.shape[1]), dtype=torch.int8, device="cuda")
    pos_q = torch.cat([pos_q, more])
    pos_s = torch.cat([pos_s, torch.zeros(2, device="cuda")])
    d, a3, h3 = new(W, torch.float32), new(Hp), new(W)
    L.moonep_int_grouped_gemm(sh, pos_q, pos_s, None, wq, ws, cu_t, d, work)
    L.moonep_int_grouped_gemm_swiglu(ffn, pos_q, pos_s, None, wq, ws, cu_t, a3, h3, work)
    torch.cuda.synchronize()
    assert torch.equal(c[:end], d[:end]) and torch.equal(h3[:end], h1[:end]) and torch.equal(a3[:end], a1[:end])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,H,Hp,form", [
    (31, 520, 96, 0),
    (100, 1000, 96, 64),
    (97, 3200, 352, 64),
    (800, 128, 96, 64),                  # one step: the second group has none
    (1000, 136, 1024, 128),
    (1031, 1000, 1056, 128),
    (4100, 64, 1056, 256),
])
def test_dense_products(rows, H, Hp, form, dtype):
    W = 2 * Hp
    assert _form(rows, 1, H, W, dense=True) == form
    say("int dense forms", rows, H, Hp, dtype, "form", form)
    sh, x, w, xq, xs, wq, ws, _ = _operands(H, W, rows, 1, 1, dtype, rows)
    ffn = _shape(H, Hp, dtype, rows, 1, 1)
    new = lambda n, dt=_dt(dtype): torch.full((rows + 2, n), NAN, device="cuda", dtype=dt)     # noqa: E731
    c, d, a0, h0, a1, h1, a2 = (new(W, torch.float32), new(W, torch.float32), new(Hp), new(W), new(Hp), new(W),
                                new(Hp))
    add = torch.randn((rows, W), device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    L.moonep_int_gemm(sh, rows, xq, xs, wq, ws, None, c)
    L.moonep_int_gemm(sh, rows, xq, xs, wq, ws, add, d)
    L.moonep_swiglu(ffn, c, a0, h0)
    L.moonep_int_gemm_swiglu(ffn, rows, xq, xs, wq, ws, a1, h1)
    L.moonep_int_gemm_swiglu(ffn, rows, xq, xs, wq, ws, a2, None)
    torch.cuda.synchronize()
    want = I.product(*I.rows(x.double().cpu().numpy()), *I.weight(w[0].double().cpu().numpy()))
    got = c[:rows].double().cpu().numpy()
    assert (np.abs(got - want) <= 3.01 * U * np.abs(want) + TINY).all()
    assert torch.equal(d[:rows], c[:rows] + add)
    assert torch.equal(h1[:rows], h0[:rows]) and torch.equal(a1[:rows], a2[:rows])
    _same_act(a1[:rows], a0[:rows], c[:rows], dtype)
    for t in (c, d, a1, h1, a2):
        assert bool(torch.isnan(t[rows:]).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_backward_of_a_layer_on_large_tiles(dtype):
    """A training layer with a shared expert whose products, forward and back, take 256-row tiles,
    and whose gradient rows are walked two positions at a time."""
    from test_gpu_int8 import _check_ffn
    cfg = small_cfg(name="int_back", R=2, S=4100, E=8, K=2, H=520, Hp=544, dtype=dtype)
    NK = cfg.N * cfg.K
    assert NK // 8192 == 2
    for h, w in ((520, 1088), (544, 520), (520, 544), (1088, 520)):
        assert _form(NK, cfg.E + cfg.R, h, w) == 256
    _check_ffn(cfg, 512, True)


def test_one_expert_with_nearly_all_rows():
    """Few rows per expert on average, so the form for few rows, and hundreds in one of them."""
    N, K, E, H, Hp = 300, 4, 256, 264, 96
    NK, W = N * K, 2 * Hp
    assert _form(NK, E + 1, H, W) == 0
    say("int one expert")
    sh, x, w, xq, xs, wq, ws, work = _operands(H, W, N, E, K, "bf16", 5)
    lens = np.zeros(E, int)
    lens[[0, 3, 17, 255]] = [2, 1, NK - 7, 4]
    cu = np.concatenate([[0], np.cumsum(lens)])
    cu_t = torch.from_numpy(cu[None]).cuda().int()
    src = torch.from_numpy(np.random.default_rng(1).permutation(NK)).cuda().int()
    c = torch.full((NK, W), NAN, device="cuda")
    L.moonep_int_grouped_gemm(sh, xq, xs, src, wq, ws, cu_t, c, work)
    torch.cuda.synchronize()
    qx, sx = I.rows(x.double().cpu().numpy())
    tok = src.cpu().numpy() // K
    got = c.double().cpu().numpy()
    for e in (0, 3, 17, 255):
        at = slice(cu[e], cu[e + 1])
        want = I.product(qx[tok[at]], sx[tok[at]], *I.weight(w[e].double().cpu().numpy()))
        assert (np.abs(got[at] - want) <= 3.01 * U * np.abs(want) + TINY).all(), e


def test_token_rows_beyond_32_bit_offsets():
    """More than 2 GiB of gathered token rows take the form for few rows, whatever their number:
    rows at both ends and on either side of 2^31 bytes, against the same rows alone."""
    N, H, Hp, E = 16400, 131072, 32, 2
    W = 2 * Hp
    assert N * H > 1 << 31
    say("int beyond 2 GiB")
    sh, ffn = _shape(H, W, "fp32", N, E, 1), _shape(H, Hp, "fp32", N, E, 1)
    gen = torch.Generator("cuda").manual_seed(0)
    xq = torch.randint(-127, 128, (N, H), dtype=torch.int8, device="cuda", generator=gen)
    xs = torch.rand(N, device="cuda", generator=gen) * 2.0 ** -20
    wq, ws = int8.weight_buffers(E, H, W)
    wq.random_(-127, 128, generator=gen)
    ws.uniform_(0.5, 1.0, generator=gen)
    work = torch.empty(L.moonep_workspace_bytes(sh) // 4, dtype=torch.int32, device="cuda")
    L.moonep_workspace_init(sh, work)
    src = torch.randperm(N, device="cuda", generator=gen).int()
    cut = 9001
    cu = torch.tensor([[0, cut, N]], dtype=torch.int32, device="cuda")
    c, act = torch.full((N, W), NAN, device="cuda"), torch.full((N, Hp), NAN, device="cuda")
    h, act0 = torch.empty_like(c), torch.empty_like(act)
    L.moonep_int_grouped_gemm(sh, xq, xs, src, wq, ws, cu, c, work)
    L.moonep_int_grouped_gemm_swiglu(ffn, xq, xs, src, wq, ws, cu, act, h, work)
    L.moonep_swiglu(ffn, c, act0, None)
    torch.cuda.synchronize()
    assert torch.equal(h, c) and torch.equal(act, act0)
    # each weight over its own positions' rows, 2048 of them at a time
    for e, (lo, hi) in enumerate(((0, cut), (cut, N))):
        q = wq[e].view(W // 16, H // 64, 4, 16, 16).permute(1, 2, 4, 0, 3).reshape(H, W).double()
        for p in range(lo, hi, 2048):
            at = src[p:min(p + 2048, hi)].long()
            want = (xq[at].double() @ q) * xs[at].double()[:, None] * ws[e].double()
            got = c[p:min(p + 2048, hi)].double()
            assert bool(((got - want).abs() <= 3.01 * U * want.abs() + TINY).all()), (e, p)


@pytest.mark.parametrize("rows", [3, 300])
def test_the_longest_sums_are_exact(rows):
    """A reduction of 131072 whole numbers of the largest magnitude, -128 (which quantisation never
    writes) in one of the operands: 127 * 128 * 131072 < 2^31."""
    H, W = 131072, 16
    say("int longest sums", rows)
    sh = _shape(H, W, "fp32", rows, 1, 1)
    xq = torch.full((rows, H), 127, dtype=torch.int8, device="cuda")
    xq[1] = -127
    xs = torch.ones(rows, device="cuda")
    wq, _ = int8.weight_buffers(1, H, W)
    wq.fill_(-128)
    wq.view(H // 64, 64, 16)[:, 16:32] = 127            # a quarter of the k of every column
    c = torch.full((rows, W), NAN, device="cuda")
    L.moonep_int_gemm(sh, rows, xq, xs, wq, None, None, c)
    torch.cuda.synchronize()
    want = torch.full((rows, W), 127 * (127 - 3 * 128) * (H // 4), dtype=torch.float64).float().cuda()
    want[1] *= -1
    assert torch.equal(c, want)
    wq.fill_(-128)
    L.moonep_int_gemm(sh, rows, xq, xs, wq, None, None, c)
    torch.cuda.synchronize()
    want.fill_(float(np.float32(-127 * 128 * H)))
    want[1] *= -1
    assert torch.equal(c, want)
