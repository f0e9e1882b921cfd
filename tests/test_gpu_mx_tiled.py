"""The tiled form of the 4-bit grouped GEMM: sizes at which the library chooses it, against
the values that the operands' bytes stand for, in float64."""
import numpy as np
import pytest
import torch

from oracle import formats as F
from redundant_expert_balancing_amd import _lib as L
from redundant_expert_balancing_amd import mx
from redundant_expert_balancing_amd.mx import MXFFN, MXProjection
from redundant_expert_balancing_amd.synth import make_dense, make_routing

from gpu_helpers import say, small_cfg

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def is_tiled(sh):
    """The library's choice for a shape (moonep_mx_grouped_gemm)."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    nk, held = sh.R * sh.S * sh.K, sh.E + sh.R
    return nk >= 8 * held and (nk + 64 * held) // 128 * -(-sh.Hp // 256) >= cus


def _nibbles(q):
    lut = torch.tensor(np.concatenate([F.E2M1, -F.E2M1]), device="cuda")
    return torch.stack([lut[(q & 15).long()], lut[(q >> 4).long()]], -1).flatten(-2)


def _scales(s):
    v = torch.exp2(s.double() - 127)
    return torch.where(s == 255, float("nan"), v)


def rows_of(q, s, H):
    """Values of token rows."""
    v = _nibbles(q)
    C = s.shape[1] // 16
    sc = _scales(s).view(-1, C, 4, 4).transpose(2, 3).reshape(len(s), C * 16)
    return v[:, :H] * sc.repeat_interleave(32, 1)[:, :H]


def weight_of(q, s, H):
    """Values [H, Hp] of one expert's weight."""
    n16, T, C = q.shape[0], q.shape[1], s.shape[1]
    v = _nibbles(q.view(n16, T, 4, 16, 16)).permute(1, 2, 4, 0, 3).reshape(T * 128, n16 * 16)
    sc = _scales(s).view(n16, C, 4, 16, 4).permute(1, 4, 2, 0, 3).reshape(C * 16, n16 * 16)
    return v[:H] * sc.repeat_interleave(32, 0)[:H]


def test_decoders_match_the_oracle():
    say("mx decoders")
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 608)) * 2.0 ** rng.integers(-3, 4, (5, 608))
    q, s = F.mx(x)
    a, b = F.mx_pack_rows(q, s)
    got = rows_of(torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda(), 608)
    assert np.array_equal(got.cpu().numpy(), F.mx_values(q, s))
    w = rng.standard_normal((48, 608))
    q, s = F.mx(w)
    a, b = F.mx_pack_weight(q, s)
    got = weight_of(torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda(), 608)
    assert np.array_equal(got.cpu().numpy(), F.mx_values(q, s).T)


class Call:
    """One rank, E experts, N tokens of K slots; cu_seqlens of the given segment lengths."""

    def __init__(self, N, K, E, H, Hp, lengths, dtype="bf16", seed=0, B=0):
        self.N, self.K, self.E, self.H, self.Hp = N, K, E, H, Hp
        self.sh = L.Shape(1, N, E, K, B, H, Hp, L.INFER, L.BF16 if dtype == "bf16" else L.FP32)
        assert is_tiled(self.sh)
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.x = torch.randn((N, H), generator=g, device="cuda").to(dt)
        self.w = torch.randn((E, H, Hp), generator=g, device="cuda").to(dt)
        self.xq, self.xs = mx.buffers(N, H)
        self.wq, self.wsc = mx.weight_buffers(E, H, Hp)
        for t in (self.xq, self.xs, self.wq, self.wsc):
            t.fill_(0xFF)
        cu = np.concatenate([[0], np.cumsum(lengths)])
        assert len(lengths) == E + B and cu[-1] <= N * K
        self.lengths, self.end = lengths, int(cu[-1])
        self.cu = torch.tensor(cu[None], dtype=torch.int32, device="cuda")
        self.src = torch.randperm(N * K, generator=g, device="cuda").int()
        self.ws = torch.empty(L.moonep_workspace_bytes(self.sh) // 4, dtype=torch.int32, device="cuda")
        L.moonep_workspace_init(self.sh, self.ws)
        self.quantise()

    def quantise(self):
        L.moonep_mx_quantize(self.sh, self.N, self.H, self.x, self.xq, self.xs)
        L.moonep_mx_quantize_weight(self.sh, self.w, self.wq, self.wsc)

    def out(self):
        return torch.full((self.N * self.K, self.Hp), 7.0, device="cuda")

    def gemm(self, c, src="src", xq=None, xs=None):
        src = self.src if isinstance(src, str) else src
        L.moonep_mx_grouped_gemm(self.sh, self.xq if xq is None else xq, self.xs if xs is None else xs,
                                 src, self.wq, self.wsc, self.cu, c, self.ws)
        return c

    def check(self, c, src):
        """c against the float64 products of the stored values; src: position -> slot."""
        xv = rows_of(self.xq, self.xs, self.H)
        at = 0
        for e, n in enumerate(self.lengths):
            if n:
                u = src[at:at + n].long()
                ok = (u >= 0) & (u < self.N * self.K)
                a = xv[torch.where(ok, u, 0) // self.K] * ok[:, None]
                w = weight_of(self.wq[e], self.wsc[e], self.H)
                want, mag = a @ w, a.abs() @ w.abs()
                # exact products; a float32 sum of H of them is off by at most H roundings of
                # the magnitudes' sum, and each of H products and sums by 2^-126 more where it lies
                # below float32's normal range (products of 1e-37 and 2^-40 do)
                err = (c[at:at + n].double() - want).abs()
                assert bool((err <= self.H * U * mag + 2 * self.H * 2.0 ** -126).all()), (e, n)
            at += n
        assert bool((c[at:] == 7.0).all())          # behind the last segment


# rows of 1, 127, 128 and 129, none, and long ones; the last positions belong to no segment
LENGTHS = [1, 127, 0, 128, 129, 9000, 3500, 3100]


@pytest.mark.parametrize("H,Hp", [(64, 512), (128, 320), (192, 512), (320, 1088), (512, 576), (576, 320),
                                  (1408, 448)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gathered_rows(H, Hp, dtype):
    """One k-tile, odd numbers of k-tiles and of steps, partial k-chunks, partial column tiles."""
    say("mx tiled gathered", H, Hp, dtype)
    c = Call(2000, 8, 8, H, Hp, LENGTHS, dtype, seed=H)
    c.check(c.gemm(c.out()), c.src)


@pytest.mark.parametrize("H,Hp", [(64, 512), (192, 320), (576, 512), (1408, 320)])
def test_rows_in_place(H, Hp):
    """src_index NULL: bit for bit what the identity gather gives on the same rows."""
    say("mx tiled in place", H, Hp)
    c = Call(16000, 1, 8, H, Hp, LENGTHS, seed=H)
    ident = torch.arange(c.N, dtype=torch.int32, device="cuda")
    a, b = c.gemm(c.out(), None), c.gemm(c.out(), ident)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    c.check(a, ident)


def test_bad_positions_and_nan_tokens():
    """Positions that name no slot give zeros; a NaN token is NaN in its own rows alone, also
    where the next row of values is read behind an odd number of k-tiles."""
    say("mx tiled bad positions")
    c = Call(2000, 8, 8, 192, 320, LENGTHS)
    c.x[5, 3] = float("nan")
    c.x[1999, 191] = float("inf")
    c.quantise()
    src = c.src.clone()
    src[0], src[77], src[128], src[9000], src[9001] = -1, c.N * c.K, 2 ** 31 - 1, -2 ** 31, -7
    got = c.gemm(c.out(), src)
    torch.cuda.synchronize()
    ok = (src >= 0) & (src < c.N * c.K)
    assert not got[:c.end][~ok[:c.end]].any()
    tok = torch.where(ok, src // c.K, -1)[:c.end]
    bad = (tok == 5) | (tok == 1999)
    assert bool(torch.isnan(got[:c.end][bad]).all()) and int(bad.sum()) > 0
    assert bool(torch.isfinite(got[:c.end][~bad]).all())
    clean = torch.where((src // c.K == 5) | (src // c.K == 1999), -1, src)
    again = c.gemm(c.out(), clean)
    torch.cuda.synchronize()
    assert torch.equal(again[:c.end][~bad], got[:c.end][~bad])
    c.x[5, 3] = 0.0
    c.x[1999, 191] = 0.0
    c.quantise()
    c.check(c.gemm(c.out(), clean), clean)


@pytest.mark.parametrize("tiled", [True, False])
def test_values_at_the_ends_of_the_range(tiled):
    """Rows of float32's largest and smallest values against weights of ordinary ones."""
    say("mx range ends", tiled)
    N, K, H, Hp, E = 2000, 8, 192, 512, 8
    c = Call(N, K, E, H, Hp, LENGTHS, "fp32")
    big = float(torch.finfo(torch.float32).max)
    c.x[0] = big
    c.x[1] = -big
    c.x[2] *= 1e-37
    c.x[3] = 0.0
    c.w *= 2.0 ** -40
    c.quantise()
    if not tiled:                       # the same rows, few at a time
        c.sh = L.Shape(1, 8, E, 1, 0, H, Hp, L.INFER, L.FP32)
        assert not is_tiled(c.sh)
        c.N, c.K, c.lengths = 8, 1, [1, 2, 0, 1, 1, 1, 1, 1]
        c.cu = torch.tensor([[0, 1, 3, 3, 4, 5, 6, 7, 8]], dtype=torch.int32, device="cuda")
        c.src = torch.tensor([0, 1, 2, 3, 1, 0, 2, 4], dtype=torch.int32, device="cuda")
    c.check(c.gemm(c.out()), c.src)


def _routing(cfg, alpha, seed=0):
    r = make_routing(cfg, 3.0, seed=seed, alpha=alpha)
    return torch.from_numpy(r.topk_idx).cuda(), torch.from_numpy(r.gates).cuda()


def _positions(l, cfg):
    """(weight row, first, last) of every segment with rows, in buffer positions."""
    cu, SK = l.cu_seqlens.cpu().numpy(), cfg.S * cfg.K
    for q in range(cfg.R):
        for i in range(cfg.E + cfg.B):
            if cu[q, i] < cu[q, i + 1]:
                yield i if i < cfg.E else cfg.E + q * cfg.B + i - cfg.E, q * SK + cu[q, i], q * SK + cu[q, i + 1]


def test_ffn_and_its_graph():
    """Plan, prefetch, both products (gathered, then in place), replayed for new tokens."""
    cfg = small_cfg(name="mx_tiled_ffn", R=2, S=2048, E=8, K=4, B=2, H=576, Hp=320, mode="infer")
    say("mx tiled ffn")
    d = make_dense(cfg, "cuda", 0, which=("x", "W1", "W2"))
    l = MXFFN(cfg)
    assert is_tiled(l.up) and is_tiled(l.down)
    for t in (l.w1q, l.w1s, l.w2q, l.w2s):
        t.fill_(0xFF)
    l.quantise_weights(d["W1"], d["W2"])
    topk, gates = _routing(cfg, 2.0)
    x = d["x"].clone()
    l.forward(topk, x, gates)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        l.forward(topk, x, gates)
    gen = torch.Generator(device="cuda").manual_seed(3)
    for rep in range(4):
        ids, w = _routing(cfg, 1.0 + rep, seed=rep)
        topk.copy_(ids), gates.copy_(w)
        x.copy_(torch.randn(x.shape, generator=gen, device="cuda").to(x.dtype))
        for t in (l.h, l.z, l.y):
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        xv, av = rows_of(l.xq, l.xs, cfg.H), rows_of(l.aq, l.as_, cfg.Hp)
        tok = l.src_index.long() // cfg.K
        for row, a, b in _positions(l, cfg):
            for got, v, wq, ws in ((l.h, xv[tok[a:b]], l.w1q, l.w1s), (l.z, av[a:b], l.w2q, l.w2s)):
                wv = weight_of(wq[row], ws[row], v.shape[1])
                err = (got[a:b].double() - v @ wv).abs()
                assert bool((err <= v.shape[1] * U * (v.abs() @ wv.abs())).all()), (rep, row)
        kept = [t.clone() for t in (l.h, l.z, l.y)]
        l.forward(topk, x, gates)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, (l.h, l.z, l.y))), rep


def test_prefetched_experts_are_read():
    """A skewed routing on four ranks: segments of prefetched experts are those of the home rows."""
    cfg = small_cfg(name="mx_tiled_pre", R=4, S=1024, E=16, K=4, B=4, H=320, Hp=512, mode="infer")
    say("mx tiled prefetch")
    d = make_dense(cfg, "cuda", 0, which=("x", "W"))
    l = MXProjection(cfg)
    assert is_tiled(l.shape)
    l.wq.fill_(0xFF), l.wscales.fill_(0xFF)
    l.quantise_weights(d["W"])
    topk, gates = _routing(cfg, 2.5)
    l.forward(topk, d["x"], gates)
    torch.cuda.synchronize()
    xv, tok = rows_of(l.xq, l.xs, cfg.H), l.src_index.long() // cfg.K
    used = l.replica_expert.cpu().numpy()
    assert (used >= 0).any()
    for row, a, b in _positions(l, cfg):
        home = row if row < cfg.E else int(used.reshape(-1)[row - cfg.E])
        assert bool((topk.reshape(-1)[l.src_index[a:b].long()] == home).all())
        v, wv = xv[tok[a:b]], weight_of(l.wq[home], l.wscales[home], cfg.H)
        assert bool(((l.out[a:b].double() - v @ wv).abs() <= cfg.H * U * (v.abs() @ wv.abs())).all()), row


def test_outputs_wider_than_a_tile_s_offsets():
    """128 rows of H' floats that pass 2^31 bytes are left to the few-row form."""
    say("mx wide outputs")
    N, H, Hp = 128, 64, 4227392                    # 127 * 4 * H' is beyond 2^31
    sh = L.Shape(1, N, 1, 1, 0, H, Hp, L.INFER, L.BF16)
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((N, H), generator=g, device="cuda").bfloat16()
    w = torch.randn((1, H, Hp), generator=g, device="cuda", dtype=torch.float32).bfloat16()
    xq, xs = mx.buffers(N, H)
    wq, wsc = mx.weight_buffers(1, H, Hp)
    ws = torch.empty(L.moonep_workspace_bytes(sh) // 4, dtype=torch.int32, device="cuda")
    L.moonep_workspace_init(sh, ws)
    L.moonep_mx_quantize(sh, N, H, x, xq, xs)
    L.moonep_mx_quantize_weight(sh, w, wq, wsc)
    c = torch.full((N, Hp), float("nan"), device="cuda")
    L.moonep_mx_grouped_gemm(sh, xq, xs, None, wq, wsc,
                             torch.tensor([[0, N]], dtype=torch.int32, device="cuda"), c, ws)
    torch.cuda.synchronize()
    xv = rows_of(xq, xs, H)
    for n0 in (0, Hp - 4096):                      # the first columns and the last
        tiles = slice(n0 // 16, n0 // 16 + 256)
        wv = weight_of(wq[0][tiles], wsc[0][tiles], H)
        err = (c[:, n0:n0 + 4096].double() - xv @ wv).abs()
        assert bool((err <= H * U * (xv.abs() @ wv.abs())).all()), n0
    assert bool(torch.isfinite(c).all())
