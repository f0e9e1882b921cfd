"""8-bit integer experts at the sizes where the rounding of gradient rows walks several positions
in a row and where its output passes the caches: stored bytes against the definition in 64 bits.

A workgroup's share is min(16, slots / 8192) positions, so it is more than one from 16384 slots
on; outputs above 256 MiB are stored past the caches.
"""
import numpy as np
import pytest
import torch

from oracle import int8 as I
from redundant_expert_balancing_amd import _lib as L
from redundant_expert_balancing_amd import int8

from gpu_helpers import say

pytestmark = pytest.mark.gpu
NAN = float("nan")


def _dt(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _rows(g):
    """(whole values, scales) of float32 rows g, as oracle.int8.rows defines them."""
    bad = ~torch.isfinite(g).all(1)
    v = torch.where(bad[:, None], 0.0, g).double()
    scale = (v.abs().amax(1) / 127.0).clamp_min(I.LEAST).float()
    q = torch.round(v / scale.double()[:, None])
    return q, torch.where(bad, NAN, scale)


def test_this_reference_is_the_oracle():
    g = torch.randn((37, 24), generator=torch.Generator().manual_seed(0)) * 2.0 ** 3
    g[3], g[4, 5], g[5, 1] = 0.0, NAN, float("inf")
    g[6] *= 2.0 ** -140
    q, s = _rows(g.cuda())
    want_q, want_s = I.rows(g.double().numpy())
    assert np.array_equal(q.cpu().numpy(), want_q)
    assert np.array_equal(s.cpu().numpy(), want_s.astype(np.float32), equal_nan=True)


def _view(rng, R, E, SK, ahead, behind):
    """cu_seqlens of R ranks: rows of random lengths, some empty, some shorter than a share; `ahead`
    positions ahead of the first row of every odd rank, `behind` behind the last of every rank."""
    EB = E + E // R
    cu = np.zeros((R, EB + 1), int)
    for q in range(R):
        first = ahead if q % 2 else 0
        share = rng.random(EB) ** 3 * (rng.random(EB) > 0.25)
        lens = np.floor(share / share.sum() * (SK - first - behind)).astype(int)
        lens[rng.integers(EB)] += SK - first - behind - lens.sum()
        cu[q] = first + np.concatenate([[0], np.cumsum(lens)])
    return cu


def _check(R, S, E, K, Hp, dtype, ahead, behind, chunk, past=False):
    say("int gradient rows, long", R, S, E, K, Hp, dtype, "share", chunk, "past the caches", past)
    N, SK, NK, EB = R * S, S * K, R * S * K, E + E // R
    width = L.int_row_bytes(Hp)
    assert max(1, min(16, NK // 8192)) == chunk and (NK * width > 1 << 28) == past
    rng = np.random.default_rng(NK)
    gen = torch.Generator("cuda").manual_seed(NK)
    sh = L.Shape(R, S, E, K, E // R, 64, Hp, L.TRAIN, L.BF16 if dtype == "bf16" else L.FP32)
    cols = 16 * -(-Hp // 16)
    wsc = torch.rand((2 * E, cols), device="cuda", generator=gen) + 0.5
    cu = _view(rng, R, E, SK, ahead, behind)
    wrow = np.full(NK, -1)
    for q in range(R):
        for i in range(EB):
            wrow[q * SK + cu[q, i]:q * SK + cu[q, i + 1]] = i if i < E else E + q * (E // R) + i - E
    src = rng.permutation(NK)
    src[rng.integers(0, NK, 40)] = -1                 # all over the shares
    src[rng.integers(0, NK, 40)] = NK
    src[NK - 1] = -7
    i32 = dict(dtype=torch.int32, device="cuda")
    cu_t, src_t = torch.tensor(cu, **i32), torch.tensor(src, **i32)
    wrow, at = torch.from_numpy(wrow).cuda(), src_t.long()
    there = (at >= 0) & (at < NK)
    at = torch.where(there, at, 0)
    gates = torch.rand((N, K), device="cuda", generator=gen)
    dy = torch.randn((N, Hp), device="cuda", generator=gen).to(_dt(dtype))
    dy[1, 0], dy[N // 2, Hp - 1] = NAN, float("inf")
    q, s = int8.buffers(NK, Hp)
    every = torch.ones(NK, dtype=torch.bool, device="cuda")

    def check(rows_of, gate, there, wrow):
        for lo in range(0, NK, 8192):
            p = slice(lo, min(lo + 8192, NK))
            live = wrow[p] >= 0
            g = (rows_of(p).double() * wsc[wrow[p].clamp_min(0), :Hp].double()).float()
            want_q, want_s = _rows(torch.where(there[p][:, None], g, 0.0))
            want_s = torch.where(there[p], want_s * gate[p], 0.0)
            assert torch.equal(q[p, :Hp][live].double(), want_q[live]), lo
            assert not q[p, Hp:][live].any(), lo
            assert torch.equal(torch.nan_to_num(s[p][live], nan=-1.0),
                               torch.nan_to_num(want_s[live], nan=-1.0)), lo
            assert bool((q[p][~live] == -86).all()) and bool(torch.isnan(s[p][~live]).all()), lo

    def run(*args):
        q.fill_(-86), s.fill_(NAN)
        L.moonep_int_quantize_grad(sh, *args, q, s)
        torch.cuda.synchronize()

    one = torch.ones(NK, device="cuda")
    run(dy, src_t, gates, wsc, cu_t)
    check(lambda p: dy[at[p] // K], gates.reshape(-1)[at], there, wrow)
    run(dy, src_t, None, wsc, cu_t)
    check(lambda p: dy[at[p] // K], one, there, wrow)
    dh = torch.randn((NK, Hp), device="cuda", generator=gen).to(_dt(dtype))
    run(dh, None, None, wsc, cu_t)
    check(lambda p: dh[p], one, every, wrow)
    run(dh, None, None, wsc, None)                    # one weight for all
    check(lambda p: dh[p], one, every, torch.zeros_like(wrow))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("R,S,E,K,Hp,chunk", [
    (4, 1027, 16, 4, 8, 2),
    (4, 1401, 8, 3, 1000, 2),             # one wavefront, two (bfloat16) or four vectors a lane
    (2, 2731, 8, 3, 1408, 2),
    (1, 50001, 4, 1, 72, 6),
    (4, 10931, 16, 3, 72, 16),            # ranks end inside a share, and the last share is short
    (2, 2051, 8, 4, 2056, 2),             # rows shared by four wavefronts
    (2, 2051, 8, 4, 4104, 2),
    (2, 2051, 8, 4, 8200, 2),             # by sixteen
])
def test_gradient_rows_over_several_positions(R, S, E, K, Hp, chunk, dtype):
    _check(R, S, E, K, Hp, dtype, ahead=7, behind=5, chunk=chunk)


@pytest.mark.parametrize("R,S,E,K,Hp,dtype,chunk", [
    (4, 10931, 16, 3, 2048, "bf16", 16),
    (4, 10931, 16, 3, 2048, "fp32", 16),
    (2, 4099, 8, 2, 16392, "fp32", 2),    # rows too wide to be held
    (2, 4099, 8, 2, 32776, "bf16", 2),
])
def test_gradient_rows_past_the_caches(R, S, E, K, Hp, dtype, chunk):
    _check(R, S, E, K, Hp, dtype, ahead=9, behind=3, chunk=chunk, past=True)


@pytest.mark.parametrize("ahead", [1, 501, 1000])
def test_a_share_that_begins_ahead_of_the_first_row(ahead):
    """Its positions ahead of the rank's first row are left as they were, its others and the rest of
    the rank are not."""
    say("int gradient rows ahead, long", ahead)
    R, S, E, K, Hp = 2, 16501, 4, 4, 40
    NK, SK = R * S * K, S * K
    assert NK // 8192 >= 16
    gen = torch.Generator("cuda").manual_seed(ahead)
    sh = L.Shape(R, S, E, K, E // R, 64, Hp, L.TRAIN, L.BF16)
    dh = torch.randn((NK, Hp), device="cuda", generator=gen).bfloat16()
    wsc = torch.ones((2 * E, 48), device="cuda")
    cu = [[ahead, ahead, ahead + 3, 20000, 20000, 40000, SK]] * R
    q0, s0 = int8.buffers(NK, Hp)
    q, s = int8.buffers(NK, Hp)
    q.fill_(-86), s.fill_(NAN)
    L.moonep_int_quantize(sh, NK, Hp, dh, q0, s0)      # scales of one: the same rows
    L.moonep_int_quantize_grad(sh, dh, None, None, wsc, torch.tensor(cu, dtype=torch.int32, device="cuda"), q, s)
    torch.cuda.synchronize()
    out = torch.arange(NK, device="cuda") % SK < ahead
    assert torch.equal(q[~out], q0[~out]) and torch.equal(s[~out], s0[~out])
    assert bool((q[out] == -86).all()) and bool(torch.isnan(s[out]).all())
