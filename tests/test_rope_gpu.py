"""dsa_qk_norm_rope on the GPU against its formula in 64 bits.

Tolerances.  A result is formed in fp32 and rounded once.  Relative to the pair
(a, b) a rotated value is made of, the fp32 error is at most 64 half steps of
2^-24: the sum of squares adds at most 1024 / 8 = 128 terms one after another
in a lane and three joins, each a rounding of a positive partial sum, and the
root halves their sum (<= 66 for 1024 elements, 38 for 576); the mean, root,
reciprocal, two products, the cosine (about two), its angle (pi * 2^-24 after the
reduction) and the two products and one sum of the rotation add about ten.  So 80
half steps of the pair bound it for every row length, and rounding to bf16 adds
half a step of the value."""
import math

import numpy as np
import pytest
import torch

import indexer_top_sparse_lightning_b200 as dsa
from tests.paged_helpers import EPS32, HALF_BF16, PAGE, ROW, Paged, assert_status_ok, randn

pytestmark = pytest.mark.gpu

FP32 = 80 * EPS32


def _freq(R):
    return (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1))).float()


def _formula(x, gamma, eps, pos, freq, r0, interleaved):
    """(value, size of the pair it is made of) in 64 bits; x [..., D], pos broadcast over x's leading dims."""
    y = x.double().clone()
    if gamma is not None:
        n = gamma.numel()
        y[..., :n] = y[..., :n] / (y[..., :n].square().mean(-1, keepdim=True) + eps).sqrt() * gamma.double()
    mag = y.abs()
    if freq is not None and freq.numel():
        h = freq.numel()
        i = torch.arange(h)
        lo, hi = (r0 + 2 * i, r0 + 2 * i + 1) if interleaved else (r0 + i, r0 + h + i)
        ang = torch.as_tensor(pos, dtype=torch.float64)[..., None] * freq.double()
        c, s = ang.cos(), ang.sin()
        a, b = y[..., lo].clone(), y[..., hi].clone()
        y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
        size = torch.hypot(a, b) * math.sqrt(2.0)
        mag[..., lo], mag[..., hi] = size, size
    return y, mag


def _assert_bf16(got, ref, mag):
    d = FP32 * mag
    err = (got.double().cpu() - ref).abs()
    bad = err > HALF_BF16 * (ref.abs() + d) + d
    assert not bad.any(), f"{int(bad.sum())} values off, worst {err[bad].max():.3e}"


def _inputs(pg, H, D, seed, scale=2.0):
    return randn(seed, pg.T, H, D, scale=scale), randn(seed + 1, pg.T, D, scale=scale)


CASES = [
    # H, D, q_norm, k_norm, rope_off, rope_dim, interleaved
    (16, ROW, 0, 512, 512, 64, True),
    (128, ROW, 512, 512, 512, 64, False),
    (1, ROW, ROW, ROW, 0, 64, False),
    (33, 128, 128, 128, 0, 64, False),
    (64, 128, 0, 0, 64, 64, True),
    (3, 64, 64, 64, 0, 64, False),
    (5, 40, 24, 40, 8, 16, False),
    (2, 192, 192, 8, 120, 48, True),
    (7, 256, 0, 256, 0, 256, False),
    (40, 512, 512, 512, 256, 128, False),
    (4, 1024, 1024, 1024, 0, 1024, False),
    (2, 8, 8, 8, 0, 0, False),
]


@pytest.mark.parametrize("H,D,qn,kn,r0,R,inter", CASES)
def test_formula(H, D, qn, kn, r0, R, inter):
    pg = Paged([1, 200, 64, 65, 5000, 37], [1, 3, 0, 65, 70, 37], seed=D + H)
    q, k = _inputs(pg, H, D, 11)
    g = torch.Generator().manual_seed(3)
    qg, kg = (torch.rand(n, generator=g) + 0.5 if n else None for n in (qn, kn))
    freq = _freq(R) if R else None
    cache0 = randn(5, pg.num_blocks, PAGE, D)
    cache = cache0.cuda()
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    out = dsa.dsa_qk_norm_rope(pg.batch(), dev(freq), q.cuda(), k.cuda(), q_gamma=dev(qg), k_gamma=dev(kg), eps=1e-5,
                               rope_off=r0, interleaved=inter, k_cache=cache)
    assert_status_ok()
    seq, pos = pg.seq_pos()
    _assert_bf16(out, *_formula(q, qg, 1e-5, np.broadcast_to(pos[:, None], (pg.T, H)), freq, r0, inter))
    rows = np.concatenate([pg.rows(b)[pg.lens[b] - pg.nq[b]:] for b in range(pg.B)])
    got = cache.cpu().view(-1, D)
    _assert_bf16(got[rows], *_formula(k, kg, 1e-5, pos, freq, r0, inter))
    untouched = np.setdiff1d(np.arange(got.shape[0]), rows)
    assert torch.equal(got[untouched], cache0.view(-1, D)[untouched])


@pytest.mark.parametrize("T", [1, 200, 3001])
def test_fp8_latent_rows(T):
    # codes of the formula's values over the tile's own scale: half an e4m3 step (2^-4 of a normal
    # value, 2^-10 of the scale below the smallest normal), plus the fp32 error
    pg = Paged([max(T, 300) + 7], [T], seed=T)
    q, k = _inputs(pg, 16, ROW, 21)
    k[0, 128:256] = 0                      # a tile of zeros keeps scale 1
    kg = torch.rand(512, generator=torch.Generator().manual_seed(1)) + 0.5
    codes0 = torch.randint(0, 120, (pg.num_blocks, PAGE, ROW), dtype=torch.uint8)
    codes, scale = codes0.cuda(), torch.zeros(pg.num_blocks, PAGE, 5, device="cuda")
    dsa.dsa_qk_norm_rope(pg.batch(), _freq(64).cuda(), q.cuda(), k.cuda(), k_gamma=kg.cuda(), interleaved=True,
                         k_cache=codes, k_scale=scale)
    assert_status_ok()
    _, pos = pg.seq_pos()
    ref, mag = _formula(k, kg, 1e-6, pos, _freq(64), 512, True)
    rows = pg.rows(0)[pg.lens[0] - T:]
    got = codes.cpu().view(-1, ROW)[rows]
    s = scale.cpu().view(-1, 5)[rows].double()
    tiles = torch.nn.functional.pad(ref, (0, 64)).view(T, 5, 128)
    am = tiles.abs().amax(-1)
    mm = torch.nn.functional.pad(mag, (0, 64)).view(T, 5, 128).amax(-1)
    want = torch.where(am > 0, am / 448, torch.ones_like(am))
    assert ((s - want).abs() <= (FP32 * mm + 2 * EPS32 * am) / 448).all()
    per = s.repeat_interleave(128, -1)[:, :ROW]
    val = got.view(torch.float8_e4m3fn).double() * per
    d = FP32 * mag + 4 * EPS32 * ref.abs()
    assert ((val - ref).abs() <= 2.0 ** -4 * (ref.abs() + d) + 2.0 ** -10 * per + d).all()
    assert (got[0, 128:256] == 0).all()
    untouched = np.setdiff1d(np.arange(codes0.view(-1, ROW).shape[0]), rows)
    assert torch.equal(codes.cpu().view(-1, ROW)[untouched], codes0.view(-1, ROW)[untouched])
    assert (scale.cpu().view(-1, 5)[untouched] == 0).all()


def test_far_positions():
    # the angle at position 1,048,575 and beyond: a 32-bit product would be off by radians' hundredths
    pg = Paged([1048576, 700], [3, 5], seed=9)
    q, k = _inputs(pg, 4, ROW, 31)
    cache = torch.zeros(pg.num_blocks, PAGE, ROW, dtype=torch.bfloat16, device="cuda")
    out = dsa.dsa_qk_norm_rope(pg.batch(), _freq(64).cuda(), q.cuda(), k.cuda(), k_cache=cache)
    far = torch.tensor([2 ** 31 - 1, 16777217, 0, 1, 999999, 2 ** 30 + 1, 12345678, 7], dtype=torch.int32)
    out2 = dsa.dsa_qk_norm_rope(pg.batch(), _freq(64).cuda(), q.cuda(), k.cuda(), k_cache=cache, positions=far.cuda())
    assert_status_ok()
    _, pos = pg.seq_pos()
    _assert_bf16(out, *_formula(q, None, 0, pos[:, None].repeat(4, 1), _freq(64), 512, False))
    _assert_bf16(out2, *_formula(q, None, 0, far.long().numpy()[:, None].repeat(4, 1), _freq(64), 512, False))


def test_strided_rows_and_in_place():
    # queries and keys as slices of one projection's output; then the rotation written over the queries
    pg = Paged([500, 90], [130, 7], seed=2)
    H, D = 6, 128
    fused = randn(41, pg.T, H + 3, D).cuda()
    q, k = fused[:, :H], fused[:, H]
    cache = torch.zeros(pg.num_blocks, PAGE, D, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(D, device="cuda")
    kw = dict(q_gamma=g, k_gamma=g, rope_off=64)
    out = dsa.dsa_qk_norm_rope(pg.batch(), _freq(64).cuda(), q, k, k_cache=cache, **kw)
    dense, c2 = q.contiguous(), torch.zeros_like(cache)
    same = dsa.dsa_qk_norm_rope(pg.batch(), _freq(64).cuda(), dense, k.contiguous(), k_cache=c2, q_out=dense, **kw)
    assert_status_ok()
    assert same.data_ptr() == dense.data_ptr()
    assert torch.equal(out, dense) and torch.equal(cache, c2)
    _, pos = pg.seq_pos()
    _assert_bf16(out, *_formula(q.cpu(), g.cpu(), 1e-6, pos[:, None].repeat(H, 1), _freq(64), 64, False))
    with pytest.raises(ValueError):
        dsa.dsa_qk_norm_rope(pg.batch(), _freq(64).cuda(), q, q_out=fused[:, :H], **kw)
    with pytest.raises(ValueError):      # rows that start off a 16-byte boundary
        dsa.dsa_qk_norm_rope(pg.batch(), None, fused.view(-1)[1:1 + pg.T * D].view(pg.T, 1, D))


def test_queries_only_keys_only_and_padding():
    # rows behind the last sequence stay as they were; either input may be absent
    pg = Paged([300, 64], [20, 1], seed=3, pad=9)
    q, k = _inputs(pg, 5, ROW, 51)
    mark = torch.full((pg.T, 5, ROW), 7.0, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(pg.num_blocks, PAGE, ROW, dtype=torch.bfloat16, device="cuda")
    both = dsa.dsa_qk_norm_rope(pg.batch(), _freq(64).cuda(), q.cuda(), k.cuda(), k_cache=cache, q_out=mark.clone())
    only_q = dsa.dsa_qk_norm_rope(pg.batch(), _freq(64).cuda(), q.cuda(), q_out=mark.clone())
    c2 = torch.zeros_like(cache)
    assert dsa.dsa_qk_norm_rope(pg.batch(), _freq(64).cuda(), None, k.cuda(), k_cache=c2) is None
    assert_status_ok()
    assert torch.equal(both, only_q) and torch.equal(cache, c2)
    assert (both[pg.real:] == 7).all()
    assert int((cache.view(-1, ROW) != 0).any(-1).sum()) == pg.real


def test_bad_page_is_reported_and_skipped():
    pg = Paged([200, 100], [2, 2], seed=4)
    q, k = _inputs(pg, 2, ROW, 61)
    pg.table[1, 1] = pg.num_blocks + 5           # the page of sequence 1's new tokens
    ws = dsa.Workspace()
    cache = torch.zeros(pg.num_blocks, PAGE, ROW, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_qk_norm_rope(pg.batch(), _freq(64).cuda(), q.cuda(), k.cuda(), k_cache=cache, workspace=ws)
    assert dsa.get_status(ws) == 6               # DSA_ERR_DEVICE_BOUNDS
    assert dsa.get_status(ws) == 0
    assert int((cache.view(-1, ROW) != 0).any(-1).sum()) == 2


def test_captured_and_on_another_stream():
    pg = Paged([3000] * 9, [1] * 9, seed=5)
    q, k = _inputs(pg, 128, ROW, 71)
    b, f, qd, kd = pg.batch(), _freq(64).cuda(), q.cuda(), k.cuda()
    cache = torch.zeros(pg.num_blocks, PAGE, ROW, dtype=torch.bfloat16, device="cuda")
    ref = dsa.dsa_qk_norm_rope(b, f, qd, kd, k_cache=cache)
    want = cache.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cache.zero_()
    torch.cuda.synchronize()
    got = dsa.dsa_qk_norm_rope(b, f, qd, kd, k_cache=cache, stream=side)
    side.synchronize()
    assert torch.equal(got, ref) and torch.equal(cache, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dsa.dsa_qk_norm_rope(b, f, qd, kd, k_cache=cache)
    cache.zero_()
    qd.mul_(2)                                   # exact, and without a norm the result doubles
    graph.replay()
    assert_status_ok()
    assert torch.equal(out, ref * 2) and torch.equal(cache, want)


@pytest.mark.parametrize("T,H", [(1, 6), (5, 1), (1, 1)])
def test_strides_that_are_never_used_may_be_any(T, H):
    # one token, or one head: the stride of a dimension of one element is not used
    pg = Paged([90], [T], seed=6)
    D = 128
    wide = randn(81, T, H * D + D + 4).cuda()                  # rows 4 elements off a 16-byte boundary
    if T == 1:
        q = wide.as_strided((1, H, D), (wide.stride(0), D, 1))
        k = wide[:, H * D:H * D + D]
        assert k.stride(0) % 8
    else:
        q = wide[:, :D].contiguous().as_strided((T, 1, D), (D, 3, 1))
        k = wide[:, D:2 * D].contiguous()
    freq = _freq(64).cuda()
    cache = torch.zeros(pg.num_blocks, PAGE, D, dtype=torch.bfloat16, device="cuda")
    want_c = torch.zeros_like(cache)
    kw = dict(rope_off=64)
    want = dsa.dsa_qk_norm_rope(pg.batch(), freq, torch.empty_strided(q.shape, (H * D, D, 1), dtype=q.dtype, device="cuda").copy_(q),
                                torch.empty_strided(k.shape, (D, 1), dtype=k.dtype, device="cuda").copy_(k), k_cache=want_c, **kw)
    got = dsa.dsa_qk_norm_rope(pg.batch(), freq, q, k, k_cache=cache, **kw)
    assert_status_ok()
    assert torch.equal(got, want) and torch.equal(cache, want_c)
    same = dsa.dsa_qk_norm_rope(pg.batch(), freq, q, q_out=q, **kw)      # in place
    assert_status_ok()
    assert same.data_ptr() == q.data_ptr() and torch.equal(same, want)


def test_one_token_of_a_larger_buffer_in_place():
    pg = Paged([90], [1], seed=7)
    buf = randn(91, 4, 9, 128).cuda()
    rest = buf.clone()
    q = buf[:1, :6]
    want = dsa.dsa_qk_norm_rope(pg.batch(), _freq(64).cuda(), q.clone().view(1, 6, 128), rope_off=0)
    dsa.dsa_qk_norm_rope(pg.batch(), _freq(64).cuda(), q, q_out=q, rope_off=0)
    assert_status_ok()
    assert torch.equal(buf[:1, :6], want)
    assert torch.equal(buf[1:], rest[1:]) and torch.equal(buf[0, 6:], rest[0, 6:])
