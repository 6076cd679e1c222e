"""dsa_chunk_attn over an FP8 latent cache on the GPU: the shapes, masks and failures at which the
warps that convert codes could go wrong, against dense causal attention in 64 bits over the values
that the codes stand for (tolerances of test_chunk_gpu.reference)."""
import math

import numpy as np
import pytest
import torch

import indexer_top_sparse_lightning_b200 as dsa
from tests.paged_helpers import DV, PAGE, ROW, Paged, assert_status_ok, fp8_rows, randn
from tests.test_chunk_gpu import SCALE, SHAPES, check, reference, run

pytestmark = pytest.mark.gpu

NAN = 0x7F


def cache(pg, seed):
    """(codes, scales, values): NaN codes, and scales NaN, infinite or huge, where nobody looks."""
    codes, scale, val = fp8_rows(randn(seed, pg.num_blocks, PAGE, ROW))
    used = np.zeros(pg.num_blocks * PAGE, bool)
    for b in range(pg.B):
        used[pg.rows(b)] = True
    codes.view(-1, ROW)[~used] = NAN
    other = scale.view(-1, 5)
    other[~used] = torch.tensor([math.nan, math.inf, -math.inf, 3e38, -0.0])
    return codes, scale, val.view(-1, ROW)


@pytest.mark.parametrize("lens,nq,H", SHAPES)
def test_dense_causal(lens, nq, H):
    pg = Paged(lens, nq, seed=H + len(lens), pad=3)
    q = randn(1 + H, pg.T, H, ROW, scale=3.0)
    codes, scale, val = cache(pg, 2)
    mark = torch.full((pg.T, H, DV), 5.0, dtype=torch.bfloat16, device="cuda")
    ml = torch.full((pg.T, H), 5.0, device="cuda")
    out, lse = run(pg, q, codes, kv_scale=scale.cuda(), out=mark, lse=ml)
    check(pg, out, lse, reference(pg, q, lambda b: val[pg.rows(b)], fp16=True))
    assert (out[pg.real:] == 5).all() and (lse[pg.real:] == 5).all()      # padding rows stay


def test_many_sequences():
    # more sequences than threads of a block; many without new tokens
    r = np.random.default_rng(8)
    lens = r.integers(1, 300, size=900)
    nq = np.minimum(lens, r.integers(0, 3, size=900))
    pg = Paged(lens, nq, seed=1)
    q = randn(3, pg.T, 8, ROW, scale=3.0)
    codes, scale, val = cache(pg, 4)
    out, lse = run(pg, q, codes, kv_scale=scale.cuda())
    check(pg, out, lse, reference(pg, q, lambda b: val[pg.rows(b)], fp16=True))


def test_growing_scores():
    # every block raises the maximum: the output so far is rescaled again and again
    pg = Paged([1500], [40], seed=3)
    q = randn(5, pg.T, 128, ROW).abs()
    ramp = torch.linspace(-20, 20, 1500)[:, None]
    x = randn(6, pg.num_blocks, PAGE, ROW)
    x.view(-1, ROW)[pg.rows(0)] = (randn(7, 1500, ROW).float() * 0.5 + ramp * 0.1).to(torch.bfloat16)
    codes, scale, val = fp8_rows(x)
    out, lse = run(pg, q, codes, kv_scale=scale.cuda())
    check(pg, out, lse, reference(pg, q, lambda b: val.view(-1, ROW)[pg.rows(b)], fp16=True))


@pytest.mark.parametrize("what", ["codes", "scales"])
@pytest.mark.parametrize("H", [16, 40, 128, 1])
def test_later_tokens_rows_do_not_reach_earlier_ones(H, what):
    # the last tokens' rows are not finite: every token before them is unaffected (tiles hold
    # several tokens when H < 128), every token that sees one gets no finite result
    n, good = 70, 50
    pg = Paged([400], [n], seed=4)
    q = randn(8, n, H, ROW, scale=3.0)
    codes, scale, val = cache(pg, 9)
    rows = pg.rows(0)
    late = rows[400 - n + good:]
    if what == "codes":
        codes.view(-1, ROW)[late, 100] = NAN
    else:
        scale.view(-1, 5)[late, 2] = math.nan
    clean = val.clone()
    clean[late] = 0
    out, lse = run(pg, q, codes, kv_scale=scale.cuda())
    ro, rl, bo, bl = reference(pg, q, lambda b: clean[rows], fp16=True)
    assert ((out[:good].double() - ro[:good]).abs() <= bo[:good]).all()
    assert ((lse[:good].double() - rl[:good]).abs() <= bl[:good]).all()
    assert not torch.isfinite(lse[good:]).any()


def test_bad_page_is_reported_and_not_seen():
    pg = Paged([600, 500], [3, 20], seed=8)
    q = randn(15, pg.T, 32, ROW, scale=3.0)
    codes, scale, val = cache(pg, 16)
    ref = reference(pg, q, lambda b: val[pg.rows(b)], fp16=True,
                    hidden=lambda b: (torch.arange(int(pg.lens[b])) // PAGE == 3) if b == 1 else
                    torch.zeros(int(pg.lens[b]), dtype=torch.bool))
    pg.table[1, 3] = pg.num_blocks
    ws = dsa.Workspace()
    out, lse = dsa.dsa_chunk_attn(pg.batch(), q.cuda(), codes.cuda(), SCALE, kv_scale=scale.cuda(), workspace=ws)
    torch.cuda.synchronize()
    assert dsa.get_status(ws) == 6
    check(pg, out, lse, ref)


def test_repeats_captures_and_streams_agree():
    # bit for bit: twice, on two streams at once, and from two graphs replayed at the same time
    pg = Paged([5000, 900, 64, 3000], [3, 200, 1, 7], seed=9)
    q = randn(17, pg.T, 64, ROW, scale=3.0).cuda()
    codes, scale, _ = cache(pg, 18)
    codes, scale = codes.cuda(), scale.cuda()
    b = pg.batch()
    call = lambda **kw: dsa.dsa_chunk_attn(b, q, codes, SCALE, kv_scale=scale, **kw)  # noqa: E731
    ref, rl = call()
    again, al = call()
    assert torch.equal(ref, again) and torch.equal(rl, al)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [call(stream=s) for _ in range(4) for s in (s1, s2)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) and torch.equal(x, rl) for o, x in outs)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = call()
        graphs.append((g, res))
    for (g, _), s in zip(graphs, (s1, s2)):
        with torch.cuda.stream(s):
            g.replay()
    assert_status_ok()
    for _, (o, x) in graphs:
        assert torch.equal(o, ref) and torch.equal(x, rl)


def test_offsets_past_32_bits():
    # the codes of the last pages lie more than 2^31 bytes into the cache
    blocks = 2 ** 31 // (PAGE * ROW) + 40
    pg = Paged([300], [2], seed=6)
    q = randn(13, pg.T, 128, ROW, scale=3.0)
    codes, scale, val = fp8_rows(randn(14, pg.num_blocks, PAGE, ROW))
    big = torch.empty(blocks, PAGE, ROW, dtype=torch.uint8, device="cuda")
    sc = torch.empty(blocks, PAGE, 5, dtype=torch.float32, device="cuda")
    big[-pg.num_blocks:], sc[-pg.num_blocks:] = codes.cuda(), scale.cuda()
    rows = pg.rows(0)
    pg.table[pg.table >= 0] += blocks - pg.num_blocks
    pg.num_blocks = blocks
    out, lse = dsa.dsa_chunk_attn(pg.batch(), q.cuda(), big, SCALE, kv_scale=sc)
    assert_status_ok()
    check(pg, out, lse, reference(pg, q, lambda b: val.view(-1, ROW)[rows], fp16=True))


def test_scratch_does_not_grow_with_the_cache():
    pg = Paged([64], [1], seed=1)
    b = pg.batch()
    q, codes = torch.zeros(1, 128, ROW, dtype=torch.bfloat16).cuda(), torch.zeros(pg.num_blocks, PAGE, ROW, dtype=torch.uint8).cuda()
    sc = torch.ones(pg.num_blocks, PAGE, 5).cuda()
    dsa.dsa_chunk_attn(b, q, codes, SCALE, kv_scale=sc)
    table = torch.full((1, 1 << 14), -1, dtype=torch.int32, device="cuda")
    table[0, 0] = b.block_table[0, 0]
    long = dsa.Batch(b.seq_lens, b.cu_q, table, pg.num_blocks, 1 << 20, 1)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    dsa.dsa_chunk_attn(long, q, codes, SCALE, kv_scale=sc)
    assert_status_ok()
    assert torch.cuda.max_memory_allocated() - before < 64 << 20


def test_timeout_is_reported_and_recoverable():
    pg = Paged([3000], [4], seed=11)
    q = randn(21, pg.T, 128, ROW).cuda()
    codes, scale, _ = cache(pg, 22)
    codes, scale = codes.cuda(), scale.cuda()
    ws = dsa.Workspace()
    call = lambda: dsa.dsa_chunk_attn(pg.batch(), q, codes, SCALE, kv_scale=scale, workspace=ws)[0]  # noqa: E731
    clean = call()
    assert dsa.get_status(ws) == 0
    words = ws.buf[:16].view(torch.int32)
    words[1], words[2] = 5000, 4
    call()
    assert dsa.get_status(ws) == 5                     # DSA_ERR_TIMEOUT
    ws.reset()
    assert torch.equal(clean, call()) and dsa.get_status(ws) == 0


def test_copied_and_converted_agree():
    # 40 tokens of 128 heads over few positions are copied, one by one they are converted in the
    # kernel: each within its bound of the same sum
    n, H = 40, 128
    pg = Paged([900], [n], seed=12)
    q = randn(31, n, H, ROW, scale=3.0)
    codes, scale, val = cache(pg, 32)
    ref = reference(pg, q, lambda b: val[pg.rows(b)], fp16=True)
    out, lse = run(pg, q, codes, kv_scale=scale.cuda())
    check(pg, out, lse, ref)
    for j in (0, 17, n - 1):
        one = Paged([900], [n], seed=12)
        one.lens, one.nq, one.cu, one.real = np.array([900 - n + j + 1]), np.array([1]), np.array([0, 1], np.int32), 1
        o, x = run(one, q[j:j + 1], codes, kv_scale=scale.cuda())
        check(one, o, x, [r[j:j + 1] for r in ref])


def _few(seed, T, H, where, k=4):
    """Queries with k elements that are not zero in each of the ranges `where`: the fp32 sum of the score's
    products has that many terms, so that what is off is the operands."""
    r = np.random.default_rng(seed)
    q = torch.zeros(T, H, ROW)
    for t in range(T):
        for h in range(H):
            for lo, hi in where:
                at = r.choice(np.arange(lo, hi), k, replace=False)
                q[t, h, at] = torch.from_numpy(r.standard_normal(k).astype(np.float32) * 3)
    return q


@pytest.mark.parametrize("mag", [-10, -4, 0, 4, 10])
@pytest.mark.parametrize("zero", [(512, 576), (384, 512), (448, 512), None])
@pytest.mark.parametrize("ratio", [-12, 0, 12])
def test_scores_of_neighbouring_tiles_are_exact(zero, mag, ratio):
    # One position a sequence, so that lse is the score itself.  The RoPE tile is 2^ratio times the
    # latents' size; a tile of zeros has the scale 1 beside neighbours of any size (mag).  The products of
    # codes are exact in fp32 and 4 or 8 of them are added (8 half steps of 2^-24 of the sum of magnitudes,
    # and as many for the four scales and the query's).  RoPE values c g4 take part as two fp16 parts: with
    # g4 = gh + gl, h = c gh rounded and l = c gl + (c gh - h), |gl| <= 2^-11 g4 (off by 2^-22 g4) and
    # |c gh - h| <= 2^-11 c g4, so l <= 2^-10 c g4 is off by 2^-21 c g4: 3 * 2^-22 in all, or by two half steps
    # of 2^-24 where it is subnormal, in a unit that is at least a 128th of tile 3's scale (the unit is that or
    # a 64th of the RoPE tile's, whose own 2^-21 covers it): 2^-31 of that scale.  The score in log2 units is put
    # together with the page's exponent, |log2 F| <= 32: eight roundings of 1.45 |S| + 48.
    B, H = 48, 8
    pg = Paged([1] * B, [1] * B, seed=14)
    x = randn(61, pg.num_blocks, PAGE, ROW).float() * 2.0 ** mag
    x[..., 512:] *= 2.0 ** ratio
    if zero:
        x[..., zero[0]:zero[1]] = 0
    codes, scale, val = fp8_rows(x.to(torch.bfloat16))
    q = _few(62, B, H, [(384, 448), (512, ROW)]) * 2.0 ** -mag
    q[..., 512:] *= 2.0 ** -ratio
    q = q.to(torch.bfloat16)
    out, lse = run(pg, q, codes, kv_scale=scale.cuda())
    rows = np.concatenate([pg.rows(b) for b in range(B)])
    v, f = val.view(-1, ROW)[rows], scale.view(-1, 5)[rows].double()
    s = torch.einsum("thd,td->th", q.double(), v) * SCALE
    size = torch.einsum("thd,td->th", q.double().abs(), v.abs()) * SCALE
    rope = torch.einsum("thd,td->th", q.double().abs()[..., 512:], v.abs()[:, 512:]) * SCALE
    step = q.double().abs()[..., 512:].sum(-1) * f[:, 3:4] * 2.0 ** -31 * SCALE
    tol = 16 * 2.0 ** -24 * size + 3 * 2.0 ** -22 * rope + step + 8 * 2.0 ** -24 * (1.45 * s.abs() + 48)
    err = (lse.cpu().double() - s).abs()
    assert (err <= tol).all(), f"worst {float((err / tol).max()):.1f} of the bound, off by {float(err.max()):.2e}"


@pytest.mark.parametrize("mag", [-6, 0, 6])
@pytest.mark.parametrize("zero", [(512, 576), (384, 512), (384, 576), (0, 128), (0, 576)])
@pytest.mark.parametrize("n", [20, 130])          # converted in the kernel; copied
def test_tiles_of_zeros(n, zero, mag):
    # some rows have tiles of zeros, which have the scale 1, between others of any size
    H = 32
    pg = Paged([700, 130], [3, n], seed=15)
    x = randn(63, pg.num_blocks, PAGE, ROW).float() * 2.0 ** mag
    x[:, ::3, zero[0]:zero[1]] = 0
    codes, scale, val = fp8_rows(x.to(torch.bfloat16))
    q = (randn(64, pg.T, H, ROW, scale=3.0).float() * 2.0 ** -mag).to(torch.bfloat16)
    out, lse = run(pg, q, codes, kv_scale=scale.cuda())
    check(pg, out, lse, reference(pg, q, lambda b: val.view(-1, ROW)[pg.rows(b)], fp16=True))


def _graphs_and_streams(call):
    """call(**kw) gives the same bits twice, on two streams at once, and from two graphs replayed at once."""
    ref, rl = call()
    again, al = call()
    assert torch.equal(ref, again) and torch.equal(rl, al)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [call(stream=s) for _ in range(4) for s in (s1, s2)]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = call()
        graphs.append((g, res))
    for (g, _), s in zip(graphs, (s1, s2)):
        with torch.cuda.stream(s):
            g.replay()
    assert_status_ok()
    assert all(torch.equal(o, ref) and torch.equal(x, rl) for o, x in outs + [r for _, r in graphs])


def test_repeats_captures_and_streams_agree_where_the_kernel_converts():
    # fewer (token, head) rows than are worth a copy of the cache
    pg = Paged([5000, 900, 64, 3000], [3, 60, 1, 7], seed=9)
    assert int(pg.nq.max()) * 64 < 4096
    q = randn(17, pg.T, 64, ROW, scale=3.0).cuda()
    codes, scale, _ = cache(pg, 18)
    b, codes, scale = pg.batch(), codes.cuda(), scale.cuda()
    _graphs_and_streams(lambda **kw: dsa.dsa_chunk_attn(b, q, codes, SCALE, kv_scale=scale, **kw))


def test_growing_scores_where_the_kernel_converts():
    pg = Paged([1500], [31], seed=3)
    q = randn(5, pg.T, 128, ROW).abs()
    x = randn(6, pg.num_blocks, PAGE, ROW)
    x.view(-1, ROW)[pg.rows(0)] = (randn(7, 1500, ROW).float() * 0.5 + torch.linspace(-2, 2, 1500)[:, None]).to(torch.bfloat16)
    codes, scale, val = fp8_rows(x)
    out, lse = run(pg, q, codes, kv_scale=scale.cuda())
    check(pg, out, lse, reference(pg, q, lambda b: val.view(-1, ROW)[pg.rows(b)], fp16=True))


@pytest.mark.parametrize("what", ["codes", "scales"])
def test_later_tokens_rows_do_not_reach_earlier_ones_where_the_kernel_converts(what):
    n, good, H = 30, 20, 128
    pg = Paged([400], [n], seed=4)
    q = randn(8, n, H, ROW, scale=3.0)
    codes, scale, val = cache(pg, 9)
    rows = pg.rows(0)
    late = rows[400 - n + good:]
    if what == "codes":
        codes.view(-1, ROW)[late, 100] = NAN
    else:
        # (of every tile in turn, the two that share an accumulator among them)
        scale.view(-1, 5)[late, np.arange(n - good) % 5] = math.nan
    clean = val.clone()
    clean[late] = 0
    out, lse = run(pg, q, codes, kv_scale=scale.cuda())
    ro, rl, bo, bl = reference(pg, q, lambda b: clean[rows], fp16=True)
    assert ((out[:good].double() - ro[:good]).abs() <= bo[:good]).all()
    assert ((lse[:good].double() - rl[:good]).abs() <= bl[:good]).all()
    assert not torch.isfinite(lse[good:]).any()
