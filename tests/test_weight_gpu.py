"""dsa_attn_weight on the GPU against its formula in 64 bits.

Tolerance.  A term is exp(s - lse): its error relative to itself is that of the
exponent, D <= (576 + 8) 2^-23 scale sum_i |q_i k_i| for the score (an fp32 sum of
576 exact products; twice the terms over an FP8 cache, and 2^-22 of the magnitudes
for the copy's rounding) plus 4 * 2^-24 (|s| + |lse|) for the subtraction in log2
units, plus 2^-21 for the exponential.  The sum of N terms, all positive, is off by
at most (N + 8) 2^-24 of itself (a lane adds N / 8 terms, then tiles one after
another), and decay * w by two more roundings."""
import math

import numpy as np
import pytest
import torch

import indexer_top_sparse_lightning_b200 as dsa
from tests.paged_helpers import PAGE, ROW, Paged, assert_status_ok, fp8_rows, randn
from tests.test_chunk_gpu import SCALE, latent

pytestmark = pytest.mark.gpu


def expect(pg, q, rows_of, lse, w0, decay, fp8=False, hidden=None):
    """(value, bound) of the weights, 64 bits, [B, stride]."""
    val, bound = w0.double().cuda().clone(), torch.zeros(w0.shape, dtype=torch.float64, device="cuda")
    H = q.shape[1]
    for b in range(pg.B):
        n, L = int(pg.nq[b]), int(pg.lens[b])
        if n == 0:
            continue
        x, t0 = rows_of(b).cuda().double(), int(pg.cu[b])
        total, off = torch.zeros(L, dtype=torch.float64, device="cuda"), torch.zeros(L, dtype=torch.float64, device="cuda")
        step = max(1, 20_000_000 // (H * L))
        for j in range(0, n, step):
            k = min(step, n - j)
            qq, l = q[t0 + j:t0 + j + k].cuda().double(), lse[t0 + j:t0 + j + k].cuda().double()[..., None]
            s = torch.einsum("thd,sd->ths", qq, x) * SCALE
            mag = torch.einsum("thd,sd->ths", qq.abs(), x.abs()) * SCALE
            pos = torch.arange(L - n + j, L - n + j + k, device="cuda")
            see = (torch.arange(L, device="cuda")[None] <= pos[:, None])[:, None] & torch.isfinite(l)
            if hidden is not None:
                see = see & ~hidden(b).cuda()
            e = torch.where(see, (s - l).exp(), torch.zeros_like(s))
            D = ((1152 + 8 + 2) if fp8 else 584) * 2.0 ** -23 * mag + 4 * 2.0 ** -24 * (s.abs() + l.abs()) + 2.0 ** -21
            total += e.sum((0, 1))
            off += torch.where(see, e * torch.expm1(D), torch.zeros_like(s)).sum((0, 1))
        old = decay * val[b, :L] if decay else torch.zeros_like(total)
        val[b, :L] = old + total
        bound[b, :L] = off + (n * H + 8) * 2.0 ** -24 * total + 2 * 2.0 ** -24 * (old.abs() + total)
    return val, bound


SHAPES = [
    # lens, new tokens, heads, decay
    ([1], [1], 1, 1.0), ([64], [1], 16, 0.5), ([65], [1], 128, 0.0), ([256], [1], 128, 1.0), ([257], [2], 64, 0.25),
    ([4096], [1], 16, 1.0), ([20000], [1], 128, 1.0), ([9000], [128], 1, 1.0),
    ([300, 1, 700, 64, 5000], [1, 1, 0, 1, 1], 128, 0.5), ([300, 1, 700, 64, 5000], [2, 1, 0, 2, 3], 33, 0.5),
    ([513, 90, 1], [200, 90, 1], 7, 1.0), ([257], [257], 16, 0.0), ([3000], [513], 64, 0.5), ([700], [700], 128, 1.0),
    ([1500, 40, 33], [600, 40, 0], 96, 0.9), ([2000], [2000], 1, 1.0), ([600], [2], 128, 1.0), ([600], [3], 128, 1.0),
]


@pytest.mark.parametrize("lens,nq,H,decay", SHAPES)
def test_formula(lens, nq, H, decay):
    pg = Paged(lens, nq, seed=H, pad=2)
    q, kv = randn(1 + H, pg.T, H, ROW, scale=3.0), latent(pg, 2)
    _, lse = dsa.dsa_chunk_attn(pg.batch(), q.cuda(), kv.cuda(), SCALE)
    w0 = torch.rand(pg.B, max(lens) + 5, generator=torch.Generator().manual_seed(3)) * 4
    if decay == 0.0:
        w0[:, ::3] = math.nan                      # not read
    w = w0.cuda()
    assert dsa.dsa_attn_weight(pg.batch(), q.cuda(), kv.cuda(), SCALE, lse, w, decay=decay).data_ptr() == w.data_ptr()
    assert_status_ok()
    val, bound = expect(pg, q, lambda b: kv.view(-1, ROW)[pg.rows(b)], lse, w0, decay)
    for b in range(pg.B):
        L = int(pg.lens[b]) if pg.nq[b] else 0     # beyond: untouched
        assert torch.equal(torch.nan_to_num(w[b, L:].cpu(), 9.0), torch.nan_to_num(w0[b, L:], 9.0))
        err = (w[b, :L].double() - val[b, :L]).abs()
        assert (err <= bound[b, :L]).all(), float((err / bound[b, :L]).max())


def test_weights_of_every_token_sum_to_the_rows():
    # each (token, head) row's softmax weights add up to one
    pg = Paged([900, 64, 5000], [40, 64, 1], seed=1)
    q, kv = randn(11, pg.T, 48, ROW, scale=3.0).cuda(), latent(pg, 12).cuda()
    _, lse = dsa.dsa_chunk_attn(pg.batch(), q, kv, SCALE)
    w = torch.zeros(3, 5000, device="cuda")
    dsa.dsa_attn_weight(pg.batch(), q, kv, SCALE, lse, w)
    assert_status_ok()
    want = torch.from_numpy(pg.nq * 48.0).cuda()
    assert ((w.double().sum(1) - want).abs() <= 1e-4 * want).all()


def test_many_sequences():
    r = np.random.default_rng(5)
    lens = r.integers(1, 300, size=500)
    nq = np.minimum(lens, r.integers(0, 2, size=500))
    pg = Paged(lens, nq, seed=2)
    q, kv = randn(21, pg.T, 8, ROW, scale=3.0), latent(pg, 22)
    _, lse = dsa.dsa_chunk_attn(pg.batch(), q.cuda(), kv.cuda(), SCALE)
    w0 = torch.rand(500, 300)
    w = w0.cuda()
    dsa.dsa_attn_weight(pg.batch(), q.cuda(), kv.cuda(), SCALE, lse, w)
    assert_status_ok()
    val, bound = expect(pg, q, lambda b: kv.view(-1, ROW)[pg.rows(b)], lse, w0, 1.0)
    assert ((w.double() - val).abs() <= bound).all()


def test_windows_of_new_tokens():
    # one long sequence among many: sums per tile for all of them do not fit the scratch at once, so
    # the new tokens are taken in windows (64 sequences of 200,000 positions leave room for five tiles
    # each; every window adds its own rounding, so twice the bound)
    lens, nq = [3000] + [70] * 63, [700] + [1] * 63
    pg = Paged(lens, nq, seed=3)
    q, kv = randn(31, pg.T, 16, ROW, scale=3.0), latent(pg, 32)
    b = pg.batch()
    b.block_table = torch.nn.functional.pad(b.block_table, (0, 3200 - b.block_table.shape[1]), value=-1)
    b.max_seq_len = 200000
    _, lse = dsa.dsa_chunk_attn(b, q.cuda(), kv.cuda(), SCALE)
    w0 = torch.rand(64, 200000)
    w = w0.cuda()
    dsa.dsa_attn_weight(b, q.cuda(), kv.cuda(), SCALE, lse, w, decay=0.5)
    assert_status_ok()
    val, bound = expect(pg, q, lambda b: kv.view(-1, ROW)[pg.rows(b)], lse, w0, 0.5)
    assert ((w.double() - val).abs() <= 2 * bound).all()


@pytest.mark.parametrize("lens,nq,H", [([500, 3000], [1, 1], 24), ([500, 3000, 64], [70, 3, 0], 24)])
def test_fp8_latent_cache(lens, nq, H):
    pg = Paged(lens, nq, seed=5)
    q = randn(41, pg.T, H, ROW, scale=3.0)
    codes, scale, val8 = fp8_rows(randn(42, pg.num_blocks, PAGE, ROW))
    _, lse = dsa.dsa_chunk_attn(pg.batch(), q.cuda(), codes.cuda(), SCALE, kv_scale=scale.cuda())
    w0 = torch.rand(pg.B, 3000)
    w = w0.cuda()
    dsa.dsa_attn_weight(pg.batch(), q.cuda(), codes.cuda(), SCALE, lse, w, kv_scale=scale.cuda())
    assert_status_ok()
    val, bound = expect(pg, q, lambda b: val8.view(-1, ROW)[pg.rows(b)], lse, w0, 1.0, fp8=True)
    assert ((w.double() - val).abs() <= bound).all()


def test_masked_places_may_hold_anything():
    # rows that see nothing (lse -inf), queries of padding and of rows behind a tile that are not
    # finite, later rows that are not finite
    pg = Paged([400, 90], [50, 3], seed=6, pad=4)
    H = 24
    q = randn(51, pg.T, H, ROW, scale=3.0)
    q[pg.real:] = math.nan
    kv = latent(pg, 52)
    clean = kv.view(-1, ROW)[pg.rows(0)].clone()
    kv.view(-1, ROW)[pg.rows(0)[395:]] = math.nan
    _, lse = dsa.dsa_chunk_attn(pg.batch(), q.cuda(), kv.cuda(), SCALE)
    lse[:45] = torch.where(torch.isfinite(lse[:45]), lse[:45], torch.zeros_like(lse[:45]))
    lse[45:50] = -math.inf                         # the tokens that see the rows that are not finite
    lse[7] = -math.inf
    w = torch.zeros(2, 500, device="cuda")
    dsa.dsa_attn_weight(pg.batch(), q.cuda(), kv.cuda(), SCALE, lse, w)
    assert_status_ok()
    clean[395:] = 0
    rows = [clean, kv.view(-1, ROW)[pg.rows(1)]]
    val, bound = expect(pg, q, lambda b: rows[b], lse, torch.zeros(2, 500), 1.0)
    assert ((w[:, :395].double() - val[:, :395]).abs() <= bound[:, :395]).all()


def test_bad_page_and_surplus_are_reported():
    pg = Paged([600, 500], [1, 1], seed=7)
    q, kv = randn(61, pg.T, 32, ROW, scale=3.0), latent(pg, 62)
    _, lse = dsa.dsa_chunk_attn(pg.batch(), q.cuda(), kv.cuda(), SCALE)
    good = kv.view(-1, ROW)[pg.rows(1)]
    pg.table[1, 3] = -5
    ws = dsa.Workspace()
    w = torch.zeros(2, 600, device="cuda")
    dsa.dsa_attn_weight(pg.batch(), q.cuda(), kv.cuda(), SCALE, lse, w, workspace=ws)
    assert dsa.get_status(ws) == 6
    rows = [kv.view(-1, ROW)[pg.rows(0)], good]
    val, bound = expect(pg, q, lambda b: rows[b], lse, torch.zeros(2, 600), 1.0,
                        hidden=lambda b: (torch.arange(int(pg.lens[b])) // PAGE == 3) & (b == 1))
    assert ((w.double() - val).abs() <= bound).all()
    # a batch that understates its longest chunk
    pg = Paged([600], [9], seed=8)
    q, kv = randn(63, 9, 128, ROW).cuda(), latent(pg, 64).cuda()
    b = pg.batch()
    _, lse = dsa.dsa_chunk_attn(b, q, kv, SCALE)
    b.max_q_per_seq = 1
    dsa.dsa_attn_weight(b, q, kv, SCALE, lse, w[:1], workspace=ws)
    assert dsa.get_status(ws) == 6


def test_repeats_streams_and_captures_agree():
    pg = Paged([5000, 900, 64, 3000], [3, 200, 1, 7], seed=9)
    q, kv = randn(71, pg.T, 64, ROW, scale=3.0).cuda(), latent(pg, 72).cuda()
    b = pg.batch()
    _, lse = dsa.dsa_chunk_attn(b, q, kv, SCALE)
    ref = dsa.dsa_attn_weight(b, q, kv, SCALE, lse, torch.zeros(4, 5000, device="cuda"))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ws = [torch.zeros(4, 5000, device="cuda") for _ in range(6)]
    torch.cuda.synchronize()
    for i in range(4):
        dsa.dsa_attn_weight(b, q, kv, SCALE, lse, ws[i], stream=(s1, s2)[i % 2])
    torch.cuda.synchronize()
    graphs = []
    for i in (4, 5):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dsa.dsa_attn_weight(b, q, kv, SCALE, lse, ws[i], decay=0.0)
        graphs.append(g)
    for g, s in zip(graphs, (s1, s2)):
        with torch.cuda.stream(s):
            g.replay()
    assert_status_ok()
    assert all(torch.equal(w, ref) for w in ws)


@pytest.mark.parametrize("nq,H", [([1, 1], 128), ([1, 2], 33), ([40, 3], 64)])
def test_rows_that_saw_nothing_add_nothing(nq, H):
    # whatever their queries hold
    pg = Paged([700, 300], nq, seed=5)
    q, kv = randn(21, pg.T, H, ROW, scale=3.0).cuda(), latent(pg, 22).cuda()
    _, lse = dsa.dsa_chunk_attn(pg.batch(), q, kv, SCALE)
    dead = torch.rand(pg.T, H, generator=torch.Generator().manual_seed(6)).cuda() < 0.3
    lse[dead] = -math.inf
    clean, dirty = q.clone(), q.clone()
    clean[dead], dirty[dead] = 0.0, math.nan
    a, b = (dsa.dsa_attn_weight(pg.batch(), x, kv, SCALE, lse, torch.zeros(2, 700, device="cuda")) for x in (clean, dirty))
    assert_status_ok()
    assert torch.equal(a, b) and float(a.sum()) > 0


@pytest.mark.parametrize("n,L,H", [(90, 70, 24), (4, 3, 16)])
def test_a_length_below_the_new_tokens_is_reported(n, L, H):
    # the tokens in front of the sequence's start (token j stands at seq_lens - nq + j) add nothing
    pg = Paged([300, n, 64], [5, n, 1], seed=12)
    q, kv = randn(81, pg.T, H, ROW, scale=3.0), latent(pg, 82, nan_elsewhere=False)
    pg.lens[1] = L
    ws, w = dsa.Workspace(), torch.zeros(3, 300, device="cuda")
    lse = torch.full((pg.T, H), 3.0)
    cut = Paged([300, n, 64], [5, n, 1], seed=12)
    cut.lens[1], cut.nq[1] = L, L
    cut.cu = np.array([0, 5, 5 + L, 6 + L], np.int32)
    cut.real = cut.T = 6 + L
    keep = torch.tensor([t for t in range(pg.T) if not 5 <= t < 5 + n - L])
    dsa.dsa_attn_weight(pg.batch(), q.cuda(), kv.cuda(), SCALE, lse.cuda(), w, workspace=ws)
    assert dsa.get_status(ws) == 6
    val, bound = expect(cut, q[keep], lambda b: kv.view(-1, ROW)[cut.rows(b)], lse[keep], torch.zeros(3, 300), 1.0)
    assert ((w.double() - val).abs() <= bound).all()


def test_more_new_tokens_than_rows_are_reported():
    # a cu_q that goes past the queries: the rows that are there keep their tokens' positions
    gone, H = 50, 24
    pg = Paged([300, 400, 64], [5, 90, 3], seed=13)
    q, kv = randn(91, pg.T, H, ROW, scale=3.0), latent(pg, 92)
    n = pg.T - gone
    ws, w = dsa.Workspace(), torch.zeros(3, 400, device="cuda")
    lse = torch.full((pg.T, H), 3.0)
    dsa.dsa_attn_weight(pg.batch(), q[:n].cuda(), kv.cuda(), SCALE, lse[:n].cuda(), w, workspace=ws)
    assert dsa.get_status(ws) == 6
    lse[n:] = -math.inf                                  # rows that are not there add nothing
    val, bound = expect(pg, q, lambda b: kv.view(-1, ROW)[pg.rows(b)], lse, torch.zeros(3, 400), 1.0)
    assert ((w.double() - val).abs() <= bound).all()


def _codes(pg, seed):
    """(codes, scales, values): NaN codes, and scales NaN, infinite or huge, where nobody looks."""
    codes, scale, val = fp8_rows(randn(seed, pg.num_blocks, PAGE, ROW))
    used = np.zeros(pg.num_blocks * PAGE, bool)
    for b in range(pg.B):
        used[pg.rows(b)] = True
    codes.view(-1, ROW)[~used] = 0x7F
    scale.view(-1, 5)[~used] = torch.tensor([math.nan, math.inf, -math.inf, 3e38, -0.0])
    return codes, scale, val.view(-1, ROW)


@pytest.mark.parametrize("lens,nq,H,decay", SHAPES)
def test_formula_over_an_fp8_cache(lens, nq, H, decay):
    pg = Paged(lens, nq, seed=H, pad=2)
    q = randn(1 + H, pg.T, H, ROW, scale=3.0)
    codes, scale, val8 = _codes(pg, 2)
    cd, sd = codes.cuda(), scale.cuda()
    _, lse = dsa.dsa_chunk_attn(pg.batch(), q.cuda(), cd, SCALE, kv_scale=sd)
    w0 = torch.rand(pg.B, max(lens) + 5, generator=torch.Generator().manual_seed(3)) * 4
    w = w0.cuda()
    dsa.dsa_attn_weight(pg.batch(), q.cuda(), cd, SCALE, lse, w, decay=decay, kv_scale=sd)
    assert_status_ok()
    val, bound = expect(pg, q, lambda b: val8[pg.rows(b)], lse, w0, decay, fp8=True)
    for b in range(pg.B):
        L = int(pg.lens[b]) if pg.nq[b] else 0     # beyond: untouched
        assert torch.equal(w[b, L:].cpu(), w0[b, L:])
        assert ((w[b, :L].double() - val[b, :L]).abs() <= bound[b, :L]).all()


def test_bad_page_of_an_fp8_cache_is_reported():
    pg = Paged([600, 500], [1, 9], seed=7)
    q = randn(61, pg.T, 32, ROW, scale=3.0)
    codes, scale, val8 = _codes(pg, 62)
    _, lse = dsa.dsa_chunk_attn(pg.batch(), q.cuda(), codes.cuda(), SCALE, kv_scale=scale.cuda())
    rows = [val8[pg.rows(b)] for b in range(2)]
    pg.table[1, 3] = -5
    ws, w = dsa.Workspace(), torch.zeros(2, 600, device="cuda")
    dsa.dsa_attn_weight(pg.batch(), q.cuda(), codes.cuda(), SCALE, lse, w, kv_scale=scale.cuda(), workspace=ws)
    assert dsa.get_status(ws) == 6
    val, bound = expect(pg, q, lambda b: rows[b], lse, torch.zeros(2, 600), 1.0, fp8=True,
                        hidden=lambda b: (torch.arange(int(pg.lens[b])) // PAGE == 3) & (b == 1))
    assert ((w.double() - val).abs() <= bound).all()


def test_repeats_streams_and_captures_agree_over_an_fp8_cache():
    pg = Paged([5000, 900, 64, 3000], [3, 200, 1, 7], seed=9)
    q = randn(71, pg.T, 64, ROW, scale=3.0).cuda()
    codes, scale, _ = _codes(pg, 72)
    codes, scale, b = codes.cuda(), scale.cuda(), pg.batch()
    _, lse = dsa.dsa_chunk_attn(b, q, codes, SCALE, kv_scale=scale)
    call = lambda w, **kw: dsa.dsa_attn_weight(b, q, codes, SCALE, lse, w, kv_scale=scale, **kw)  # noqa: E731
    ref = call(torch.zeros(4, 5000, device="cuda"))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ws = [torch.zeros(4, 5000, device="cuda") for _ in range(6)]
    torch.cuda.synchronize()
    for i in range(4):
        call(ws[i], stream=(s1, s2)[i % 2])
    torch.cuda.synchronize()
    graphs = []
    for i in (4, 5):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(ws[i], decay=0.0)
        graphs.append(g)
    for g, s in zip(graphs, (s1, s2)):
        with torch.cuda.stream(s):
            g.replay()
    assert_status_ok()
    assert all(torch.equal(w, ref) for w in ws)
