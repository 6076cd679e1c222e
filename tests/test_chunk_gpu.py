"""dsa_chunk_attn on the GPU against dense causal attention in 64 bits.

Tolerances (per output element, derived below; computed from the reference's own
quantities).  The kernel rounds each weight to bf16 (relative 2^-8) and divides
by the sum of the rounded weights, so with w the exact weights the error of O is
at most  2^-8 (1 + 2^-7) sum_s w_s |v_s - o|  plus what an error of the scores
does: a score off by at most D changes the weights by a factor within exp(+-2D),
which adds (exp(2D) - 1) of the same sum.  A score is a sum of 576 exact products in
fp32, each addition off by at most 2^-23 of the running sum of magnitudes, so
D <= (576 + 8) 2^-23 * scale * sum_i |q_i k_i| (8: the scaling and the subtraction of
the running maximum), with 2^-21 for the exponential.  The value product adds
(n + 8) 2^-23 of sum_s w_s |v_s|, the merge of partial results 130 more of 2^-24
(both kept as (n + 140) 2^-23), and the output is rounded once (2^-8 of it).
Over an FP8 cache the rows are rounded to two fp16 values for the scores (2^-22 of each
value: that much of sum_i |q_i k_i| in D, whose sum has twice the terms), to one for the
output (2^-11 of sum_s w_s |v_s|), and the weights are fp16 and divided by
their sum before rounding: 2^-11 of sum_s w_s |v_s|.  A product w f of a weight and its
page's factor that is subnormal is off by 2^-32 of the largest such product (held near
2^7), and meets v / f < 2^14, where f 2^14 is at most 2.3 times the page's largest
value: 2.3 n 2^-32 of the largest weight times the largest value covers all n.
lse: D + 2^-21, plus (n + 140) 2^-23 for the sum of n weights, plus 2^-22 of itself."""
import math

import numpy as np
import pytest
import torch

import indexer_top_sparse_lightning_b200 as dsa
from tests.paged_helpers import DV, HALF_BF16, PAGE, ROW, Paged, assert_status_ok, fp8_rows, randn

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(ROW)


def reference(pg, q, rows_of, scale=SCALE, hidden=None, fp16=False):
    """Per real token: (out, lse, bound of out's error, bound of lse's); 64 bits on the GPU.
    rows_of(b): the latent rows of sequence b's positions; hidden(b): positions nobody sees;
    fp16: over an FP8 cache."""
    H = q.shape[1]
    res = [[], [], [], []]
    for b in range(pg.B):
        n, L = int(pg.nq[b]), int(pg.lens[b])
        if n == 0:
            continue
        x = rows_of(b).cuda().double()
        t0 = int(pg.cu[b])
        step = max(1, 40_000_000 // (H * L))
        for j in range(0, n, step):
            k = min(step, n - j)
            qq = q[t0 + j:t0 + j + k].cuda().double()
            s = torch.einsum("thd,sd->ths", qq, x) * scale
            mag = torch.einsum("thd,sd->ths", qq.abs(), x.abs()) * scale
            pos = torch.arange(L - n + j, L - n + j + k, device="cuda")
            dark = torch.arange(L, device="cuda")[None] > pos[:, None]
            if hidden is not None:
                dark = dark | hidden(b).cuda()[None]
            s = s.masked_fill(dark[:, None], -math.inf)
            mag = mag.masked_fill(dark[:, None], 0.0)
            lse = torch.logsumexp(s, -1)
            w = (s - lse[..., None]).exp().nan_to_num(0.0)
            v = x[:, :DV]
            o = w @ v
            we, re = (2.0 ** -11, 2.0 ** -11) if fp16 else (2.0 ** -8, 0.0)
            D = ((1152 if fp16 else 576) + 8 + (2 if fp16 else 0)) * 2.0 ** -23 * mag.amax(-1) + 2.0 ** -21
            spread = torch.stack([(w[i, :, :, None] * (v[None] - o[i, :, None]).abs()).sum(1) for i in range(k)]) \
                if k * H * L * DV < 2e8 else (w @ v.abs() + o.abs())      # >= sum w |v - o|
            acc = (L + 140) * 2.0 ** -23
            if fp16:
                bo = torch.expm1(2 * D)[..., None] * spread + (acc + re + we) * (w @ v.abs())
                bo = bo + 2.3 * L * 2.0 ** -32 * w.amax(-1, keepdim=True) * v.abs().amax()
            else:
                bo = (we * (1 + 2 * we) + torch.expm1(2 * D)[..., None]) * spread + acc * (w @ v.abs())
            bo = bo + HALF_BF16 * (o.abs() + bo)
            bl = D + acc + 2.0 ** -22 * lse.abs()
            for r, y in zip(res, (o, lse, bo, bl)):
                r.append(y)
    return [torch.cat(r) for r in res]


def check(pg, out, lse, ref):
    ro, rl, bo, bl = ref
    got, gl = out[:pg.real].double(), lse[:pg.real].double()
    err = (got - ro).abs()
    assert torch.isfinite(got).all()
    assert (err <= bo).all(), f"out: {int((err > bo).sum())} off, worst {float((err / bo).max()):.2f} of the bound"
    dark = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(gl), dark)
    el = (gl - rl).abs()[~dark]
    assert (el <= bl[~dark]).all(), f"lse: worst {float((el / bl[~dark]).max()):.2f} of the bound"


def latent(pg, seed, nan_elsewhere=True):
    """A cache whose rows at the sequences' positions are N(0, 1); all others NaN and infinities."""
    x = randn(seed, pg.num_blocks, PAGE, ROW)
    if nan_elsewhere:
        used = np.concatenate([pg.rows(b) for b in range(pg.B)])
        other = torch.ones(pg.num_blocks * PAGE, dtype=torch.bool)
        other[used] = False
        bad = torch.tensor([math.nan, math.inf, -math.inf], dtype=torch.bfloat16).repeat(ROW // 3)
        x.view(-1, ROW)[other] = bad
    return x


def run(pg, q, kv, **kw):
    out, lse = dsa.dsa_chunk_attn(pg.batch(), q.cuda(), kv.cuda(), SCALE, **kw)
    assert_status_ok()
    return out, lse


SHAPES = [
    ([1], [1], 1), ([64], [1], 16), ([65], [1], 128), ([128], [1], 128), ([129], [3], 128), ([4096], [1], 16),
    ([1000], [1], 128), ([20000], [2], 128), ([9000], [1], 1),
    ([300, 1, 700, 64, 5000], [3, 1, 0, 64, 1], 128), ([300, 1, 700, 64, 5000], [3, 1, 0, 64, 1], 40),
    ([300, 1, 700, 64, 2000], [3, 1, 7, 64, 0], 16), ([513, 90, 1], [200, 90, 1], 7),
    ([257], [257], 16), ([257], [257], 128), ([3000], [513], 64), ([700], [700], 128), ([1500, 40], [600, 40], 96),
    ([2000], [2000], 1),
]


@pytest.mark.parametrize("lens,nq,H", SHAPES)
def test_dense_causal(lens, nq, H):
    pg = Paged(lens, nq, seed=H + len(lens), pad=3)
    q = randn(1 + H, pg.T, H, ROW, scale=3.0)
    kv = latent(pg, 2)
    mark = torch.full((pg.T, H, DV), 5.0, dtype=torch.bfloat16, device="cuda")
    ml = torch.full((pg.T, H), 5.0, device="cuda")
    out, lse = run(pg, q, kv, out=mark, lse=ml)
    check(pg, out, lse, reference(pg, q, lambda b: kv.view(-1, ROW)[pg.rows(b)]))
    assert (out[pg.real:] == 5).all() and (lse[pg.real:] == 5).all()      # padding rows stay


def test_many_sequences():
    # more sequences than threads of a block; many without new tokens
    r = np.random.default_rng(7)
    lens = r.integers(1, 300, size=700)
    nq = np.minimum(lens, r.integers(0, 3, size=700))
    pg = Paged(lens, nq, seed=1)
    q = randn(3, pg.T, 8, ROW, scale=3.0)
    kv = latent(pg, 4)
    out, lse = run(pg, q, kv)
    check(pg, out, lse, reference(pg, q, lambda b: kv.view(-1, ROW)[pg.rows(b)]))


def test_peaked_and_growing_scores():
    # scores that grow along the context by far more than the lazy maximum's 2^8
    pg = Paged([1500], [40], seed=3)
    q = randn(5, pg.T, 128, ROW).abs()
    kv = latent(pg, 6)
    rows = pg.rows(0)
    ramp = torch.linspace(-20, 20, 1500)[:, None]
    kv.view(-1, ROW)[rows] = (randn(7, 1500, ROW).float() * 0.5 + ramp * 0.1).to(torch.bfloat16)
    out, lse = run(pg, q, kv)
    check(pg, out, lse, reference(pg, q, lambda b: kv.view(-1, ROW)[pg.rows(b)]))


@pytest.mark.parametrize("H", [16, 40, 128, 1])
def test_later_tokens_rows_do_not_reach_earlier_ones(H):
    # the last tokens' latent rows are not finite: every token before them must be unaffected
    # (tiles hold several tokens when H < 128), every token that sees one gets no finite result
    n, good = 70, 50
    pg = Paged([400], [n], seed=4)
    q = randn(8, n, H, ROW, scale=3.0)
    kv = latent(pg, 9)
    rows = pg.rows(0)
    bad = torch.tensor([math.nan, math.inf, -math.inf, 1.0], dtype=torch.bfloat16).repeat(ROW // 4)
    kv.view(-1, ROW)[rows[400 - n + good:]] = bad
    out, lse = run(pg, q, kv)
    sub = Paged([400], [n], seed=4)
    clean = kv.clone()
    clean.view(-1, ROW)[rows[400 - n + good:]] = 0
    ro, rl, bo, bl = reference(sub, q, lambda b: clean.view(-1, ROW)[rows])
    assert ((out[:good].double() - ro[:good]).abs() <= bo[:good]).all()
    assert ((lse[:good].double() - rl[:good]).abs() <= bl[:good]).all()
    assert not torch.isfinite(lse[good:]).any()


def test_fp8_latent_cache():
    pg = Paged([500, 3000, 64, 70], [70, 1, 0, 70], seed=5, pad=2)
    q = randn(11, pg.T, 24, ROW, scale=3.0)
    codes, scale, val = fp8_rows(randn(12, pg.num_blocks, PAGE, ROW))
    used = np.zeros(pg.num_blocks * PAGE, bool)
    for b in range(pg.B):
        used[pg.rows(b)] = True
    codes.view(-1, ROW)[~used] = 0x7F                  # NaN codes where nobody looks
    out, lse = run(pg, q, codes, kv_scale=scale.cuda())
    check(pg, out, lse, reference(pg, q, lambda b: val.view(-1, ROW)[pg.rows(b)], fp16=True))


def test_fp8_scales_of_any_size():
    # pages whose scales lie far apart, queries far from 1: the powers of two that keep the fp16
    # operands in range (a tile of zeros among them)
    pg = Paged([700, 130], [3, 65], seed=12)
    q = randn(31, pg.T, 20, ROW)
    q[0] *= 2.0 ** -30
    q[1] *= 2.0 ** 12
    codes, scale, _ = fp8_rows(randn(32, pg.num_blocks, PAGE, ROW))
    for b in range(2):
        for i, page in enumerate(pg.table[b][pg.table[b] >= 0]):
            scale[page] *= 2.0 ** ((-20, 3, 0, -7)[i % 4])
    codes[pg.table[0][0], 3, 128:256] = 0
    val = (codes.view(torch.float8_e4m3fn).double() *
           scale.double().repeat_interleave(128, -1)[..., :ROW])
    out, lse = run(pg, q, codes, kv_scale=scale.cuda())
    check(pg, out, lse, reference(pg, q, lambda b: val.view(-1, ROW)[pg.rows(b)], fp16=True))


@pytest.mark.parametrize("spread", [1, 6, 12])
def test_fp8_scales_that_differ_by_tile(spread):
    # Every tile of every position has its own power of two, 2^-spread .. 2^spread, some are zero.
    # On top of the tolerances above: the last two tiles share an accumulator in units of u, tile
    # 3's scale, or a 64th of the fifth's where that is more than 64 times as large.  There tile 3's
    # codes take a factor rounded to fp16 and are rounded once more (2 * 2^-11 of them); the fifth's
    # factor and rests are fp16 with a smallest step of 2^-24 (off by half of it, and by half of it
    # times the code).  A value is (code f / F) F, F the page's power of two, with f / F in two fp16 parts:
    # off by 2^-25 (|code| + 1) F.
    pg = Paged([517, 130], [3, 65], seed=13)
    q = randn(41, pg.T, 24, ROW)
    codes, scale, _ = fp8_rows(randn(42, pg.num_blocks, PAGE, ROW))
    g = torch.Generator().manual_seed(spread)
    scale *= 2.0 ** torch.randint(-spread, spread + 1, scale.shape, generator=g)
    scale[torch.rand(scale.shape, generator=g) < 0.05] = 0.0
    c, f = codes.view(torch.float8_e4m3fn).double().view(-1, ROW), scale.double().view(-1, 5)
    val = c * f.repeat_interleave(128, -1)[:, :ROW]
    out, lse = run(pg, q, codes, kv_scale=scale.cuda())
    ro, rl, bo, bl = reference(pg, q, lambda b: val[pg.rows(b)], fp16=True)
    used = torch.zeros(len(f), dtype=torch.bool)
    used[np.concatenate([pg.rows(b) for b in range(pg.B)])] = True
    top = (f[:, :4].amax(-1) * used).view(-1, PAGE).amax(-1).repeat_interleave(PAGE)
    F = torch.where(top > 0, 2.0 ** (torch.floor(torch.log2(top.clamp_min(1e-300))) - 6), 1.0)
    big = f[:, 4] > 64 * f[:, 3]
    u = torch.where(big, f[:, 4] / 64, f[:, 3])
    at = 0
    for b in range(pg.B):
        r, n, L = pg.rows(b), int(pg.nq[b]), int(pg.lens[b])
        qq = q[pg.cu[b]:pg.cu[b] + n].double()
        x = val[r]
        dark = torch.arange(L)[None] > torch.arange(L - n, L)[:, None]
        w = (torch.einsum("thd,sd->ths", qq, x) * SCALE).masked_fill(dark[:, None], -math.inf).softmax(-1)
        off = torch.einsum("thd,sd->ths", qq[..., 384:512].abs(), x[:, 384:512].abs() * big[r][:, None]) * 2.0 ** -10 \
            + torch.einsum("thd,sd->ths", qq[..., 512:].abs(), (c[r][:, 512:].abs() + 1) * u[r][:, None]) * 2.0 ** -25
        Dx = (SCALE * off).masked_fill(dark[:, None], 0.0).amax(-1)
        ev = 2.0 ** -25 * (c[r][:, :DV].abs() + 1) * F[r][:, None]
        base = w @ x[:, :DV].abs()
        more = 1.1 * torch.expm1(2 * Dx)[..., None] * (base + ro[at:at + n].abs().cpu()) + w @ ev
        bo[at:at + n] += (more * (1 + 2.0 ** -8)).cuda()
        bl[at:at + n] += Dx.cuda()
        at += n
    check(pg, out, lse, (ro, rl, bo, bl))


def test_offsets_past_32_bits():
    # pages behind the first 4.3 GB (2^31 elements) of the cache
    pg = Paged([300, 1000], [5, 1], seed=6)
    q = randn(13, pg.T, 128, ROW, scale=3.0)
    kv = latent(pg, 14)
    ref = reference(pg, q, lambda b: kv.view(-1, ROW)[pg.rows(b)])
    shift = 2 ** 31 // (PAGE * ROW) + 7
    big = torch.empty(pg.num_blocks + shift, PAGE, ROW, dtype=torch.bfloat16, device="cuda")
    big[shift:] = kv.cuda()
    pg.table[pg.table >= 0] += shift
    pg.num_blocks += shift
    out, lse = dsa.dsa_chunk_attn(pg.batch(), q.cuda(), big, SCALE)
    assert_status_ok()
    check(pg, out, lse, ref)


def test_bad_page_is_reported_and_not_seen():
    pg = Paged([600, 500], [3, 20], seed=8)
    q = randn(15, pg.T, 32, ROW, scale=3.0)
    kv = latent(pg, 16)
    ref = reference(pg, q, lambda b: kv.view(-1, ROW)[pg.rows(b)],
                    hidden=lambda b: (torch.arange(int(pg.lens[b])) // PAGE == 3) if b == 1 else
                    torch.zeros(int(pg.lens[b]), dtype=torch.bool))
    pg.table[1, 3] = pg.num_blocks
    ws = dsa.Workspace()
    out, lse = dsa.dsa_chunk_attn(pg.batch(), q.cuda(), kv.cuda(), SCALE, workspace=ws)
    torch.cuda.synchronize()
    assert dsa.get_status(ws) == 6
    check(pg, out, lse, ref)


def test_repeats_captures_and_streams_agree():
    # bit for bit: twice, from two graphs captured over one set of inputs and replayed at the same
    # time, and on two streams at once
    pg = Paged([5000, 900, 64, 3000], [3, 200, 1, 7], seed=9)
    q, kv = randn(17, pg.T, 64, ROW, scale=3.0).cuda(), latent(pg, 18).cuda()
    b = pg.batch()
    ref, rl = dsa.dsa_chunk_attn(b, q, kv, SCALE)
    again, al = dsa.dsa_chunk_attn(b, q, kv, SCALE)
    assert torch.equal(ref, again) and torch.equal(rl, al)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [dsa.dsa_chunk_attn(b, q, kv, SCALE, stream=s) for _ in range(4) for s in (s1, s2)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) and torch.equal(l, rl) for o, l in outs)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = dsa.dsa_chunk_attn(b, q, kv, SCALE)
        graphs.append((g, res))
    for (g, _), s in zip(graphs, (s1, s2)):
        with torch.cuda.stream(s):
            g.replay()
    assert_status_ok()
    for _, (o, l) in graphs:
        assert torch.equal(o, ref) and torch.equal(l, rl)
    q.mul_(0.5)
    new, _ = dsa.dsa_chunk_attn(b, q, kv, SCALE)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1][0], new)


def test_same_as_sparse_attention_over_every_position():
    # the framework's sparse attention with every position selected is the same sum
    pg = Paged([700, 64], [1, 1], seed=10)
    q, kv = randn(19, pg.T, 128, ROW, scale=3.0), latent(pg, 20, nan_elsewhere=False)
    idx = np.full((2, 1024), -1, np.int32)
    for b in range(2):
        idx[b, :pg.lens[b]] = np.arange(pg.lens[b])
    so, sl = dsa.sparse_mla_attn(pg.batch(), q.cuda(), kv.cuda(), torch.from_numpy(idx).cuda(), SCALE)
    ref = reference(pg, q, lambda b: kv.view(-1, ROW)[pg.rows(b)])
    out, lse = run(pg, q, kv)
    check(pg, out, lse, ref)
    # two results, each within the bound (the merge of the sparse kernel rounds its parts once more)
    assert ((out.double() - so.double()).abs() <= 2 * ref[2] + 2 * HALF_BF16 * ref[0].abs()).all()


def test_timeout_is_reported_and_recoverable():
    pg = Paged([3000], [4], seed=11)
    q, kv = randn(21, pg.T, 128, ROW).cuda(), latent(pg, 22).cuda()
    ws = dsa.Workspace()
    clean, _ = dsa.dsa_chunk_attn(pg.batch(), q, kv, SCALE, workspace=ws)
    assert dsa.get_status(ws) == 0
    words = ws.buf[:16].view(torch.int32)
    words[1], words[2] = 5000, 4
    dsa.dsa_chunk_attn(pg.batch(), q, kv, SCALE, workspace=ws)
    assert dsa.get_status(ws) == 5                     # DSA_ERR_TIMEOUT
    ws.reset()
    again, _ = dsa.dsa_chunk_attn(pg.batch(), q, kv, SCALE, workspace=ws)
    assert dsa.get_status(ws) == 0 and torch.equal(clean, again)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_length_below_the_new_tokens_is_reported(fp8):
    # token j stands at seq_lens - nq + j: the first tokens of such a sequence stand in front of its start and
    # see nothing, their rows stay as they were; the others are attended to as ever
    n, L, H = 90, 70, 24
    pg = Paged([300, n, 64], [5, n, 1], seed=12)
    q = randn(41, pg.T, H, ROW, scale=3.0)
    kv, kw = latent(pg, 42, nan_elsewhere=False), {}
    if fp8:
        kv, scale, val = fp8_rows(kv)
        kw = dict(kv_scale=scale.cuda())
    else:
        val = kv
    pg.lens[1] = L
    ws = dsa.Workspace()
    out = torch.full((pg.T, H, DV), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((pg.T, H), 5.0, device="cuda")
    dsa.dsa_chunk_attn(pg.batch(), q.cuda(), kv.cuda(), SCALE, out=out, lse=lse, workspace=ws, **kw)
    assert dsa.get_status(ws) == 6
    cut = Paged([300, n, 64], [5, n, 1], seed=12)              # the tokens that stand in the sequence
    cut.lens[1], cut.nq[1] = L, L
    cut.cu = np.array([0, 5, 5 + L, 6 + L], np.int32)
    cut.real = cut.T = 6 + L
    keep = torch.tensor([t for t in range(pg.T) if not 5 <= t < 5 + n - L])
    check(cut, out[keep.cuda()], lse[keep.cuda()],
          reference(cut, q[keep], lambda b: val.view(-1, ROW)[cut.rows(b)], fp16=fp8))
    assert (out[5:5 + n - L] == 5).all() and (lse[5:5 + n - L] == 5).all()


def test_more_new_tokens_than_rows_are_reported():
    # a cu_q that goes past the queries: the rows that are there keep their tokens' positions
    lens, nq, H, gone = [300, 400, 64], [5, 90, 3], 24, 50
    pg = Paged(lens, nq, seed=13)
    q, kv = randn(51, pg.T, H, ROW, scale=3.0), latent(pg, 52)
    ref = [r[:pg.T - gone] for r in reference(pg, q, lambda b: kv.view(-1, ROW)[pg.rows(b)])]
    ws = dsa.Workspace()
    out, lse = dsa.dsa_chunk_attn(pg.batch(), q[:pg.T - gone].cuda(), kv.cuda(), SCALE, workspace=ws)
    assert dsa.get_status(ws) == 6
    pg.real = pg.T - gone
    check(pg, out, lse, ref)
