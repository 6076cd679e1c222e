"""The operators around the sparse attention as they are used together: a prompt is written to the
caches and attended to densely, its weights are accumulated over the prompt and two decode steps,
the caches are cut by them, and decoding goes on, dense and sparse, over the kept positions."""
import math

import numpy as np
import pytest
import torch

import indexer_top_sparse_lightning_b200 as dsa
from tests.paged_helpers import HALF_BF16, PAGE, ROW, Paged, assert_status_ok, randn
from tests.test_chunk_gpu import SCALE, check, reference
from tests.test_evict_gpu import choose
from tests.test_rope_gpu import _assert_bf16, _formula, _freq
from tests.test_weight_gpu import expect

pytestmark = pytest.mark.gpu

H = 16


def _step(pg, freq, gamma, q, k, cache, weight, positions=None):
    """One step of a serving loop: rotate and write, attend, accumulate."""
    b = pg.batch()
    qr = dsa.dsa_qk_norm_rope(b, freq, q, k, k_gamma=gamma, interleaved=True, k_cache=cache, positions=positions)
    out, lse = dsa.dsa_chunk_attn(b, qr, cache, SCALE)
    dsa.dsa_attn_weight(b, qr, cache, SCALE, lse, weight, decay=0.75)
    return qr, out, lse


def test_prompt_decode_evict_decode():
    lens = np.array([700, 333, 64])
    full = Paged(lens + 3, lens * 0 + 1, seed=1, spare=40)          # pages for the prompt and three more tokens
    freq, gamma = _freq(64).cuda(), (torch.rand(512) + 0.5).cuda()
    cache = torch.zeros(full.num_blocks, PAGE, ROW, dtype=torch.bfloat16, device="cuda")
    keys = torch.randn(full.num_blocks, PAGE, 128, device="cuda").to(torch.bfloat16)
    weight = torch.zeros(3, 768, device="cuda")
    ref_w = torch.zeros(3, 768, dtype=torch.float64)
    ref_b = torch.zeros(3, 768, dtype=torch.float64)

    def at(length, nq):
        pg = Paged(length, nq, seed=1, spare=0)
        pg.table, pg.num_blocks = full.table, full.num_blocks
        return pg

    for i, (length, nq) in enumerate([(lens, lens), (lens + 1, [1, 1, 1]), (lens + 2, [1, 1, 1])]):
        pg = at(length, nq)
        q, k = randn(10 + i, pg.T, H, ROW, scale=2.0), randn(20 + i, pg.T, ROW, scale=2.0)
        qr, out, lse = _step(pg, freq, gamma, q.cuda(), k.cuda(), cache, weight)
        assert_status_ok()
        seq, pos = pg.seq_pos()
        _assert_bf16(qr, *_formula(q, None, 0, np.ascontiguousarray(np.broadcast_to(pos[:, None], (pg.T, H))), _freq(64), 512, True))
        written = np.concatenate([pg.rows(b)[pg.lens[b] - pg.nq[b]:] for b in range(3)])
        c = cache.cpu()
        _assert_bf16(c.view(-1, ROW)[written], *_formula(k, gamma.cpu(), 1e-6, pos, _freq(64), 512, True))
        check(pg, out, lse, reference(pg, qr.cpu(), lambda b: c.view(-1, ROW)[pg.rows(b)]))
        val, bound = expect(pg, qr.cpu(), lambda b: c.view(-1, ROW)[pg.rows(b)], lse, ref_w.float() * 0, 0.75)
        for b in range(3):
            L = int(pg.lens[b])
            ref_w[b, :L] = 0.75 * ref_w[b, :L] + val[b, :L].cpu()
            ref_b[b, :L] = 0.75 * ref_b[b, :L] + bound[b, :L].cpu() + 2.0 ** -22 * ref_w[b, :L]
    assert ((weight.cpu().double() - ref_w).abs() <= ref_b).all()

    # cut to 128 positions, into free pages of the same caches
    keep, pg = 128, at(lens + 2, [1, 1, 1])
    table = torch.from_numpy(full.free[:12].reshape(3, 4).copy()).cuda()
    new_weight = torch.zeros(3, 192, device="cuda")
    idx, count = dsa.dsa_cache_evict(pg.batch(), weight, keep, table, [cache, keys], [cache, keys], sink=4, recent=16,
                                     new_weight=new_weight)
    assert_status_ok()
    w = weight.cpu().numpy()
    kept = [choose(w[b], int(pg.lens[b]), keep, 4, 16) for b in range(3)]
    for b in range(3):
        assert int(count[b]) == len(kept[b])
        np.testing.assert_array_equal(idx[b, :len(kept[b])].cpu().numpy(), kept[b])

    # decoding goes on behind the kept rows: the token's place in the text is no longer its place in the cache
    small = Paged(np.array([len(x) for x in kept]) + 1, [1, 1, 1], seed=1, spare=0)
    small.table, small.num_blocks = table.cpu().numpy(), full.num_blocks
    q, k = randn(31, 3, H, ROW, scale=2.0), randn(32, 3, ROW, scale=2.0)
    text = torch.from_numpy((lens + 2).astype(np.int32))
    before = cache.clone()
    qr, out, lse = _step(small, freq, gamma, q.cuda(), k.cuda(), cache, new_weight, positions=text.cuda())
    assert_status_ok()
    _assert_bf16(qr, *_formula(q, None, 0, text.long().numpy()[:, None].repeat(H, 1), _freq(64), 512, True))
    c = cache.cpu()
    for b in range(3):          # the kept rows are the old ones, the new row follows them
        rows = small.rows(b)
        assert torch.equal(c.view(-1, ROW)[rows[:-1]], before.cpu().view(-1, ROW)[pg.rows(b)[kept[b]]])
        _assert_bf16(c.view(-1, ROW)[rows[-1:]], *_formula(k[b:b + 1], gamma.cpu(), 1e-6, text[b:b + 1].long().numpy(), _freq(64), 512, True))
    ref = reference(small, qr.cpu(), lambda b: c.view(-1, ROW)[small.rows(b)])
    check(small, out, lse, ref)
    # ... and the framework's own sparse attention reads the same pages
    sel = np.full((3, 192), -1, np.int32)
    for b in range(3):
        sel[b, :small.lens[b]] = np.arange(small.lens[b])
    so, sl = dsa.sparse_mla_attn(small.batch(), qr, cache, torch.from_numpy(sel).cuda(), SCALE)
    torch.cuda.synchronize()
    assert dsa.get_status() == 0
    assert ((out.double() - so.double()).abs() <= 2 * ref[2] + 2 * HALF_BF16 * ref[0].abs()).all()


def test_a_decode_step_captured_in_a_graph():
    # rotation, attention and weights of one decode step, captured once and replayed on new inputs
    pg = Paged([900, 64, 2000, 1], [1, 1, 1, 1], seed=3)
    freq, gamma = _freq(64).cuda(), torch.ones(512, device="cuda")
    cache = randn(41, pg.num_blocks, PAGE, ROW).cuda()
    start = cache.clone()
    weight = torch.zeros(4, 2048, device="cuda")
    q, k = randn(42, 4, H, ROW, scale=2.0).cuda(), randn(43, 4, ROW).cuda()
    b = pg.batch()

    def step():
        qr = dsa.dsa_qk_norm_rope(b, freq, q, k, k_gamma=gamma, k_cache=cache)
        out, lse = dsa.dsa_chunk_attn(b, qr, cache, SCALE)
        dsa.dsa_attn_weight(b, qr, cache, SCALE, lse, weight, decay=0.0)
        return out, lse

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for seed in (51, 52):
        q.copy_(randn(seed, 4, H, ROW, scale=2.0))
        k.copy_(randn(seed + 10, 4, ROW))
        cache.copy_(start)
        g.replay()
        torch.cuda.synchronize()
        w = weight.clone()
        out, lse = (t.clone() for t in got)
        cache.copy_(start)
        weight.zero_()
        want = step()
        assert_status_ok()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(w, weight)


def test_a_fresh_workspace_is_made_on_the_call_s_stream():
    # its zeros must be there before the kernels look at the area, whatever stream they run on
    pg = Paged([200], [1], seed=3)
    q, kv = randn(1, pg.T, 16, ROW).cuda(), randn(2, pg.num_blocks, PAGE, ROW).cuda()
    torch.cuda.synchronize()
    side, ws = torch.cuda.Stream(), dsa.Workspace(torch.device("cuda"))
    made = []
    get = ws.get
    ws.get = lambda n: (made.append(torch.cuda.current_stream()), get(n))[1]
    dsa.dsa_chunk_attn(pg.batch(), q, kv, 0.05, workspace=ws, stream=side)
    torch.cuda.synchronize()
    assert made[0] == side and dsa.get_status(ws) == 0


def test_a_capture_does_not_make_the_status_area(monkeypatch):
    monkeypatch.setattr(dsa, "_status_ws", {})
    pg = Paged([200], [1], seed=3)
    q, kv = randn(1, pg.T, 16, ROW).cuda(), randn(2, pg.num_blocks, PAGE, ROW).cuda()
    b, g = pg.batch(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(RuntimeError, match="status_workspace"):
            dsa.dsa_chunk_attn(b, q, kv, 0.05)
        q.add_(0)
    dsa.status_workspace()
    dsa.dsa_chunk_attn(b, q, kv, 0.05)
    assert_status_ok()
