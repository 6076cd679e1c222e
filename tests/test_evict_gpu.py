"""dsa_cache_evict on the GPU: choices and copies are exact, so they are compared bit by bit
with a sort on the CPU."""
import math

import numpy as np
import pytest
import torch

import indexer_top_sparse_lightning_b200 as dsa
from tests.paged_helpers import PAGE, Paged, assert_status_ok

pytestmark = pytest.mark.gpu


def choose(w, L, keep, sink, recent):
    """Positions that stay, ascending."""
    if L <= keep:
        return np.arange(L)
    x = np.where(np.isnan(w[:L]), -np.inf, w[:L].astype(np.float64)) + 0.0
    nan = np.isnan(w[:L])
    held = np.zeros(L, bool)
    held[:sink] = True
    if recent:
        held[L - recent:] = True
    # held first, then by weight (NaN behind everything), then by position
    order = np.lexsort((np.arange(L), -x, nan & ~held, ~held))
    order = np.concatenate([order[held[order]], order[~held[order]]])
    return np.sort(order[:keep])


class NewPages:
    def __init__(self, B, rows, seed, spare=3):
        n = max(1, -(-rows // PAGE))
        ids = np.random.default_rng(seed).permutation(B * n + spare).astype(np.int32)
        self.table, self.num_blocks = ids[:B * n].reshape(B, n), B * n + spare

    def rows(self, b, k):
        j = np.arange(k)
        return self.table[b, j // PAGE].astype(np.int64) * PAGE + j % PAGE


def weights(B, n, seed, kind="mixed"):
    r = np.random.default_rng(seed)
    w = r.standard_normal((B, n)).astype(np.float32)
    if kind == "mixed":            # heavy tails, many zeros of both signs
        w = np.exp(2 * w)
        w[r.random((B, n)) < 0.4] = 0.0
        w[r.random((B, n)) < 0.1] = -0.0
    elif kind == "ties":
        w = np.floor(w * 2).astype(np.float32)
    elif kind == "odd":            # everything a float can hold
        w = r.integers(0, 2 ** 32, (B, n), dtype=np.uint64).astype(np.uint32).view(np.float32).copy()
        w[r.random((B, n)) < 0.2] = np.nan
        w[r.random((B, n)) < 0.1] = np.inf
        w[r.random((B, n)) < 0.1] = -np.inf
    return w


ARRAYS = [((64, 576), torch.bfloat16), ((64, 576), torch.uint8), ((64, 5), torch.float32), ((64, 128), torch.bfloat16),
          ((64, 2), torch.uint8), ((64, 3), torch.uint8)]


def check(lens, keep, sink, recent, kind="mixed", seed=0, arrays=ARRAYS, stride=None):
    pg = Paged(lens, [1] * len(lens), seed=seed)
    w = weights(pg.B, stride or int(pg.lens.max()), seed + 1, kind)
    g = torch.Generator().manual_seed(seed + 2)
    old = [torch.randint(0, 250, (pg.num_blocks, *s, 4 if d == torch.float32 else 1), generator=g, dtype=torch.uint8)
           for s, d in arrays]
    old = [o.view(d).squeeze(-1) if d == torch.float32 else o.squeeze(-1).to(d) for o, (s, d) in zip(old, arrays)]
    most = min(keep, int(pg.lens.max()))
    pages = NewPages(pg.B, most, seed + 3)
    new = [torch.full((pages.num_blocks, *s), 7, dtype=d) for s, d in arrays]
    dev_new = [t.cuda() for t in new]
    nw = torch.full((pg.B, most + 3), -5.0, device="cuda")
    idx, count = dsa.dsa_cache_evict(pg.batch(), torch.from_numpy(w).cuda(), keep, torch.from_numpy(pages.table).cuda(),
                                     [o.cuda() for o in old], dev_new, sink=sink, recent=recent, new_weight=nw)
    assert_status_ok()
    idx, count, nw = idx.cpu().numpy(), count.cpu().numpy(), nw.cpu().numpy()
    for b in range(pg.B):
        want = choose(w[b], int(pg.lens[b]), keep, sink, recent)
        assert count[b] == len(want)
        np.testing.assert_array_equal(idx[b, :len(want)], want)
        assert (idx[b, len(want):] == -1).all()
        np.testing.assert_array_equal(nw[b, :len(want)].view(np.uint32), w[b][want].view(np.uint32))
        assert (nw[b, len(want):] == -5.0).all()
        src, dst = pg.rows(b)[want], pages.rows(b, len(want))
        for o, n in zip(old, new):
            n.view(-1, n.shape[-1])[dst] = o.view(-1, o.shape[-1])[src]
    for n, d in zip(new, dev_new):                 # kept rows, and nothing else
        assert torch.equal(n.view(torch.uint8), d.cpu().view(torch.uint8))


@pytest.mark.parametrize("lens,keep,sink,recent", [
    ([1], 1, 0, 0), ([2], 1, 0, 0), ([2], 1, 0, 1), ([2], 1, 1, 0), ([64], 64, 0, 0), ([65], 64, 0, 0), ([63], 64, 3, 3),
    ([500, 3, 64, 1000], 100, 0, 0), ([500, 3, 64, 1000], 100, 4, 32), ([500, 90], 100, 50, 50),
    ([9000, 20000, 16384], 3000, 4, 512), ([40000, 100], 39999, 1, 1), ([33000], 1, 0, 0),
])
@pytest.mark.parametrize("kind", ["mixed", "ties", "odd"])
def test_choice_and_copies(lens, keep, sink, recent, kind):
    check(lens, keep, sink, recent, kind, seed=len(lens) + keep)


def test_weights_all_equal_keep_the_lowest_positions():
    pg = Paged([5000], [1], seed=1)
    w = torch.zeros(1, 5000, device="cuda")
    idx, _ = dsa.dsa_cache_evict(pg.batch(), w, 777, torch.zeros(1, 13, dtype=torch.int32, device="cuda"), [], [], recent=10)
    assert_status_ok()
    want = np.concatenate([np.arange(767), np.arange(4990, 5000)])
    np.testing.assert_array_equal(idx[0].cpu().numpy(), want)


def test_ranges_longer_than_shared_memory():
    check([500000, 370000, 17], 60000, 16, 4096, "mixed", seed=9, arrays=ARRAYS[1:3])
    check([450000], 449000, 0, 0, "ties", seed=10, arrays=ARRAYS[4:5])


def test_many_sequences():
    r = np.random.default_rng(11)
    check(r.integers(1, 400, size=700).tolist(), 90, 2, 5, "ties", seed=12, arrays=ARRAYS[3:5])


def test_into_free_pages_of_the_same_cache():
    pg = Paged([300, 200], [1, 1], seed=13, spare=6)
    cache = torch.randn(pg.num_blocks, PAGE, 576).to(torch.bfloat16)
    w = weights(2, 300, 14)
    table = pg.free[:4].reshape(2, 2)
    dev = cache.cuda()
    idx, count = dsa.dsa_cache_evict(pg.batch(), torch.from_numpy(w).cuda(), 100, torch.from_numpy(table.copy()).cuda(), [dev], [dev])
    assert_status_ok()
    for b in range(2):
        want = choose(w[b], int(pg.lens[b]), 100, 0, 0)
        j = np.arange(100)
        cache.view(-1, 576)[table[b, j // PAGE].astype(np.int64) * PAGE + j % PAGE] = cache.view(-1, 576)[pg.rows(b)[want]].clone()
    assert torch.equal(dev.cpu(), cache)


def test_bad_pages_are_reported_and_skipped():
    pg = Paged([300], [1], seed=15)
    cache = torch.randn(pg.num_blocks, PAGE, 576).to(torch.bfloat16).cuda()
    new = torch.zeros(3, PAGE, 576, dtype=torch.bfloat16, device="cuda")
    w = torch.arange(300, dtype=torch.float32, device="cuda").view(1, 300)
    ws = dsa.Workspace()
    dsa.dsa_cache_evict(pg.batch(), w, 128, torch.tensor([[1, 3]], dtype=torch.int32, device="cuda"), [cache], [new], workspace=ws)
    assert dsa.get_status(ws) == 6
    assert (new[1] != 0).any(-1).all() and (new[[0, 2]] == 0).all()
    good = pg.table.copy()
    pg.table[0, 3] = -1
    new.zero_()
    dsa.dsa_cache_evict(pg.batch(), w, 128, torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"), [cache], [new], workspace=ws)
    assert dsa.get_status(ws) == 6
    kept = np.arange(172, 300)
    want = torch.zeros(128, 576, dtype=torch.bfloat16)
    rows = cache.cpu().view(-1, 576)[good[0, kept // PAGE].astype(np.int64) * PAGE + kept % PAGE]
    fine = torch.from_numpy(kept // PAGE != 3)
    want[fine] = rows[fine]
    assert torch.equal(torch.cat([new[1], new[0]]).cpu(), want)


def test_captured_and_on_another_stream():
    pg = Paged([9000, 700], [1, 1], seed=16)
    w = torch.from_numpy(weights(2, 9000, 17)).cuda()
    cache = torch.randn(pg.num_blocks, PAGE, 128).to(torch.bfloat16).cuda()
    pages = NewPages(2, 500, 18)
    table, b = torch.from_numpy(pages.table).cuda(), pg.batch()
    new = [torch.zeros(pages.num_blocks, PAGE, 128, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    idx, count = dsa.dsa_cache_evict(b, w, 500, table, [cache], new[:1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    idx2, _ = dsa.dsa_cache_evict(b, w, 500, table, [cache], new[1:2], stream=side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        idx3, _ = dsa.dsa_cache_evict(b, w, 500, table, [cache], new[2:])
    g.replay()
    assert_status_ok()
    assert torch.equal(idx, idx2) and torch.equal(idx, idx3)
    assert torch.equal(new[0], new[1]) and torch.equal(new[0], new[2])


def test_refusals():
    pg = Paged([300], [1], seed=19)
    b = pg.batch()
    w = torch.zeros(1, 300, device="cuda")
    t = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    for bad in (dict(keep=0), dict(keep=100, sink=-1), dict(keep=100, sink=60, recent=41), dict(keep=129)):
        with pytest.raises((dsa.DsaError, ValueError)):
            dsa.dsa_cache_evict(b, w, bad.pop("keep"), t, [], [], **bad)
    with pytest.raises(dsa.DsaError):
        dsa.dsa_cache_evict(b, w, 100, t, [], [], new_weight=w)
    with pytest.raises(dsa.DsaError):
        dsa.dsa_cache_evict(b, w[:, :200].contiguous(), 100, t, [], [])
    with pytest.raises(ValueError):
        dsa.dsa_cache_evict(b, w, 100, t, [torch.zeros(1, 64, 4, device="cuda")], [torch.zeros(2, 64, 4, device="cuda")])


def test_long_sequences_in_turns():
    # more long sequences than groups of CTAs, some short ones among them
    r = np.random.default_rng(21)
    lens = [70000 if i % 3 else 900 for i in range(40)]
    lens[5] = 69999
    check(lens, 2000, 4, 64, "ties", seed=22, arrays=ARRAYS[4:5])


def test_long_sequences_captured_and_on_two_streams():
    pg = Paged([300000, 200], [1, 1], seed=23)
    w = torch.from_numpy(weights(2, 300000, 24)).cuda()
    b = pg.batch()
    table = torch.zeros(2, 160, dtype=torch.int32, device="cuda")
    call = lambda **kw: dsa.dsa_cache_evict(b, w, 10000, table, [], [], sink=3, **kw)[0]  # noqa: E731
    idx = call()
    np.testing.assert_array_equal(idx[0].cpu().numpy(), choose(w[0].cpu().numpy(), 300000, 10000, 3, 0))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    many = [call(stream=s) for _ in range(10) for s in (s1, s2)]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, call()))
    for (g, _), s in zip(graphs, (s1, s2)):
        with torch.cuda.stream(s):
            for _ in range(5):
                g.replay()
    assert_status_ok()
    assert all(torch.equal(idx, x) for x in many + [x for _, x in graphs])


@pytest.mark.parametrize("L", [300, 70000])
def test_without_arrays_no_page_is_looked_at(L):
    # the new weights alone: ids of a larger pool, or of no page at all, are nobody's concern
    pg = Paged([L], [1], seed=25)
    w = torch.from_numpy(weights(1, L, 26)).cuda()
    b, ws = pg.batch(), dsa.Workspace()
    table = torch.tensor([[7, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    new = torch.full((1, 128), -5.0, device="cuda")
    idx, _ = dsa.dsa_cache_evict(b, w, 128, table, [], [], new_weight=new, workspace=ws)
    assert dsa.get_status(ws) == 0
    want = choose(w[0].cpu().numpy(), L, 128, 0, 0)
    np.testing.assert_array_equal(idx[0].cpu().numpy(), want)
    assert torch.equal(new[0].cpu(), w[0].cpu()[torch.from_numpy(want)])


def test_a_count_that_32_bits_would_wrap_is_refused():
    pg = Paged([300], [1], seed=27)
    w, t = torch.zeros(1, 300, device="cuda"), torch.zeros(1, 5, dtype=torch.int32, device="cuda")
    idx = torch.empty(1, 4, dtype=torch.int32, device="cuda")
    for keep in (2 ** 32 + 4, 2 ** 31):
        with pytest.raises(ValueError, match="keep"):
            dsa.dsa_cache_evict(pg.batch(), w, keep, t, [], [], out_idx=idx)
