"""Host-side refusals of the operators around the sparse attention: bad arguments
return a code before anything is launched (no GPU needed)."""
import ctypes

import pytest

import indexer_top_sparse_lightning_b200 as dsa
from indexer_top_sparse_lightning_b200 import build

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return dsa.load_library()


def _batch(**kw):
    b = dict(batch=1, num_tokens=1, seq_lens=8, cu_q=8, block_table=8, max_blocks_per_seq=1, num_blocks=1,
             max_seq_len=64, max_q_per_seq=1)
    b.update(kw)
    return dsa._Batch(**b)


def _rope(**kw):
    d = dict(q=16, q_stride_t=2 * 576, q_stride_h=576, k=16, k_stride_t=576, H=2, D=576, q_gamma=None, k_gamma=16,
             q_norm=0, k_norm=512, eps=1e-6, inv_freq=16, rope_dim=64, rope_off=512, interleaved=0, positions=None,
             kv_dtype=0)
    d.update(kw)
    return dsa._Rope(**d)


def _call_rope(lib, batch=None, q_out=32, k_cache=16, k_scale=None, status=256, **kw):
    return lib.dsa_qk_norm_rope(ctypes.byref(batch if batch is not None else _batch()), ctypes.byref(_rope(**kw)),
                                q_out, k_cache, k_scale, status, None)


@pytest.mark.parametrize("bad,code", [
    (dict(q=None, k=None), INVALID), (dict(D=572), UNSUPPORTED), (dict(D=1032), UNSUPPORTED), (dict(D=0), UNSUPPORTED),
    (dict(rope_dim=24), UNSUPPORTED), (dict(rope_dim=-16), UNSUPPORTED), (dict(rope_off=4), UNSUPPORTED),
    (dict(rope_off=-8), UNSUPPORTED), (dict(rope_off=520), INVALID), (dict(inv_freq=None), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(H=0), INVALID), (dict(q=8), INVALID),
    (dict(k=8), INVALID), (dict(q_stride_t=4), INVALID), (dict(q_stride_h=-576), INVALID), (dict(k_stride_t=3), INVALID),
    (dict(k_norm=520), INVALID), (dict(k_norm=584), INVALID), (dict(k_norm=12), INVALID), (dict(k_gamma=None), INVALID),
    (dict(k_gamma=20), INVALID), (dict(q_norm=512), INVALID), (dict(kv_dtype=2), INVALID),
])
def test_rope_rejects_bad_inputs(lib, bad, code):
    if bad == dict(k_norm=520):
        bad = dict(k_norm=520, D=512, rope_off=448)     # more elements than the row has
    assert _call_rope(lib, **bad) == code


@pytest.mark.parametrize("bad", [dict(q_out=None), dict(q_out=24), dict(k_cache=None), dict(k_cache=8),
                                 dict(status=None), dict(kv_dtype=1), dict(kv_dtype=1, k_scale=18)])
def test_rope_rejects_bad_outputs(lib, bad):
    assert _call_rope(lib, **bad) == INVALID


def test_rope_rejects_fp8_rows_of_another_width(lib):
    assert _call_rope(lib, kv_dtype=1, k_scale=16, D=128, k_norm=128, rope_off=64) == UNSUPPORTED


def test_rope_rejects_in_place_on_strided_queries(lib):
    assert _call_rope(lib, q=32, q_stride_t=3 * 576) == INVALID


@pytest.mark.parametrize("bad", [dict(batch=0), dict(num_tokens=0), dict(seq_lens=None), dict(cu_q=None),
                                 dict(block_table=None), dict(num_blocks=0), dict(max_blocks_per_seq=0)])
def test_rope_rejects_bad_batch(lib, bad):
    assert _call_rope(lib, batch=_batch(**bad)) == INVALID


def _attn(**kw):
    d = dict(q=16, kv_cache=16, H=128, sm_scale=0.04, kv_dtype=0, kv_scale=None)
    d.update(kw)
    return dsa._Attn(**d)


def _call_chunk(lib, batch=None, out=16, lse=None, status=256, scratch=256, nbytes=1 << 40, **kw):
    return lib.dsa_chunk_attn(ctypes.byref(batch if batch is not None else _batch()), ctypes.byref(_attn(**kw)), out, lse,
                              status, scratch, nbytes, None)


def _call_weight(lib, batch=None, lse=16, weight=16, stride=64, decay=1.0, status=256, scratch=256, nbytes=1 << 40, **kw):
    return lib.dsa_attn_weight(ctypes.byref(batch if batch is not None else _batch()), ctypes.byref(_attn(**kw)), lse, weight,
                               stride, decay, status, scratch, nbytes, None)


BAD_ATTN = [(dict(H=0), UNSUPPORTED), (dict(H=129), UNSUPPORTED), (dict(q=None), INVALID), (dict(q=8), INVALID),
            (dict(kv_cache=None), INVALID), (dict(sm_scale=0.0), INVALID), (dict(sm_scale=float("nan")), INVALID),
            (dict(kv_dtype=2), INVALID), (dict(kv_dtype=1), INVALID), (dict(kv_dtype=1, kv_scale=18), INVALID)]
BAD_BATCH = [dict(batch=0), dict(num_tokens=0), dict(seq_lens=None), dict(cu_q=None), dict(block_table=None),
             dict(num_blocks=0), dict(max_seq_len=65), dict(max_seq_len=0), dict(max_q_per_seq=0)]


@pytest.mark.parametrize("bad,code", BAD_ATTN)
def test_dense_operators_reject_bad_inputs(lib, bad, code):
    assert _call_chunk(lib, **bad) == code
    assert _call_weight(lib, **bad) == code
    assert lib.dsa_chunk_scratch_size(ctypes.byref(_batch()), ctypes.byref(_attn(**bad))) == 0
    assert lib.dsa_weight_scratch_size(ctypes.byref(_batch()), ctypes.byref(_attn(**bad))) == 0


@pytest.mark.parametrize("bad", BAD_BATCH)
def test_dense_operators_reject_bad_batches(lib, bad):
    assert _call_chunk(lib, batch=_batch(**bad)) == INVALID
    assert _call_weight(lib, batch=_batch(**bad)) == INVALID
    assert _call_evict(lib, batch=_batch(**bad)) == INVALID
    assert lib.dsa_evict_scratch_size(ctypes.byref(_batch(**bad))) == 0


def test_dense_operators_reject_more_rows_than_32_bits_count(lib):
    many = _batch(num_tokens=2 ** 24)
    assert _call_chunk(lib, batch=many) == UNSUPPORTED
    assert _call_weight(lib, batch=many) == UNSUPPORTED


def _call_evict(lib, batch=None, idx=16, length=16, status=256, scratch=256, nbytes=1 << 40, arrays=None, **kw):
    rows = (dsa._CacheArray * 16)(*(arrays or [(16, 16, 1152)]))
    d = dict(weight=16, weight_stride=64, new_weight=None, new_weight_stride=0, keep=32, sink=0, recent=0, new_table=16,
             new_max_blocks=1, new_num_blocks=1, arrays=rows, n_arrays=len(arrays or [1]))
    d.update(kw)
    return lib.dsa_cache_evict(ctypes.byref(batch if batch is not None else _batch()), ctypes.byref(dsa._Evict(**d)), idx, length,
                               status, scratch, nbytes, None)


@pytest.mark.parametrize("bad,code", [
    (dict(weight=None), INVALID), (dict(weight_stride=63), INVALID), (dict(keep=0), INVALID), (dict(sink=-1), INVALID),
    (dict(recent=-1), INVALID), (dict(sink=16, recent=17), INVALID), (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), INVALID),
    (dict(new_table=None), INVALID), (dict(new_max_blocks=0), INVALID), (dict(new_num_blocks=0), INVALID),
    (dict(new_weight=32, new_weight_stride=31), INVALID), (dict(new_weight=16, new_weight_stride=64), INVALID),
    (dict(n_arrays=-1), INVALID), (dict(n_arrays=9), UNSUPPORTED), (dict(idx=None), INVALID), (dict(length=None), INVALID),
    (dict(status=None), INVALID), (dict(arrays=[(None, 16, 1152)]), INVALID), (dict(arrays=[(16, None, 1152)]), INVALID),
    (dict(arrays=[(16, 16, 0)]), INVALID), (dict(arrays=[(16, 16, 2049)]), UNSUPPORTED),
])
def test_evict_rejects_bad_inputs(lib, bad, code):
    assert _call_evict(lib, **bad) == code


def test_python_entry_points_want_cuda_tensors():
    import torch
    t = torch.zeros(1, dtype=torch.int32)
    b = dsa.Batch(t, torch.zeros(2, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32), 1, 1, 1)
    q, kv = torch.zeros(1, 2, 576, dtype=torch.bfloat16), torch.zeros(1, 64, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dsa.dsa_qk_norm_rope(b, None, q)
    with pytest.raises(ValueError):
        dsa.dsa_qk_norm_rope(b, None)
    with pytest.raises(ValueError):
        dsa.dsa_chunk_attn(b, q, kv, 0.04)
    with pytest.raises(ValueError):
        dsa.dsa_attn_weight(b, q, kv, 0.04, torch.zeros(1, 2), torch.zeros(1, 1))
    with pytest.raises(ValueError):
        dsa.dsa_cache_evict(b, torch.zeros(1, 1), 1, t.view(1, 1), [], [])
    with pytest.raises(TypeError):
        dsa.dsa_chunk_attn(b, None, kv, 0.04)


def test_evict_rejects_new_weights_inside_the_old(lib):
    base = 1 << 20
    near = dict(weight=base, weight_stride=64, new_weight_stride=32)
    assert _call_evict(lib, new_weight=base + 4 * 63, **near) == INVALID
    assert _call_evict(lib, new_weight=base - 4 * 31, **near) == INVALID


def test_cache_evict_rejects_counts_that_32_bits_would_wrap():
    import torch
    w, t = torch.zeros(1, 64), torch.zeros(1, 1, dtype=torch.int32)
    b = dsa.Batch(t.view(1), torch.zeros(2, dtype=torch.int32), t, 1, 64, 1)
    for kw in (dict(keep=32, sink=2 ** 32), dict(keep=32, recent=2 ** 32), dict(keep=-1)):
        with pytest.raises(ValueError):
            dsa.dsa_cache_evict(b, w, kw.pop("keep"), t, [], [], **kw)


def test_rope_rejects_an_unaligned_status(lib):
    assert _call_rope(lib, status=2) == INVALID


def test_first_calls_of_two_threads_share_one_status_area(monkeypatch):
    # kernels and captured graphs hold its address: the area that a thread was given must be the one that stays
    import threading
    import time

    import torch

    class Area:
        def __init__(self, device):
            self.device = device

        def get(self, n):
            time.sleep(0.05)

    monkeypatch.setattr(dsa, "_status_ws", {})
    monkeypatch.setattr(dsa, "Workspace", Area)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda *a: time.sleep(0.05))
    start, got = threading.Barrier(4), []

    def first():
        start.wait()
        got.append(dsa.status_workspace(0))

    threads = [threading.Thread(target=first) for _ in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert len({id(w) for w in got}) == 1 and dsa.status_workspace(0) is got[0]
