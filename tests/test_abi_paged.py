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
