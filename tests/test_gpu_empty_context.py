"""GPU tests of contexts whose every page lies outside the pool: the tokens are
excluded from the softmax and flagged, so a row gets out = 0 and lse = -inf like
that of an empty context, whether one CTA serves it or split segments are
merged."""
import numpy as np
import pytest
import torch

import mla_decode_attention_run_gb300 as M
import oracle
import ref_step as R
from gpu_util import check_attention
from test_gpu_fp4 import _attend, _built, _pool4, _workload  # noqa: F401  (_built: the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [M.MLA_KV_FP4_E2M1, M.MLA_KV_FP8_E4M3])
@pytest.mark.parametrize("heads,lens,q_lens", [(16, [4096, 50], None), (16, [40], None), (32, [4096], None), (128, [700, 3], None),
                                               (4, [2000], [9]), (16, [70], [20])])
def test_context_wholly_outside_the_pool(heads, lens, q_lens, dtype):
    w = _workload(heads, lens, 1, q_lens)
    pool = _pool4(np.random.default_rng(1), w.num_slots, 9)
    dpool = pool if dtype == M.MLA_KV_FP4_E2M1 else R.e4m3_rows(pool[:, :272], pool[:, 272:])
    out, lse, _ = _attend(w, torch.from_numpy(dpool).cuda(), dtype, 0.05, indices=np.full(len(w.kv_indices), -1))
    assert M.mla_get_last_error() == M.FLAG_INDEX_OOB
    assert torch.isneginf(lse).all() and (out == 0).all()


@pytest.mark.parametrize("dtype", [M.MLA_KV_FP4_E2M1, M.MLA_KV_FP8_E4M3])
def test_beside_requests_with_a_context(dtype):
    """One request of a batch outside the pool, the others against the oracle."""
    w = _workload(16, [3000, 2500, 90], 1)
    pool = _pool4(np.random.default_rng(1), w.num_slots, 9)
    wide = R.e4m3_rows(pool[:, :272], pool[:, 272:])
    idx = w.kv_indices.copy()
    idx[w.kv_indptr[1]:w.kv_indptr[2]] = w.num_slots
    out, lse, _ = _attend(w, torch.from_numpy(pool if dtype == M.MLA_KV_FP4_E2M1 else wide).cuda(), dtype, 0.05, indices=idx)
    assert M.mla_get_last_error() == M.FLAG_INDEX_OOB
    assert torch.isneginf(lse[1]).all() and (out[1] == 0).all()
    o_ref, l_ref = oracle.decode_fp8(w.q_bf16, wide[:, :512], wide[:, 512:], w.kv_indptr, w.kv_indices, w.seq_lens, 1, 0.05, w.softmax_scale)
    check_attention(out[[0, 2]], lse[[0, 2]], o_ref[[0, 2]], l_ref[[0, 2]], "beside")
