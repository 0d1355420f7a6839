"""GPU tests of BF16-pool decode where nothing finite has been seen yet: a
context outside the pool gives out = 0 and lse = -inf, a tile of such tokens
before others changes nothing, and NaN cache rows give NaN wherever they lie."""
import numpy as np
import pytest
import torch

import mla_decode_attention_run_gb300 as M
from gpu_util import check_attention, dev_bf16, gpu_decode
from test_gpu_fp4 import _built, _workload  # noqa: F401  (_built: the module's fixture)

pytestmark = pytest.mark.gpu


def _pool(w):
    torch.manual_seed(3)
    return torch.randn(w.num_slots, 576, device="cuda").to(torch.bfloat16)


def _ref(w, pool, keep):
    """64-bit decode over the tokens of `keep` (bool per page-table entry)."""
    x = pool.double().cpu().numpy()
    q = dev_bf16(w.q_bf16, "cpu").double().numpy()
    o, lse = np.zeros((w.batch, w.heads, 512)), np.full((w.batch, w.heads), -np.inf)
    for b in range(w.batch):
        at = np.arange(w.kv_indptr[b], w.kv_indptr[b + 1])
        k = x[w.kv_indices[at[keep[at]]]]
        if len(k):
            s = q[b] @ k.T * w.softmax_scale
            m = s.max(-1, keepdims=True)
            p = np.exp(s - m)
            o[b], lse[b] = p / p.sum(-1, keepdims=True) @ k[:, :512], (m + np.log(p.sum(-1, keepdims=True)))[:, 0]
    return o, lse


@pytest.mark.parametrize("heads,lens,out_of_pool", [
    (16, [40, 90], {0: range(40)}), (4, [4096, 200], {0: range(4096)}), (32, [700, 200], {0: range(64), 1: range(64, 200)}),
    (16, [300, 64], {0: range(128), 1: range(64)}),
])
def test_tokens_outside_the_pool(heads, lens, out_of_pool):
    w = _workload(heads, lens, 1)
    pool, idx, keep = _pool(w), w.kv_indices.copy(), np.ones(len(w.kv_indices), bool)
    for b, ts in out_of_pool.items():
        idx[w.kv_indptr[b] + np.array(ts)] = -1
        keep[w.kv_indptr[b] + np.array(ts)] = False
    out, lse, _ = gpu_decode(w, pool[:, :512], pool[:, 512:], kv_dtype=M.MLA_KV_BF16, k_scale=1.0, kv_indices=idx)
    assert M.mla_get_last_error() == M.FLAG_INDEX_OOB
    o_ref, l_ref = _ref(w, pool, keep)
    check_attention(out, lse, o_ref, l_ref, "BF16 pool")
    empty = np.isneginf(l_ref)
    assert np.array_equal(np.isneginf(lse.cpu().numpy()), empty) and (out[torch.from_numpy(empty).cuda()] == 0).all()


@pytest.mark.parametrize("channel", [5, 540])
@pytest.mark.parametrize("heads,lens,hits", [(16, [1, 5], [0]), (32, [200, 90], range(64)), (4, [4096, 3], range(256, 384)), (16, [65, 64], [64])])
def test_nan_rows(heads, lens, hits, channel):
    w = _workload(heads, lens, 1)
    pool = _pool(w)
    o_ref, l_ref = _ref(w, pool, np.ones(len(w.kv_indices), bool))
    pool[torch.from_numpy(w.kv_indices[w.kv_indptr[0] + np.array(hits)].astype(np.int64)).cuda(), channel] = float("nan")
    out, lse, _ = gpu_decode(w, pool[:, :512], pool[:, 512:], kv_dtype=M.MLA_KV_BF16, k_scale=1.0)
    assert M.mla_get_last_error() == 0
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    check_attention(out[1:], lse[1:], o_ref[1:], l_ref[1:], "the other request")
