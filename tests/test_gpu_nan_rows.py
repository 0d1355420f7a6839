"""GPU tests of cache rows that hold a NaN, 4-bit (a block with exponent 15)
and 8-bit (0x7F): by the definition the score of such a token is NaN, so every
query row that sees it has out = NaN and lse = NaN in all of its channels,
wherever the token lies in a tile, a split segment or a context, and every
other query row is that of a pool without the NaN (against the CPU oracle on
that pool, at the attention tests' tolerances)."""
import numpy as np
import pytest
import torch

import mla_decode_attention_run_gb300 as M
import oracle
import ref_step as R
from gpu_util import check_attention
from test_gpu_fp4 import _attend, _built, _pool4, _workload  # noqa: F401  (_built: the module's fixture)

pytestmark = pytest.mark.gpu

POOLS = [M.MLA_KV_FP4_E2M1, M.MLA_KV_FP8_E4M3]
PARTS = ["k_pe", "c_kv", "both"]


def _poison(pool, slots, part):
    """The slots' rows with one NaN block: c_kv channels 96..111, k_pe channels 48..63."""
    bad = pool.copy()
    if part != "k_pe":
        bad[slots, 256 + 3] |= 0x0F
    if part != "c_kv":
        bad[slots, 272 + 33] |= 0xF0
    return bad


def _check(w, hits, part, dtype, nan_query=None, k_scale=0.05):
    """hits: per request, the tokens whose rows hold a NaN."""
    pool = _pool4(np.random.default_rng(1), w.num_slots, 9)
    slots = [w.kv_indices[w.kv_indptr[b] + t // w.page_size] * w.page_size + t % w.page_size for b, ts in hits.items() for t in ts]
    bad = _poison(pool, slots, part)
    clean = R.e4m3_rows(pool[:, :272], pool[:, 272:])
    dpool = bad if dtype == M.MLA_KV_FP4_E2M1 else R.e4m3_rows(bad[:, :272], bad[:, 272:])
    qo = w.extra.get("qo_indptr")
    a = (w.q_bf16, clean[:, :512], clean[:, 512:])
    b = (w.kv_indptr, w.kv_indices, w.seq_lens, w.page_size, k_scale, w.softmax_scale)
    o_ref, l_ref = oracle.decode_fp8(*a, *b) if qo is None else oracle.extend_fp8(*a, qo, *b)
    nan = np.zeros(l_ref.shape, bool)
    for r, ts in hits.items():
        if qo is None:
            nan[r] = len(ts) > 0
        else:
            for n in range(qo[r], qo[r + 1]):
                nan[n] = any(t < w.seq_lens[r] + 1 - qo[r + 1] + n for t in ts)
    if nan_query is not None:
        w.q_bf16[nan_query + (100,)] = 0x7FC0
        nan[nan_query] = True
    out, lse, _ = _attend(w, torch.from_numpy(dpool).cuda(), dtype, k_scale)
    assert M.mla_get_last_error() == 0
    o, l = out.float().cpu().numpy(), lse.cpu().numpy()
    assert np.isnan(l[nan]).all() and np.isnan(o[nan]).all()
    assert not np.isnan(l[~nan]).any() and not np.isnan(o[~nan]).any()
    if (~nan).any():
        check_attention(out[torch.from_numpy(~nan).cuda()], lse[torch.from_numpy(~nan).cuda()], o_ref[~nan], l_ref[~nan], "rows without a NaN")


@pytest.mark.parametrize("dtype", POOLS)
@pytest.mark.parametrize("part", PARTS)
@pytest.mark.parametrize("heads,lens,hits", [
    (16, [1, 5], {0: [0]}),                                     # nothing but a NaN
    (32, [1, 5], {0: [0]}),
    (4, [200, 200, 64], {0: range(64), 2: range(64)}),          # a tile of NaN, before finite ones and alone
    (64, [200, 200, 64], {0: range(64), 2: range(64)}),
    (16, [2049, 0], {0: [2048]}),                               # a token that is a split segment of its own
    (32, [2305, 1281, 1537, 2433], {0: [2304], 2: [1536]}),
    (16, [4096], {0: range(256, 384)}),                         # a whole split segment
    (128, [700, 90], {0: [699]}),
])
def test_decode(heads, lens, hits, part, dtype):
    _check(_workload(heads, lens, 1), hits, part, dtype)


def test_the_lone_tokens_above_are_segments_of_their_own():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for heads, lens, b in ((16, [2049, 0], 0), (32, [2305, 1281, 1537, 2433], 0)):
        segs, _ = M.mla_decode_schedule(np.concatenate(([0], np.cumsum(lens))), lens, len(lens), heads, 1, M.MLA_KV_FP4_E2M1, sms)
        last = segs[(segs[:, 1] == b) & (segs[:, 3] == lens[b])][0]
        assert last[3] - last[2] == 1 and last[4] >= 0


@pytest.mark.parametrize("dtype", POOLS)
@pytest.mark.parametrize("part", PARTS)
@pytest.mark.parametrize("heads,lens,q_lens,hits", [
    (16, [1, 9], [1, 9], {0: [0]}),                             # 16 rows of one token to a block
    (1, [1, 40], [1, 3], {0: [0]}),
    (1, [200], [40], {0: [199]}),                               # the last of 40 new tokens: the other 39 do not see it
    (4, [200, 130], [40, 9], {0: [180, 199], 1: [125]}),
    (16, [300, 70], [70, 70], {0: [299], 1: [0]}),
    (2, [129, 64], [17, 64], {0: [128], 1: [33, 40]}),          # the NaN token starts a tile
    (128, [200], [3], {0: [199]}),                              # several blocks to a token: none hides a token from itself
    (7, [2000], [30], {0: [1990]}),                             # blocks split over CTAs
    (16, [200, 64], [4, 4], {0: range(64)}),                    # a tile of NaN before the new tokens
    (3, [700], [64], {0: range(660, 700, 3)}),
    (1, [200], [9], {0: [199]}),                                # blocks of 16 rows (the others above: 32)
    (4, [130, 3000], [3, 4], {0: [128], 1: [2998]}),
])
def test_extend(heads, lens, q_lens, hits, part, dtype):
    _check(_workload(heads, lens, 3 if heads == 4 else 1, q_lens), hits, part, dtype)


@pytest.mark.parametrize("dtype", POOLS)
def test_extend_with_a_nan_query_row(dtype):
    """A non-finite query row does not make the tokens that others see pass for NaN rows."""
    _check(_workload(4, [200], 1, [40]), {0: [199]}, "c_kv", dtype, nan_query=(3, 1))
    _check(_workload(1, [90], 1, [33]), {}, "c_kv", dtype, nan_query=(0, 0))
    _check(_workload(1, [90], 1, [33]), {0: [89]}, "c_kv", dtype, nan_query=(0, 0))
