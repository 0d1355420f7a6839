"""Attention over 4-bit rows against the 8-bit kernels on the same rows widened,
bit for bit: a 4-bit row widens exactly, both multiply the same tiles in the
same order, and both add the same sums in the same order."""
import pytest
import torch

import mla_decode_attention_run_gb300 as M
from test_gpu_fp4 import _attend, _built, _pools, _workload  # noqa: F401  (_built: the module's fixture)

pytestmark = pytest.mark.gpu


def _check(w, max_e=9, k_scale=0.05):
    pool, wide = _pools(w, max_e)
    out4, lse4, _ = _attend(w, torch.from_numpy(pool).cuda(), M.MLA_KV_FP4_E2M1, k_scale)
    out8, lse8, _ = _attend(w, torch.from_numpy(wide).cuda(), M.MLA_KV_FP8_E4M3, k_scale)
    assert M.mla_get_last_error() == 0
    assert torch.equal(out4, out8) and torch.equal(lse4, lse8)


@pytest.mark.parametrize("heads,lens,ps", [
    (16, [64] * 300, 1), (16, [100] * 200, 1), (5, [128] * 100, 2), (1, [3000, 1, 0, 65], 1), (16, [300, 5000, 1024, 77], 64),
    (16, [4096], 1), (32, [200] * 200, 3), (128, [90] * 100, 1), (64, [2000] * 3, 16),
])
def test_decode(heads, lens, ps):
    _check(_workload(heads, lens, ps))


@pytest.mark.parametrize("heads,lens,q_lens,ps", [
    (16, [64] * 200, [4] * 200, 1), (16, [400] * 60, [17] * 60, 1), (4, [40, 17, 33], [3, 17, 5], 1), (128, [700, 300], [3, 1], 64),
])
def test_extend(heads, lens, q_lens, ps):
    _check(_workload(heads, lens, ps, q_lens))


@pytest.mark.parametrize("max_e,k_scale", [(14, 2e-4), (2, 4.0), (0, 30.0)])
def test_exponent_range(max_e, k_scale):
    _check(_workload(16, [100] * 150, 1), max_e, k_scale)
