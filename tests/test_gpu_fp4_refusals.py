"""Row strides that a 4-bit plan refuses, at each call that runs one: shorter
than a row (status 1), or past 31 bits (status 2; refused before any launch, so
the pools are never read)."""
import pytest
import torch

import mla_decode_attention_run_gb300 as M
from test_gpu_fp4 import _built  # noqa: F401  (the module's fixture)

pytestmark = pytest.mark.gpu


def _call(name, ckv_stride, kpe_stride, slots=4):
    """The C entry point `name` on a 4-bit plan of one token, with the given strides; returns (status, out)."""
    i32 = dict(dtype=torch.int32, device="cuda")
    if name == "mla_extend_run":
        plan = M.mla_extend_plan([0, 1], [0, 1], [1], 1, 16, 1, M.MLA_KV_FP4_E2M1)
    else:
        plan = M.mla_decode_plan([0, 1], [1], 1, 16, 1, M.MLA_KV_FP4_E2M1)
    pool = torch.zeros(slots, 320, dtype=torch.uint8, device="cuda")
    q = torch.zeros(1, 16, 576, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.ones(1, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 16, device="cuda")
    ws = torch.empty(max(plan.workspace_bytes, 256), dtype=torch.uint8, device="cuda")
    indptr, idx, lens = torch.tensor([0, 1], **i32), torch.zeros(1, **i32), torch.ones(1, **i32)
    args = [plan.handle, q.data_ptr(), 16 * 576, 576, pool.data_ptr(), ckv_stride, pool.data_ptr() + 272, kpe_stride, slots,
            indptr.data_ptr(), idx.data_ptr(), lens.data_ptr(), 1.0, 0.07, out.data_ptr(), lse.data_ptr()]
    args += [None] if name == "mla_decode_run_static_scratch" else [ws.data_ptr(), ws.numel(), None]
    status = getattr(M.library(), name)(*args)
    torch.cuda.synchronize()
    return status, out


@pytest.mark.parametrize("name", ["mla_decode_run", "mla_extend_run", "mla_decode_run_static_scratch"])
def test_strides(name):
    for strides in ((256, 320), (320, 32), (16, 320), (320, 16), (0x7FFFFFF0, 32)):
        status, out = _call(name, *strides)
        assert status == 1 and (out == 1).all(), strides
    for strides in ((1 << 31, 320), (320, 1 << 31), (1 << 40, 1 << 40), (320, 312), (328, 320), (-320, 320), (320, 0)):
        status, out = _call(name, *strides)
        assert status == 2 and (out == 1).all(), strides
    status, out = _call(name, 320, 320)
    assert status == 0 and (out == 0).all()                     # one token of zeros
    assert M.mla_get_last_error() == 0
