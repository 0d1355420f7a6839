"""Pools of another type than the plan's are refused by the Python entry points
before the library sees a pointer: a 4-bit pool's rows are shorter than those an
8-bit or BF16 plan reads, and a 4-bit plan takes byte rows only."""
import pytest
import torch

import mla_decode_attention_run_gb300 as M

RUNS = [M.mla_decode_run, M.mla_extend_run, M.mla_decode_run_static_scratch]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _run(run, kv_dtype, ckv, kpe, slots=8, device="cpu"):
    plan = M.Plan()
    plan.kv_dtype = kv_dtype
    z = torch.zeros(4, dtype=torch.int32, device=device)
    q = torch.zeros(1, 16, 576, dtype=torch.bfloat16, device=device)
    run(plan, q, ckv, kpe, slots, z, z, z, 1.0, 0.07, torch.zeros(1, 16, 512, dtype=torch.bfloat16, device=device),
        torch.zeros(1, 16, device=device), stream=0)


@pytest.mark.parametrize("run", RUNS)
def test_other_plans_refuse_a_4_bit_pool(run):
    pool = torch.zeros(8, 320, dtype=torch.uint8)
    for args in ((pool, pool[:, 272:]), (pool[:, :272], pool[:, 272:]), (torch.zeros(8, 512, dtype=torch.uint8), pool[:, 272:])):
        with pytest.raises(ValueError):
            _run(run, M.MLA_KV_FP8_E4M3, *args)
    with pytest.raises(ValueError):
        _run(run, M.MLA_KV_BF16, torch.zeros(8, 320, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16))


@pytest.mark.parametrize("run", RUNS)
def test_a_4_bit_plan_refuses_other_pools(run):
    fp8, bf16 = torch.zeros(8, 576, dtype=torch.float8_e4m3fn), torch.zeros(8, 576, dtype=torch.bfloat16)
    for pool in (fp8, bf16):
        with pytest.raises(TypeError):
            _run(run, M.MLA_KV_FP4_E2M1, pool[:, :512], pool[:, 512:])
    pool = torch.zeros(8, 320, dtype=torch.uint8)
    with pytest.raises(TypeError):
        _run(run, M.MLA_KV_FP4_E2M1, pool, fp8[:, 512:])
    with pytest.raises(ValueError):                             # on the CPU
        _run(run, M.MLA_KV_FP4_E2M1, pool, pool[:, 272:])


@pytest.mark.gpu
@pytest.mark.parametrize("run", RUNS)
def test_a_4_bit_plan_refuses_short_pools_on_the_device(run):
    pool = torch.zeros(8, 320, dtype=torch.uint8, device="cuda")
    for ckv, kpe, slots in ((pool, pool[:, 272:], 9), (pool, pool[:7, 272:], 8), (pool[:, :256], pool[:, 272:], 8),
                            (pool, pool[:, 290:], 8), (pool, pool[:, 272:].cpu(), 8), (pool.view(-1), pool[:, 272:], 8)):
        with pytest.raises(ValueError):
            _run(run, M.MLA_KV_FP4_E2M1, ckv, kpe, slots, "cuda")


@pytest.mark.gpu
def test_plans_know_their_pool_type():
    plan = M.mla_decode_plan([0, 5], [5], 1, 16, 1)
    assert plan.kv_dtype == M.MLA_KV_FP8_E4M3
    plan = M.mla_decode_plan([0, 5], [5], 1, 16, 1, M.MLA_KV_FP4_E2M1, plan=plan)
    assert plan.kv_dtype == M.MLA_KV_FP4_E2M1
    assert M.mla_extend_plan([0, 2], [0, 5], [5], 1, 16, 1, M.MLA_KV_FP4_E2M1).kv_dtype == M.MLA_KV_FP4_E2M1
