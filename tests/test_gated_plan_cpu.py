"""Which kernel a grouped product on bf16 rows takes (no GPU needed)."""
import pytest

import unpermute_count_expert_amd as moe

FWD, DGRAD, WGRAD, GATED, GATED_BWD = (moe.MOE_GEMM_BF16_FORWARD, moe.MOE_GEMM_BF16_DGRAD, moe.MOE_GEMM_BF16_WGRAD,
                                       moe.MOE_GEMM_BF16_SILU_MUL, moe.MOE_GEMM_BF16_DGRAD_SILU_MUL)


def plan(*args):
    p = moe.moe_grouped_gemm_bf16_plan_info(*args, 256)
    return p["tile_rows"], p["staggered"]


@pytest.mark.parametrize("args,want", [
    # one token of a layer of 128 experts, 768 x 2048, top-8
    ((FWD, 128, 1536, 2048, 8), (16, False)), ((GATED, 128, 768, 2048, 8), (16, False)),
    ((GATED_BWD, 128, 2048, 768, 8), (16, False)), ((DGRAD, 128, 1536, 2048, 8), (16, False)),
    # 512 and 4096 tokens
    ((GATED, 128, 768, 2048, 4096), (64, True)), ((GATED_BWD, 128, 2048, 768, 32768), (128, False)),
    ((FWD, 128, 1536, 2048, 4096), (128, True)), ((FWD, 128, 1536, 2048, 16384), (256, True)),
    # 16384 tokens
    ((FWD, 128, 1536, 2048, 131072), (256, False)), ((GATED, 128, 768, 2048, 131072), (256, False)),
    ((GATED_BWD, 128, 2048, 768, 131072), (256, False)), ((WGRAD, 128, 1536, 2048, 1), (256, False)),
    # 130 tokens over 64 experts with wide rows: the 64 x 128 tiles; none past 512 experts
    ((GATED, 64, 672, 2176, 520), (64, True)), ((GATED_BWD, 64, 2176, 672, 520), (64, False)),
    ((GATED, 512, 32, 136, 20480), (64, True)), ((GATED, 513, 32, 136, 20480), (128, True))])
def test_plan(args, want):
    assert plan(*args) == want


@pytest.mark.parametrize("args", [(-1, 8, 64, 64, 1), (5, 8, 64, 64, 1), (FWD, 0, 64, 64, 1), (FWD, 1025, 64, 64, 1),
                                  (FWD, 8, 12, 64, 1), (FWD, 8, 0, 64, 1), (FWD, 8, 65544, 64, 1), (FWD, 8, 64, -8, 1),
                                  (FWD, 8, 64, 65544, 1), (GATED, 8, 32776, 64, 1), (GATED_BWD, 8, 64, 32776, 1),
                                  (FWD, 8, 64, 64, 0), (FWD, 8, 64, 64, -1)])
def test_plan_refuses(args):
    with pytest.raises(moe.MoeError):
        plan(*args)
    with pytest.raises(moe.MoeError):
        moe.moe_grouped_gemm_bf16_plan_info(FWD, 8, 64, 64, 1, -1)


def test_plan_of_the_widest():
    for op in (FWD, DGRAD, WGRAD, GATED, GATED_BWD):
        n, k = 32768 if op == GATED else 65536, 32768 if op == GATED_BWD else 65536
        for E in (1, 1024):
            for rows in (1, 1 << 31, (1 << 63) - 1):
                for cus in (1, 256):
                    p = moe.moe_grouped_gemm_bf16_plan_info(op, E, n, k, rows, cus)
                    assert p["tile_rows"] in (16, 64, 128, 256)
                    assert not p["staggered"] or op in (FWD, GATED)
