"""Host-side checks: slot and row counts that no int32 index reaches are refused before any CUDA work."""
import pytest

A = 1 << 20        # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def moe():
    import expert_dispatch_streaming_gb300 as m
    return m


@pytest.mark.parametrize("T,k", [(1 << 30, 2), (1 << 30, 4), (1 << 29, 8), ((1 << 31) - 1, 3)])
def test_too_many_slots(moe, T, k):
    with pytest.raises(moe.MoEError) as ei:
        moe.moe_permute(A, A, T, k, 8, A, stream=0)
    assert ei.value.status == moe.MOE_ERR_INVALID_ARG
    with pytest.raises(moe.MoEError) as ei:
        moe.moe_combine(A, A, A, T, k, 8, None, None, None, A, stream=0)
    assert ei.value.status == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("rows", [(1 << 31) - 8, (1 << 31) - 1])
def test_too_many_rows_of_a_4_bit_product(moe, rows):
    assert moe.moe_grouped_gemv_int4_workspace_size((1 << 31) - 9, 1, 16, 32) > 0
    assert moe.moe_grouped_gemv_int4_workspace_size(rows, 1, 16, 32) == 0
    for off, E in ((None, 1), (A, 4)):
        with pytest.raises(moe.MoEError) as ei:
            moe.moe_grouped_gemv_int4(A, A, A, None, off, E, 16, 32, 32, rows, "bf16", A, A, 256, stream=0)
        assert ei.value.status == moe.MOE_ERR_INVALID_ARG
