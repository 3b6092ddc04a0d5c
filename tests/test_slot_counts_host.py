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
