"""Bundle tables of moe_grouped_swiglu_fp8: the C call reads E entries, so it is handed E of them.
The library call is replaced by a recorder; no GPU is used."""
import ctypes as C

import pytest

A = 1 << 20


@pytest.fixture
def calls(monkeypatch):
    import expert_dispatch_streaming_gb300 as moe
    seen, lib = [], moe._lib

    class Recorder:
        def __getattr__(self, name):
            return getattr(lib, name)

        def moe_grouped_swiglu_fp8(self, xq, xs, offsets, table, E, *rest):
            seen.append([table[i] for i in range(len(table))])
            return 0

    monkeypatch.setattr(moe, "_lib", Recorder())
    return moe, seen


def call(moe, table, E):
    moe.moe_grouped_swiglu_fp8(A, A, A, table, E, 128, 128, 8, A, A, 1 << 30, 0)


def test_a_short_list_is_filled_with_null(calls):
    moe, seen = calls
    call(moe, [A, None, A + 16], 6)
    assert seen == [[A, None, A + 16, None, None, None]]


@pytest.mark.parametrize("n", [4, 5, 9])
def test_tables_of_enough_entries_are_taken(calls, n):
    moe, seen = calls
    call(moe, [A] * n, 4)
    call(moe, moe.bundle_table([A] * n), 4)
    assert seen == [[A] * n] * 2


def test_a_short_table_is_refused(calls):
    moe, seen = calls
    whole = (C.c_void_p * 8)(*[A] * 8)
    for table in (moe.bundle_table([A] * 7), (C.c_void_p * 2).from_buffer(whole)):
        with pytest.raises(moe.MoEError) as ei:
            call(moe, table, 8)
        assert ei.value.status == moe.MOE_ERR_INVALID_ARG
    assert not seen


@pytest.mark.parametrize("E", [0, -1, 257, 1 << 30])
def test_counts_of_experts_out_of_range_reach_the_call(calls, E):
    """(it refuses them; nothing of that size is allocated for it)"""
    moe, seen = calls
    call(moe, [A], E)
    assert len(seen) == 1 and len(seen[0]) <= 256
