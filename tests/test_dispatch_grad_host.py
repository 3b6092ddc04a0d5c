"""Host-side checks of the slot sort, the gradients and the 4-bit products: workspace sizes and the
refusals of every entry point (sizes, alignment, null pointers, workspaces).  No GPU is used: a
refused call returns before any CUDA work, and every call here is refused or has nothing to do."""
import pytest

A = 1 << 20        # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def moe():
    import expert_dispatch_streaming_gb300 as m
    return m


def refused(moe, fn, args, **bad):
    for name, value in bad.items():
        assert name in args
        with pytest.raises(moe.MoEError) as ei:
            fn(*{**args, name: value}.values(), stream=0)
        assert ei.value.status == moe.MOE_ERR_INVALID_ARG, (name, value)


def test_sort_refusals(moe):
    assert moe.moe_sort_tokens_workspace_size(-1, 8, 2) == 0
    assert moe.moe_sort_tokens_workspace_size(4, 257, 2) == 0
    assert moe.moe_sort_tokens_workspace_size(4, 8, 9) == 0
    assert moe.moe_sort_tokens_workspace_size(1 << 30, 8, 2) == 0        # 2^31 slots
    n = moe.moe_sort_tokens_workspace_size(4, 8, 2)
    assert n > 0
    ok = dict(ids=A, T=4, E=8, k=2, counts=A, offsets=A, pos=A, src=A, ws=A, ws_bytes=n)
    for name, values in dict(ids=(None, A + 2), T=(-1, 1 << 30), E=(0, 257), k=(0, 9),
                             counts=(None, A + 1), offsets=(None, A + 2), pos=(None, A + 2),
                             src=(None, A + 2), ws=(None, A + 2), ws_bytes=(n - 1, 0)).items():
        for v in values:
            refused(moe, moe.moe_sort_tokens, ok, **{name: v})


def test_permute_backward_refusals(moe):
    ok = dict(dx_perm=A, pos=A, add=None, T=4, k=2, H=64, out="bf16", dx=A)
    for name, values in dict(dx_perm=(None, A + 8), pos=(None, A + 2), add=(A + 8,), T=(-1, 1 << 30),
                             k=(0, 9), H=(0, 63, -8), out=(2, -1), dx=(None, A + 8)).items():
        for v in values:
            refused(moe, moe.moe_permute_backward, ok, **{name: v})
    moe.moe_permute_backward(None, None, None, 0, 2, 64, "fp32", None, stream=0)


def test_combine_backward_refusals(moe):
    ok = dict(dout=A, y_perm=A, pos=A, w=A, T=4, k=2, H=64, shared=A, shared_gate=A, dy_perm=A,
              dw=A, dshared=A, dshared_gate=A)
    for name, values in dict(dout=(None, A + 8), y_perm=(None, A + 8), pos=(None, A + 2),
                             w=(None, A + 2), T=(-1, 1 << 30), k=(0, 9), H=(0, 12),
                             shared=(None, A + 8), shared_gate=(None, A + 2), dy_perm=(A + 8,),
                             dw=(A + 2,), dshared=(A + 8,), dshared_gate=(A + 2,)).items():
        for v in values:
            refused(moe, moe.moe_combine_backward, ok, **{name: v})
    none = dict(ok, dy_perm=None, dw=None, dshared=None)
    refused(moe, moe.moe_combine_backward, none, dshared_gate=None)      # nothing to compute
    moe.moe_combine_backward(None, None, None, None, 0, 2, 64, None, None, None, None, stream=0)


def test_gate_backward_refusals(moe):
    ok = dict(logits=A, ids=A, dw=A, T=4, E=8, k=2, gating="softmax", scale=1.0, dlogits=A)
    for name, values in dict(logits=(None, A + 2), ids=(None, A + 2), dw=(None, A + 2), T=(-1,),
                             E=(0, 1, 257), k=(0, 9), gating=(3, -1, 16), dlogits=(None, A + 2)
                             ).items():
        for v in values:
            refused(moe, moe.moe_gate_backward, ok, **{name: v})
    moe.moe_gate_backward(None, None, None, 0, 8, 2, "softmax", 1.0, None, stream=0)


def test_gemv_refusals(moe):
    size = moe.moe_grouped_gemv_int4_workspace_size
    assert size(4, 0, 8, 32) == size(4, 257, 8, 32) == size(-1, 1, 8, 32) == 0
    assert size(4, 1, 0, 32) == size(4, 1, 8, 48) == size(4, 1, 8, 0) == 0
    n = size(4, 8, 100, 96)
    assert n > 0
    ok = dict(x=A, w=A, w_scale=A, w_zero=A + 1, offsets=A, E=8, N=100, K=96, group=32, max_rows=4,
              out="bf16", y=A, ws=A, ws_bytes=n)
    for name, values in dict(x=(None, A + 8), w=(None, A + 8), w_scale=(None, A + 1),
                             offsets=(None, A + 2), E=(0, 257), N=(0, -1, 1 << 29), K=(0, 16, 100),
                             group=(0, 16, 48, 256), max_rows=(-1,), out=(2, -1), y=(None, A + 8),
                             ws=(None, A + 128), ws_bytes=(n - 1,)).items():
        for v in values:
            refused(moe, moe.moe_grouped_gemv_int4, ok, **{name: v})
    moe.moe_grouped_gemv_int4(None, None, None, None, None, 1, 8, 32, 32, 0, "fp32", None, None, 0,
                              stream=0)
