"""GPU tests of the order of kernels that may start beside the end of the one before them (the slot sort,
the gradients and the 4-bit products are launched so, whatever MOE_OPT_PDL says): a chain of them, call
after call on the same buffers, against the same calls with a synchronisation after each, which leaves
nothing to overlap with.  Every stage is deterministic, so results are equal to the bit."""
import pytest
import torch

from test_gpu_dispatch_grad import gen, make_ids, moe  # noqa: F401

pytestmark = pytest.mark.gpu

T, E, k, H, GROUP = 3001, 64, 8, 256, 64
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def inputs(moe, seed):  # noqa: F811
    g = gen(seed)
    return dict(
        ids=torch.from_numpy(make_ids(T, E, k, 0.1, seed)).cuda(),
        x=torch.randn((T, H), generator=g, device="cuda").to(BF),
        w=torch.rand((T, k), generator=g, device="cuda"),
        z=torch.randn((T, E), generator=g, device="cuda"),
        w4=torch.randint(0, 256, (E, H, H // 2), generator=g, device="cuda", dtype=U8),
        s=(torch.rand((E, H, H // GROUP), generator=g, device="cuda") * 0.02).to(BF),
        zp=torch.randint(0, 16, (E, H, H // GROUP), generator=g, device="cuda", dtype=U8))


def between(moe):  # noqa: F811
    """What one call of the chain leaves for the next: one set, used by every pass."""
    nb = moe.moe_sort_tokens_workspace_size(T, E, k)
    return dict(counts=torch.empty(E, dtype=I32, device="cuda"),
                offsets=torch.empty(E + 1, dtype=I32, device="cuda"),
                pos=torch.empty((T, k), dtype=I32, device="cuda"),
                src=torch.empty(T * k, dtype=I32, device="cuda"),
                ws=torch.empty(nb, dtype=U8, device="cuda"),
                ws4=torch.empty(256, dtype=U8, device="cuda"),
                xp=torch.empty((T * k, H), dtype=BF, device="cuda"),
                y=torch.zeros((T * k, H), dtype=BF, device="cuda"),
                dy=torch.zeros((T * k, H), dtype=BF, device="cuda"))


def outputs():
    return dict(out=torch.empty((T, H), dtype=BF, device="cuda"), dw=torch.empty((T, k), device="cuda"),
                dz=torch.empty((T, E), device="cuda"), dx=torch.empty((T, H), device="cuda"))


def calls(moe, i, b, o):  # noqa: F811
    """The chain as a list of calls, each given the stream it runs on."""
    return [
        lambda s=None: moe.moe_sort_tokens(i["ids"], T, E, k, b["counts"], b["offsets"], b["pos"], b["src"],
                                           b["ws"], b["ws"].numel(), s),
        lambda s=None: moe.moe_permute(i["x"], b["src"], T, k, H, b["xp"], s),
        lambda s=None: moe.moe_grouped_gemv_int4(b["xp"], i["w4"], i["s"], i["zp"], b["offsets"], E, H, H,
                                                 GROUP, T * k, "bf16", b["y"], b["ws4"], 256, s),
        lambda s=None: moe.moe_combine(b["y"], b["pos"], i["w"], T, k, H, None, None, None, o["out"], s),
        lambda s=None: moe.moe_combine_backward(o["out"], b["y"], b["pos"], i["w"], T, k, H, None, None,
                                                b["dy"], o["dw"], stream=s),
        lambda s=None: moe.moe_gate_backward(i["z"], i["ids"], o["dw"], T, E, k, "softmax_renorm", 1.0,
                                             o["dz"], s),
        lambda s=None: moe.moe_permute_backward(b["dy"], b["pos"], o["out"], T, k, H, "fp32", o["dx"], s),
    ]


def synchronised(moe, i):  # noqa: F811
    b, o = between(moe), outputs()
    for call in calls(moe, i, b, o):
        torch.cuda.synchronize()
        call()
    torch.cuda.synchronize()
    return o


@pytest.fixture(scope="module")
def sets(moe):  # noqa: F811
    all_inputs = [inputs(moe, seed) for seed in range(3)]
    return [(i, synchronised(moe, i)) for i in all_inputs]


def same(got, want):
    for n in want:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("pdl", [False, True])
def test_calls_in_a_row(moe, sets, pdl):  # noqa: F811
    """Thirty passes without anything else on the stream, inputs changing from pass to pass: each pass's
    outputs are kept, what lies between the calls is written over by the next pass."""
    b = between(moe)
    kept = [outputs() for _ in range(30)]
    torch.cuda.synchronize()
    moe.set_pdl(pdl)
    try:
        for n, o in enumerate(kept):
            for call in calls(moe, sets[n % 3][0], b, o):
                call()
    finally:
        moe.set_pdl(False)
    torch.cuda.synchronize()
    for n, o in enumerate(kept):
        same(o, sets[n % 3][1])


def test_one_call_behind_another(moe, sets):  # noqa: F811
    """Each pair of the chain's calls alone: the second one starts with nothing but the first before it,
    which the GPU is still running; the inputs of the first are those of another set."""
    for n in range(len(calls(moe, sets[0][0], between(moe), outputs())) - 1):
        b, o = between(moe), outputs()
        for i, want in (sets[0], sets[1]):
            chain = calls(moe, i, b, o)
            for at, call in enumerate(chain):
                if at != n + 1:
                    torch.cuda.synchronize()
                call()
            torch.cuda.synchronize()
            same(o, want)


def test_two_streams_by_events(moe, sets):  # noqa: F811
    """The chain's calls in turn on two streams, ordered by events alone."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    b = between(moe)
    kept = [outputs() for _ in range(9)]
    torch.cuda.synchronize()
    turn, last = 0, None
    for n, o in enumerate(kept):
        for call in calls(moe, sets[n % 3][0], b, o):
            s = streams[turn % 2]
            if last is not None:
                s.wait_event(last)
            call(s)
            last = s.record_event()
            turn += 1
    torch.cuda.synchronize()
    for n, o in enumerate(kept):
        same(o, sets[n % 3][1])


def test_captured_fork_and_join(moe, sets):  # noqa: F811
    """One graph whose branches part after combine's gradient (the gating's gradient on one stream, the
    permute's on the other) and meet again in a call that reads the first's result, replayed on the inputs of
    every set."""
    i, b, o = {n: v.clone() for n, v in sets[0][0].items()}, between(moe), outputs()
    again, ref = torch.empty((T, E), device="cuda"), torch.empty((T, E), device="cuda")
    s0, s1 = torch.cuda.Stream(), torch.cuda.Stream()
    chain = calls(moe, i, b, o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s0):
        for call in chain[:5]:
            call(s0)
        s1.wait_event(s0.record_event())
        chain[5](s1)
        chain[6](s0)
        s0.wait_event(s1.record_event())
        moe.moe_gate_backward(o["dz"], i["ids"], o["dw"], T, E, k, "softmax", 1.0, again, s0)
    for new, want in sets * 3:
        for n, v in new.items():
            i[n].copy_(v)
        torch.cuda.synchronize()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        same(o, want)
        moe.moe_gate_backward(want["dz"], new["ids"], want["dw"], T, E, k, "softmax", 1.0, ref)
        assert torch.equal(again, ref)
