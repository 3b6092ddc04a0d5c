"""GPU tests of FP8 bundles packed on the device."""
import numpy as np
import pytest
import torch

from test_gpu_fp8 import bundles_of, fp8_weights, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import expert_dispatch_streaming_gb300 as m
    return m


@pytest.mark.parametrize("H,I", [(384, 256), (128, 128), (1024, 1024)])
def test_device_packed_bundle_is_the_host_packed_one_byte_for_byte(moe, H, I):
    """The gaps after the scale arrays too: a checksum covers the whole bundle."""
    g = gen(9)
    w13, s13 = fp8_weights(g, 1, 2 * I, H)
    w2, s2 = fp8_weights(g, 1, H, I)
    d = bundles_of(moe, H, I, w13, s13, w2, s2)[0].cpu().numpy()
    host = np.zeros_like(d)
    moe.moe_pack_bundle_fp8(H, I, w13[0].view(torch.uint8).cpu(), s13[0].cpu(),
                            w2[0].view(torch.uint8).cpu(), s2[0].cpu(), host)
    assert np.array_equal(d, host)
    assert moe.moe_checksum64(d, d.size) == moe.moe_checksum64(host, host.size)
