"""gated_norm and rope in place on parts of one buffer that lie beside each other, on the
GPU, against the 64-bit forms (bounds of test_gpu_gated_norm and test_gpu_rope)."""
import pytest
import torch

import kda_prefill_gb300 as kda
from tests import test_gpu_gated_norm as norm_tests
from tests import test_gpu_rope as rope_tests

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 40, 700])
@pytest.mark.parametrize("by_turns", [False, True])
def test_gated_norm_in_place_beside_its_gate(T, by_turns):
    shape = (1, T, 4, 2, 128) if by_turns else (1, T, 2, 4, 128)
    buf = torch.randn(shape, device="cuda").bfloat16()
    was = buf.clone()
    parts = [b.unbind(3 if by_turns else 2) for b in (buf, was)]
    (x, z), (x0, z0) = parts
    assert kda.gated_norm(x, None, gate=z, out=x) is x
    norm_tests.check(x[0], x0[0], None, z0[0], "sigmoid", 1e-6)
    assert torch.equal(z, z0)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T", [1, 50])
def test_rope_on_heads_by_turns(layout, T):
    buf = torch.randn(1, T, 3, 3, 128, device="cuda").bfloat16()
    was = buf.clone()
    freq, _ = kda.rope_frequencies(128)
    pos = torch.arange(T, device="cuda")
    # q and k in place, then from one part to the third
    kda.rope(buf[:, :, :, 0], buf[:, :, :, 1], pos, freq, layout=layout)
    for i in (0, 1):
        rope_tests.check(buf[0, :, :, i], was[0, :, :, i], pos, freq, layout, 1.0)
    assert torch.equal(buf[:, :, :, 2], was[:, :, :, 2])
    mid = buf.clone()
    kda.rope(buf[:, :, :, 0], None, pos, freq, layout=layout, q_out=buf[:, :, :, 2])
    rope_tests.check(buf[0, :, :, 2], mid[0, :, :, 0], pos, freq, layout, 1.0)
    assert torch.equal(buf[:, :, :, :2], mid[:, :, :, :2])
