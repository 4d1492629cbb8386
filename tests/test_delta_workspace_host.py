"""CPU tests of the gated delta rule's workspace: what a batch without chunks needs, and that the
bound holds for every batch."""
import random

import pytest

import kda_prefill_gb300 as kda
from tests.test_delta_host import delta_abi
from tests.test_ops_host import lib  # noqa: F401

STEP_MAX, CHUNK, HEADER = 16, 64, 256


@pytest.mark.parametrize("cu,T,enough", [
    ([0, 16, 32], 32, True), ([0, 1, 2], 2, True), ([0, 0, 0], 0, True), ([0, 0, 16], 16, True),
    ([0, 17, 32], 32, False), ([0, 15, 32], 32, False), ([0, 0, 17], 17, False),
])
def test_a_batch_without_chunks_needs_its_header_alone(lib, cu, T, enough):  # noqa: F811
    """Past the workspace's check the call goes on to the GPU, which is not there."""
    rc, err = delta_abi(lib, cu=cu, T=T, ws_bytes=HEADER)
    assert (rc != -5) == enough, (rc, err)
    assert enough or "workspace of 256 bytes" in err
    assert delta_abi(lib, cu=cu, T=T, ws_bytes=HEADER - 1)[0] == -5


def test_bounds_on_the_device_say_nothing(lib):  # noqa: F811
    rc, err = delta_abi(lib, host=None, T=32, ws_bytes=HEADER)
    assert rc == -5 and "workspace of 256 bytes" in err
    assert delta_abi(lib, host=None, T=16, ws_bytes=HEADER)[0] != -5


def test_wrong_bounds_are_refused_as_such(lib):  # noqa: F811
    assert delta_abi(lib, cu=[0, 5, 3], T=3, ws_bytes=HEADER)[0] == -1
    assert delta_abi(lib, cu=[0, 5, 9], T=8, ws_bytes=HEADER)[0] == -1
    assert delta_abi(lib, N=-1, ws_bytes=HEADER)[0] == -1


def test_the_bound_holds():
    """The chunks of sequences of more than 16 tokens, whatever their lengths."""
    size = kda.gated_delta_workspace_size
    assert size(16, 16, 12) == size(1, 1, 1) == HEADER
    block = size(64, 1, 1) - HEADER
    block //= 2  # one for the tokens, one for the sequence
    rng = random.Random(5)
    for _ in range(300):
        n = rng.choice([1, 2, 5, 40])
        lens = [rng.choice([0, 1, 15, 16, 17, 18, 63, 64, 65, rng.randint(0, 500)]) for _ in range(n)]
        T, H = sum(lens), rng.choice([1, 3])
        chunks = sum(-(-x // CHUNK) for x in lens if x > STEP_MAX)
        assert size(T, n, H) >= HEADER + chunks * H * block, lens
