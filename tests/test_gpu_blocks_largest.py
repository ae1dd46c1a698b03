"""An append into blocks that reads and writes more than 2^31 bytes."""

from __future__ import annotations

import pytest

from tests.test_gpu_blocks import test_large_calls_write_what_small_ones_do as large_and_small

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import recurrent_state_amd as k
    k.lib()
    return k


def test_a_call_of_many_bytes_writes_what_small_ones_do(kda):
    large_and_small(kda, 128, 64, 98304)
