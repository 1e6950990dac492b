"""The roofline's traffic comes from committed counter summaries, which count only for the kernel sources they
were taken on."""

import pytest

import bench


@pytest.mark.parametrize("kernel", ["chunk_prep_kernel", "chunk_state_kernel", "recurrent_step_kernel",
                                    "replay_kernel"])
def test_traffic_is_of_these_sources(kernel):
    assert (bench.committed_traffic(kernel) or 0) > 0
