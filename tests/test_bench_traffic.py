"""The bench's memory traffic per kernel is a measurement of given sources: every
entry has to be one of the present sources, or the bench line loses the figure."""
import pytest

import bench


@pytest.mark.parametrize("kernel", sorted(bench.MEASURED_TRAFFIC_MIB))
def test_traffic_belongs_to_the_sources(kernel):
    _, _, read, written = bench.MEASURED_TRAFFIC_MIB[kernel]
    assert bench.measured_traffic(kernel) == (read + written) * 2 ** 20
