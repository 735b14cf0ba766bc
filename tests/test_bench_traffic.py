"""The bench line's DRAM figure: a capture's, reported while the sources of the
captured kernel are the ones it was taken of."""
import bench


def test_the_default_workload_has_its_traffic():
    for key, t in bench.KERNEL_TRAFFIC.items():
        assert bench.measured_traffic(key) == (t["bytes"], t["profile"]), key
