"""The DRAM traffic that bench.py reports beside its times comes from captures of the kernels as they
are: it is left out once a source file they are built from has changed. A file that only other
kernels need is not to be mixed into those."""
import bench


def test_the_adamw_capture_is_of_these_sources():
    assert bench.adamw_traffic(1 << 20) == round(bench.ADAMW_TRAFFIC_PER_ELEM * (1 << 20))


def test_the_newton_schulz_capture_is_of_these_sources():
    assert bench.source_digest(bench.NS_SOURCES) == bench.NS_SRC_DIGEST
