"""What bench.py reports from committed summaries belongs to the committed sources."""
import bench


def test_the_headline_kernels_traffic_was_counted_on_these_sources():
    """The counters' summary holds a digest of the kernel's sources and is not used once
    they differ: a change to them takes the counters anew."""
    n = bench.traffic_from_profile(bench.TRAFFIC_PROFILE, bench.HEADLINE_SOURCES)
    assert n is not None
    assert 237383680 <= n < 1.1 * 237383680  # the sweep's algorithmic bytes
