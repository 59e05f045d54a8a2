"""bench.py prices the decode kernel with the committed counters' HBM bytes only
while they were taken on the decode sources as they are; this says when they
were not, and the counters have to be taken again."""
import bench


def test_committed_counters_are_of_the_current_decode_sources():
    assert bench.committed_traffic("skinny_decode") is not None
