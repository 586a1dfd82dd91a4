"""The benchmark reports the DRAM traffic of its dominant calls from the counters under profiles/, as
long as the sources are those that were measured.  A change to one of these sources needs its
counters taken again (the commands stand beside them)."""
import pytest


@pytest.mark.parametrize("workload,call", [("train_step", "octo_attn_bwd"), ("train_tree", "octo_attn_bwd"), ("episode", "octo_attn_bwd"),
                                           ("decode", "octo_decode"), ("decode_small", "octo_decode")])
def test_profiled_traffic_is_of_these_sources(workload, call):
    import bench
    traffic, note = bench.profiled_traffic(workload, call, 10 ** 9)
    assert traffic is not None and traffic > 0, note
