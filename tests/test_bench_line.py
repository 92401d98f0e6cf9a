"""bench.py's line, what needs no GPU: the DRAM traffic figures it reports belong to
the kernels as they are."""
import bench


def test_traffic_figures_describe_the_current_kernels():
    """A figure is reported while the sources it was captured with stand; the default
    run's calls (down at M = 128 under both partition rules, decode attention) and
    gate at M = 32 keep theirs."""
    assert {h for _, h in bench.NCU_TRAFFIC.values()} == {bench.tc_source_hash()}
    assert {("down", 128, 4), ("down", 128, 7), ("gate", 32, 2)} <= set(bench.NCU_TRAFFIC)
    assert {h for _, h in bench.ATTN_TRAFFIC.values()} == {bench.tc_source_hash(bench.ATTN_SOURCES)}
