"""The DRAM traffic that the benchmark reports beside its default workload is
a committed ncu figure; it holds for the kernel sources of this tree."""
import bench


def test_the_default_workloads_figure_was_taken_on_these_sources():
    bytes_per_launch, source = bench.recorded_traffic_with_source("block_swiglu_llama8b_chain")
    assert bytes_per_launch is not None, source
