"""The bench's DRAM traffic of an attention launch is of the kernel that it runs: the
captures that it quotes were taken on the present sources (attn.cu and its PTX
helpers; a change of either needs a new capture, and helpers of other kernels belong
in headers of their own)."""
import bench


def test_the_recorded_traffic_is_of_the_present_kernel():
    now = bench.kernel_source_hash()
    assert {r["source"] for r in bench.NCU_TRAFFIC.values()} == {now}
