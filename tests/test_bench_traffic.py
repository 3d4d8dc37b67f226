"""The default workload's recorded DRAM traffic belongs to the decode kernel's current sources: the bench reports none
for others."""
import bench


def test_the_traffic_record_is_of_the_current_decode_sources():
    assert bench.recorded_traffic("llama2-13b", 16) is not None
