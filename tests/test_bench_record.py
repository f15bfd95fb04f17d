"""The benchmark's record of the FFN GEMM's DRAM traffic is the one of the GEMM
source that is here (it is keyed by the source's hash, and reads as null where
the hash is another one)."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_gemm_traffic_record_is_of_this_source():
    sys.path.insert(0, ROOT)
    try:
        import bench
    finally:
        sys.path.remove(ROOT)
    key = bench.src_hash("hif4_gemm.cuh", "hif4_sm100.cuh", "hif4_encode.cuh", "hif4_internal.cuh")
    assert bench.NCU_TRAFFIC.get(("gemm", key))
