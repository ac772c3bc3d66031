"""The DRAM traffic that bench.py reports comes from a committed capture, and is
left out when the sources of the captured kernel have changed since.  What
that kernel is not built from has to stay outside the comparison."""
import json
import os

import bench


def test_listed_sources_hold_no_code_of_the_paged_cache():
    csrc = os.path.join(bench.ROOT, "megatron_tensor_transformer_plan_b200", "csrc")
    for name in bench.DECODE_SOURCES:
        with open(os.path.join(csrc, name), encoding="utf-8") as f:
            assert "paged" not in bench._code_only(f.read()).lower(), name


def test_what_counts_as_code():
    code = bench._code_only
    assert code("a b; // x") == code("a  b; /* y\n z */") == "a b;"
    assert code('#include "tpl_attn.cuh"\nint x;') == "int x;"            # not listed
    listed = '#include "tpl_gemv.cuh"\nint x;'
    assert "tpl_gemv.cuh" in code(listed) and code(listed) != code("int x;")
    assert "cuda.h" in code("#include <cuda.h>\nint x;")


def test_the_capture_names_its_sources():
    with open(os.path.join(bench.ROOT, "profiles", "gemv_gate_up_stack.json"), encoding="utf-8") as f:
        capture = json.load(f)
    assert len(capture["source_hash"]) == len(bench.kernel_source_hash())
    if capture["source_hash"] == bench.kernel_source_hash():
        assert bench.recorded_traffic() == capture["dram_bytes_per_launch"] > 0
    else:
        assert bench.recorded_traffic() is None
