"""Rules of the kernels' sources that no run can show.

A kernel launched as a programmatic dependent is resident while the kernel before it on the stream still runs, and
waits for it (wait_primary_grid).  What it reads after that wait may have been written during its own lifetime, so it
must not come through the read-only path: no __ldg, and no const __restrict__ pointer, which lets the compiler take
that path by itself."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_10_gb300", "csrc")
# device functions that such kernels call after their wait
HELPERS = ["sparse_block", "lane_bounds", "four_scores", "exact_score", "row_blocks", "prefill_unit"]


def functions():
    """(file, name, signature, body) of every function of the kernels' sources."""
    for f in sorted(os.listdir(CSRC)):
        if not f.endswith((".cu", ".cuh")):
            continue
        text = re.sub(r"//.*", "", open(os.path.join(CSRC, f), encoding="utf-8").read())
        for m in re.finditer(r"(__global__|__device__)[^;{}]*?\b(\w+)\s*\(([^;{}]*)\)\s*\{", text):
            depth, at = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[at], 0)
                at += 1
            yield f, m.group(2), m.group(0), text[m.end():at]


def waiting_kernels():
    return [x for x in functions() if "__global__" in x[2] and "wait_primary_grid()" in x[3]]


def test_the_waiting_kernels_are_found():
    names = {re.search(r"(\w+_kernel)", sig).group(1) for _, _, sig, _ in waiting_kernels()}
    assert {"append_int_kernel", "read_kernel", "key_bounds_kernel", "block_score_kernel", "select_kernel",
            "decode_int_kernel", "decode_kernel", "decode_mma_kernel", "merge_kernel", "prefill_tc_kernel"} <= names


@pytest.mark.parametrize("at", range(len(waiting_kernels())))
def test_no_read_only_loads_after_the_wait(at):
    f, _, sig, body = waiting_kernels()[at]
    assert "__restrict__" not in sig, (f, sig)
    assert "__ldg(" not in body[body.index("wait_primary_grid()"):], f
    # a pointer made const __restrict__ inside would do the same
    assert "__restrict__" not in body, f


@pytest.mark.parametrize("name", HELPERS)
def test_no_read_only_loads_in_what_they_call(name):
    found = [(f, body) for f, n, sig, body in functions() if n == name]
    assert found, name
    for f, body in found:
        assert "__ldg(" not in body, f
