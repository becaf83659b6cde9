"""Prefill calls of both element types at the same time: they take their work from counters of one pool, so no two of
them may hold the same one."""
import numpy as np
import pytest
import torch

import quant_util as qu
from test_gpu_prefill_scored import Case

def test_types_take_their_counters_from_one_sequence():
    """The source: the slot that a launch takes next is not a variable of each type's own."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(qu.__file__), "..", "paged_kv_cache_10_gb300", "csrc", "pkv_prefill.cu")).read()
    body = src[src.index("cudaError_t launch_prefill("):]
    body = body[:body.index("\n}\n")]
    assert not re.search(r"static\s+std::atomic", body) and len(re.findall(r"\nstd::atomic<uint32_t> \w+\{0\};", src)) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("rounds", [40])
def test_two_types_on_two_streams(rounds):
    from paged_kv_cache_10_gb300 import build, pagedkv as pk
    build.build()
    pk.get_device_error()
    cs = [Case(pk, t, 128, 2, 4, t, {}, seed=1) for t in ("f16", "bf16")]
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    for c in cs:
        c.qd, c.outs = c.q.cuda(), [torch.full_like(c.q, 7.0, device="cuda") for _ in range(rounds)]
        c.args, c.st = (i32(c.start), c.n_max, i32(c.tables), i32(c.lens)), torch.cuda.Stream()
    torch.cuda.synchronize()
    for r in range(rounds):
        for c in cs:
            pk.paged_attention_prefill(c.qd, c.kd, c.vd, c.pools.desc, *c.args, c.scale, c.outs[r], stream=c.st)
    torch.cuda.synchronize()
    for c in cs:
        c.check(c.outs[0])
        assert all(torch.equal(o, c.outs[0]) for o in c.outs)
    assert pk.get_device_error() == 0
