"""Every call that takes a workspace has a query of its size, without a GPU where
the size does not depend on one."""
import ctypes
import inspect
import struct

import zero_sharded_mixed_zero1_gb300 as z
from zero_sharded_mixed_zero1_gb300 import build as zbuild
from zero_sharded_mixed_zero1_gb300 import clip as zc

EINVAL = -1


def test_each_call_with_a_workspace_has_a_query():
    """(The feed-forward block has one for its three calls.)"""
    calls = {n for n in dir(z) if n.startswith("zero1_") and callable(getattr(z, n))
             and "workspace" in inspect.signature(getattr(z, n)).parameters}
    assert calls
    for name in calls:
        query = "zero1_gated_ffn_workspace" if name.startswith("zero1_gated_ffn") else name.replace("_backward", "") + "_workspace"
        assert hasattr(z, query), name


def test_the_shards_norm_takes_what_its_query_says_and_no_less():
    zbuild.build()
    lib, n = zc._lib(), z.zero1_shard_grad_sumsq_workspace()
    plan, hp = z.zero1_plan(1000, 2, 8), z.AdamW(global_batch=64, step=3)
    at = lambda k: (1 << 32) + (k << 26)  # noqa: E731  (nothing reads from there)
    call = lambda size: lib.zero1_shard_grad_sumsq(ctypes.byref(plan), 0, 2, struct.pack("=2Q", at(1), at(2)),  # noqa: E731
                                                   ctypes.byref(hp.c_struct()), at(3), None, 0, at(4), size, None)
    assert call(n - 1) == EINVAL and b"workspace" in lib.zero1_last_error()
