"""awq_kv_attention where a cache or a table holds what is allowed but unusual,
against the float64 oracle. Each test runs the few-row kernel (tiles of 8 and
of 16 rows) and the many-row one."""

import numpy as np
import pytest
import torch

import weight_only_int4_gemv_b200 as awq
from kv_util import Setup, check, to64
from test_gpu_kv_attention import queries

pytestmark = pytest.mark.gpu

KINDS = [1, 10, 70]                 # rows of a sequence and head, at one query head to a key head


def is_many(cache, batch, tokens, heads):
    """Whether the call takes the many-row kernel, by its workspace: 32 bytes and two parts of 256 rows for each CTA.
    (No number of CTAs below 845 makes a few-row kernel's a multiple of that.)"""
    n = awq.awq_kv_attention_workspace_bytes(cache, batch, tokens, heads)
    return n % (32 + 2 * 256 * (cache.head_dim + 2) * 4) == 0


def attend(s, q, lens, new, table=None, window=0, sinks=0):
    """The call, with a table wide enough that more than 64 rows take the many-row kernel."""
    many = max(new) > 64
    batch = s.batch(lens, new, max(new), table=table, wide=many)
    assert is_many(s.cache, batch, q.shape[0], q.shape[1]) == many
    return awq.awq_kv_attention(q, s.cache, batch, window=window, sinks=sinks)


@pytest.mark.parametrize("rows", KINDS)
@pytest.mark.parametrize("dtype,fmt,dim", [("fp16", "int8", 128), ("bf16", "e4m3", 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 20)])
def test_pages_out_of_range_are_as_if_masked(rows, dtype, fmt, dim, window, sinks):
    """Blocks whose page the table does not name have no weight, whatever shared memory held before, and the keys
    around them keep theirs."""
    lens, new = [333, 150], [rows, max(rows - 3, 1)]
    s = Setup(lens, 2, dim, 16, fmt, seed=41)
    table = s.table.copy()
    gone = [[1, 4, 8, 9, 15, 17, 20], [0, 3, 7]]
    for b, blocks in enumerate(gone):
        table[b, blocks] = [-1 - i if i % 2 else s.n_pages + i for i in range(len(blocks))]
    keep = [np.ones(n, bool) for n in lens]
    for k, blocks in zip(keep, gone):
        for i in blocks:
            k[16 * i:16 * i + 16] = False
    q = queries(s.rng, sum(new), 2, dim, dtype)
    attend(s, q, lens, new)             # another call's data in shared memory
    assert awq.awq_device_error() == 0
    got = attend(s, q, lens, new, table, window, sinks)
    assert awq.awq_device_error() == 16
    want, tol = s.expect(to64(q), lens, new, window=window, sinks=sinks, keep=keep)
    check(got, want, tol)
