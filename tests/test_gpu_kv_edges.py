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


def put(s):
    """The oracle's codes and scales into the device's cache."""
    for t, a in ((s.cache.k_pages, s.ref.codes[0]), (s.cache.v_pages, s.ref.codes[1]),
                 (s.cache.k_scales, s.ref.scales[0]), (s.cache.v_scales, s.ref.scales[1])):
        t.copy_(torch.from_numpy(a))


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


@pytest.mark.parametrize("rows", KINDS)
@pytest.mark.parametrize("dtype,fmt,dim", [("fp16", "int8", 128), ("bf16", "e4m3", 64)])
def test_scales_of_zero(rows, dtype, fmt, dim):
    """A block of scale 0 holds zeros whatever its codes: its keys have logits of 0, its values count as 0 with their
    keys' weights."""
    lens, new = [300, 84, 20], [rows, min(rows, 33), 1]
    s = Setup(lens, 2, dim, 16, fmt, seed=42)
    for w, blocks in ((0, [(0, 2), (0, 7), (1, 0)]), (1, [(0, 3), (0, 7), (0, 8), (1, 1), (2, 0), (2, 1)])):
        for b, i in blocks:
            s.ref.scales[w][int(s.table[b, i]), i % 2 if b < 2 else slice(None)] = 0.0
    # codes that an own quantizer may leave in such a block
    s.ref.codes[1][int(s.table[0, 3]), 1] = 0
    s.ref.codes[1][int(s.table[0, 8]), 0] = 255 if fmt == "int8" else 0x7e
    put(s)
    q = queries(s.rng, sum(new), 2, dim, dtype)
    want, tol = s.expect(to64(q), lens, new)
    assert (want[-1] == 0).all()
    check(attend(s, q, lens, new), want, tol)
    assert awq.awq_device_error() == 0
