"""awq_kv_attention where a cache or a table holds what is allowed but unusual,
and awq_kv_dequant's rounding, against the float64 oracle. Each attention test
runs the few-row kernel (tiles of 8 and of 16 rows) and the many-row one."""

import numpy as np
import pytest
import torch

import weight_only_int4_gemv_b200 as awq
from kv_util import DT, Setup, check, i32, to64
from test_gpu_kv_attention import queries

pytestmark = pytest.mark.gpu

KINDS = [1, 10, 70]                 # rows of a sequence and head, at one query head to a key head


def is_many(cache, batch, tokens, heads):
    """Whether the call takes the many-row kernel, by its workspace: 32 bytes and two parts of 256 rows for each CTA.
    (No number of CTAs below 845 makes a few-row kernel's a multiple of that.)"""
    n = awq.awq_kv_attention_workspace_bytes(cache, batch, tokens, heads)
    return n % (32 + 2 * 256 * (cache.head_dim + 2) * 4) == 0


def attend(s, q, lens, new, table=None, window=0, sinks=0, scale=None):
    """The call, with a table wide enough that more than 64 rows take the many-row kernel."""
    many = max(new) > 64
    batch = s.batch(lens, new, max(new), table=table, wide=many)
    assert is_many(s.cache, batch, q.shape[0], q.shape[1]) == many
    return awq.awq_kv_attention(q, s.cache, batch, scale=scale, window=window, sinks=sinks)


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


@pytest.mark.parametrize("rows", KINDS)
@pytest.mark.parametrize("dtype,fmt,dim", [("fp16", "int8", 128), ("bf16", "e4m3", 64)])
@pytest.mark.parametrize("value", [2.0 ** -61, 2.0 ** -120, 1e-42])
def test_value_scales_below_the_smallest(rows, dtype, fmt, dim, value):
    """Blocks whose value scale lies below 2^-60, down to subnormal numbers, alone or beside others: their values count
    as 0 (the oracle's are below 2^-52), their keys as they are."""
    lens, new = [300, 84, 20], [rows, min(rows, 33), 1]
    s = Setup(lens, 2, dim, 16, fmt, seed=48)
    for b, i in [(0, 3), (0, 7), (0, 8), (1, 1), (2, 0), (2, 1)]:
        s.ref.scales[1][int(s.table[b, i]), i % 2 if b < 2 else slice(None)] = value
    put(s)
    q = queries(s.rng, sum(new), 2, dim, dtype)
    want, tol = s.expect(to64(q), lens, new)
    assert (np.abs(want[-1]) < 2.0 ** -52).all()
    check(attend(s, q, lens, new), want, tol)
    assert awq.awq_device_error() == 0


@pytest.mark.parametrize("rows", KINDS)
@pytest.mark.parametrize("which", ["k_scales", "v_scales"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf"), -1.0])
@pytest.mark.parametrize("dtype,fmt", [("fp16", "int8"), ("bf16", "e4m3")])
def test_a_spoilt_block_shows_in_every_row_that_sees_it(rows, which, value, dtype, fmt):
    """A scale that is no non-negative number makes NaN of all rows of its head that see the block, and of no other."""
    lens, new = [100 + rows], [rows]
    for block in (4, 6):                  # 64 .. 79, which the window leaves, and 96 .. 111, which the first rows reach
        s = Setup(lens, 2, 128, 16, fmt, seed=43)
        getattr(s.cache, which)[int(s.table[0, block]), 0] = value
        q = queries(s.rng, rows, 2, 128, dtype)
        want, tol = s.expect(to64(q), lens, new, window=50)
        got = attend(s, q, lens, new, window=50)
        p = 100 + np.arange(rows)
        sees = (p >= 16 * block) & (p - 50 < 16 * block + 15)
        check(got[:, 1:], want[:, 1:], tol[:, 1:], "the other head")
        clean, bad = np.flatnonzero(~sees), np.flatnonzero(sees)
        assert len(bad)
        check(got[torch.from_numpy(clean).cuda(), :1], want[clean, :1], tol[clean, :1], "rows that do not see it")
        y = got[torch.from_numpy(bad).cuda(), 0]
        assert torch.isnan(y).all(), f"block {block}: {(~torch.isnan(y)).sum()} values are no NaN"


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("sign", [1, -1])
def test_a_first_token_with_an_infinity_shows(many, fmt, sign):
    """A token that opens a block, with an infinity in its key: no other token's zero code lies in the block."""
    n = 33
    new = 97 if many else 1                # a prompt up to that token, or the token alone
    lens = [n + 64] if many else [n]
    s = Setup(lens, 1, 64, 16, fmt, seed=44)
    rows = torch.from_numpy(s.rng.standard_normal((2, lens[0], 1, 64))).cuda().half()
    batch = s.batch(lens, lens)
    awq.awq_kv_append(rows[0], rows[1], s.cache, batch)
    rows[0, -1, 0, 5] = float("inf")
    awq.awq_kv_append(rows[0, -1:], rows[1, -1:], s.cache, s.batch(lens, [1]))
    q = queries(s.rng, new, 1, 64, "fp16")
    q[:, 0, 5] = 2.0 * sign
    got = attend(s, q, lens, [new])
    assert torch.isnan(got[-1]).all()
    if many:
        assert torch.isfinite(got[:-1]).all()


@pytest.mark.parametrize("fmt,scale", [("e4m3", None), ("int8", 8.0), ("e4m3", -8.0)])
def test_loudest_bf16_queries_over_keys_of_zero(fmt, scale):
    """bf16 rows near the type's largest number have logits of 0 on keys of 0."""
    for rows in KINDS:
        s = Setup([150], 1, 64, 16, fmt, seed=45)
        s.ref.codes[0][:] = 128 if fmt == "int8" else 0
        s.ref.scales[0][:] = 2.0 ** -60
        put(s)
        q = (queries(s.rng, rows, 1, 64, "bf16").sign() * 2.0 ** 126).to(torch.bfloat16)
        want, tol = s.expect(np.zeros((rows, 1, 64)), [150], [rows])
        check(attend(s, q, [150], [rows], scale=scale), want, tol, str(rows))


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dtype,fmt", [("fp16", "int8"), ("bf16", "e4m3")])
def test_a_long_tail_keeps_its_mass(many, dtype, fmt):
    """A few keys with a weight of 1, 2^14 others with 2^-25.2 each, whose values alone are not 0: the output is their
    share of the sum, about 2^-14. Weights are fp16 against a running maximum lifted to 2^7, where half a step of the
    subnormal numbers is 2^-32 of the largest: 2^14 of them move y by 2^-18 at most; logits, statistics and the
    weights' own rounding as in kv_util. As many sequences (of the same pages) as there are CTAs or so, so that a
    sequence's keys meet one running maximum and are not cut into runs with maxima of their own."""
    n, new, dim, seqs = (1 << 14) + 200, 70 if many else 1, 64, 148 if many else 592
    s = Setup([n], 1, dim, 64, fmt, filled=False)
    one, top, zero = (255, 127.0, 128) if fmt == "int8" else (0x7e, 448.0, 0)     # the largest code, its number, 0's
    for t, c in ((s.cache.k_pages, zero), (s.cache.v_pages, one)):
        t.fill_(c)
    s.cache.k_scales.fill_(1.0 / top)
    s.cache.v_scales.fill_(1.0 / top)
    for token in (range(0, 64, 16) if many else range(0, 128, 16)):
        page, at = int(s.table[0, token // 64]), token % 64
        s.cache.k_pages[page, 0, at, 0] = one                # the loud keys: (1, 0, 0, ..), a block each, so that every
        s.cache.v_pages[page, 0, at] = zero                  # warp of the few-row kernel meets one
    loud = 4 if many else 8
    q = torch.zeros(seqs * new, 1, dim, device="cuda", dtype=DT[dtype])
    q[:, 0, 0] = 16.0
    x = 25.2 * np.log(2.0)
    scale = float(np.float32(x / 16.0))
    batch = s.batch([n] * seqs, [new] * seqs, new, table=np.repeat(s.table, seqs, 0), wide=many)
    assert is_many(s.cache, batch, q.shape[0], 1) == many
    got = awq.awq_kv_attention(q, s.cache, batch, scale=scale)
    assert awq.awq_device_error() == 0
    seen = n - new + 1 + np.arange(new)                   # keys of each row
    tail = (seen - loud) * np.exp(-16.0 * scale) / loud
    want = tail / (1 + tail)
    d = 2.0 ** -16 * x + 2.0 ** -17
    tol = (2.0 ** -11 + 2 * d) * want + 2.0 ** -32 * seen
    shape = (seqs, new, 1, dim)
    check(got, *(np.broadcast_to(a[None, :, None, None], shape).reshape(got.shape) for a in (want, tol)))


@pytest.mark.parametrize("rows", KINDS)
def test_waits_give_up_and_recover(rows):
    """Pipeline waits made to run out without a fault: with a limit of 1 ns the first wait for a slot, or a place for
    q rows, that is not free gives up, other copies in flight; with longer ones a later wait may. The call records bit
    3, lets its copies and products land and returns; with the limit restored the next call gives the bits of the one
    before. Sequences share their pages and are many, so that CTAs have more tiles than slots and several items."""
    seqs = 48
    lens, new = [3000] * seqs, [rows] * seqs
    s = Setup([3000], 2, 128, 16, "int8", seed=47)
    s.table = np.repeat(s.table, seqs, 0)
    q = queries(s.rng, sum(new), 2, 128, "bf16")
    first = attend(s, q, lens, new)
    want, tol = s.expect(to64(q[:rows]), lens[:1], new[:1])
    check(first[:rows], want, tol)
    assert awq.awq_device_error() == 0
    for limit in (1, 1, 500, 1000, 2000, 4000):
        try:
            awq.awq_debug_set_wait_limit_ns(limit)
            attend(s, q, lens, new)
            torch.cuda.synchronize()
            error = awq.awq_device_error()
        finally:
            awq.awq_debug_set_wait_limit_ns(0)
        assert error == 8 or limit > 1 and error == 0, limit
        assert torch.equal(attend(s, q, lens, new), first)
        assert awq.awq_device_error() == 0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_dequant_rounds_once(fmt, dtype):
    """Each value is one rounding of the exact product: float64 holds it (24 + 8 bits), and rounds it to 16 bits once."""
    n = 4096
    s = Setup([n], 2, 64, 64, fmt, seed=46)
    k, v = awq.awq_kv_dequant(s.cache, s.batch([n], [n]), n, dtype)
    for w, y in ((0, k), (1, v)):
        exact = s.ref.values(w, s.table[0], 0, n)
        mantissa = 11 if dtype is torch.float16 else 8
        lowest = -14 if dtype is torch.float16 else -126
        e = np.maximum(np.floor(np.log2(np.abs(np.where(exact == 0, 1.0, exact)))), lowest) - (mantissa - 1)
        want = np.rint(exact / 2.0 ** e) * 2.0 ** e       # a power of two divides exactly; ties to even
        assert np.array_equal(to64(y), want), f"{(to64(y) != want).sum()} values"


@pytest.mark.parametrize("rows", KINDS)
@pytest.mark.parametrize("pad", [8, 16])
@pytest.mark.parametrize("dtype,fmt,dim", [("fp16", "int8", 64), ("bf16", "e4m3", 128)])
def test_strided_outputs_of_a_layer_among_others(rows, pad, dtype, fmt, dim):
    """Rows of out that are columns of wider ones (at 16 and at 32 bytes' alignment), a block table that is a slice, a
    cache that is one layer of an array: the bits of the dense call, and nothing beside the columns written."""
    lens, new = [700, 130, 40], [rows, min(rows, 130), 0]
    s = Setup(lens, 2, dim, 32, fmt, seed=49, layers=3)
    q = queries(s.rng, sum(new), 6, dim, dtype)
    many = rows * 3 > 64
    extra = 40000 // s.page if many else 3
    table = torch.cat((torch.from_numpy(s.table), torch.full((3, extra + 5), -1, dtype=torch.int32)), 1).cuda()
    batch = awq.KvBatch(table[:, :s.table.shape[1] + extra], i32(lens), i32(np.concatenate([[0], np.cumsum(new)])), rows)
    assert is_many(s.cache, batch, sum(new), 6) == many
    want, tol = s.expect(to64(q), lens, new)
    dense = awq.awq_kv_attention(q, s.cache, batch)
    check(dense, want, tol)
    buffer = torch.full((sum(new), 6 * dim + 2 * pad), 3.0, dtype=q.dtype, device="cuda")
    out = buffer[:, pad:-pad].unflatten(1, (6, dim))
    assert awq.awq_kv_attention(q, s.cache, batch, out=out) is out
    assert torch.equal(out, dense)
    assert (buffer[:, :pad] == 3.0).all() and (buffer[:, -pad:] == 3.0).all()


@pytest.mark.parametrize("rows", KINDS)
def test_batches_without_rows_of_any_sequence(rows):
    """All sequences bring 0 rows: nothing is written, nothing recorded."""
    s = Setup([100, 64], 2, 64, 16, "int8", seed=50)
    q = queries(s.rng, rows, 2, 64, "fp16")
    kept = [t.clone() for t in (s.cache.k_pages, s.cache.v_pages, s.cache.k_scales, s.cache.v_scales)]
    for lens in ([100, 64], [0, 0]):
        for n in (1, 2):
            batch = awq.KvBatch(torch.from_numpy(s.table[:n]).cuda(), i32(lens[:n]), i32([0] * (n + 1)), rows)
            for b in (batch, s.batch(lens, [0, 0], rows, wide=True)):
                out = torch.full_like(q, 5.0)
                awq.awq_kv_attention(q, s.cache, b, out=out)
                turned = awq.awq_kv_append(q, q, s.cache, b, q=q, q_out=torch.full_like(q, 5.0))
                back = awq.awq_kv_dequant(s.cache, b, rows, q.dtype, torch.full_like(q, 5.0), torch.full_like(q, 5.0))
                for t in (out, turned, *back):
                    assert (t == 5.0).all()
    assert awq.awq_device_error() == 0
    for a, b in zip(kept, (s.cache.k_pages, s.cache.v_pages, s.cache.k_scales, s.cache.v_scales)):
        assert torch.equal(a, b)


def test_more_rows_than_the_bound_said():
    """max_q_len chooses the kernel and nothing else."""
    lens, new = [333, 90], [140, 3]
    s = Setup(lens, 2, 128, 16, "int8", seed=51)
    q = queries(s.rng, sum(new), 8, 128, "fp16")
    want, tol = s.expect(to64(q), lens, new)
    for bound in (1, 4, 16, 140, None):
        for wide in (False, True):
            check(awq.awq_kv_attention(q, s.cache, s.batch(lens, new, bound, wide=wide)), want, tol, f"{bound} {wide}")
    assert awq.awq_device_error() == 0


@pytest.mark.parametrize("rows", KINDS)
@pytest.mark.parametrize("window,sinks", [(5, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 1), (399, 0), (400, 1), (1, 399)])
def test_windows_and_sinks_of_any_size(rows, window, sinks):
    lens, new = [400, 80], [rows, min(rows, 80)]
    s = Setup(lens, 2, 64, 16, "e4m3", seed=52)
    q = queries(s.rng, sum(new), 2, 64, "bf16")
    want, tol = s.expect(to64(q), lens, new, window=window, sinks=sinks)
    check(attend(s, q, lens, new, window=window, sinks=sinks), want, tol)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_takes_and_gives_strided_rows(fmt):
    """k, v, q and q_out as columns of wider rows, of which nothing else is written; a captured append and read-back,
    replayed on a stream of its own."""
    lens, new = [50, 33], [20, 33]
    made = []
    for strided in (False, True):
        s = Setup(lens, 2, 128, 16, fmt, seed=53, layers=2)
        x = torch.from_numpy(s.rng.standard_normal((53, 8, 128))).cuda().half()
        q, k, v = (t.contiguous() for t in x.split((4, 2, 2), 1))
        out = torch.zeros_like(q)
        if strided:
            rows = torch.full((53, 8 * 128 + 24), 9.0, dtype=torch.float16, device="cuda")
            q, k, v = (rows[:, a:a + t[0].numel()].unflatten(1, t.shape[1:]).copy_(t)
                       for a, t in ((8, q), (8 + 512, k), (16 + 768, v)))
            wide = torch.full((53, 4 * 128 + 16), 9.0, dtype=torch.float16, device="cuda")
            out = wide[:, 8:-8].unflatten(1, (4, 128))
        batch = s.batch(lens, new)
        back = [torch.zeros(53, 2, 128, dtype=torch.float16, device="cuda") for _ in range(2)]

        def step():
            awq.awq_kv_append(k, v, s.cache, batch, q=q, q_out=out)
            awq.awq_kv_dequant(s.cache, batch, 53, torch.float16, *back)

        if strided:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    step()
                graph.replay()
                graph.replay()
            torch.cuda.current_stream().wait_stream(side)
            assert (wide[:, :8] == 9.0).all() and (wide[:, -8:] == 9.0).all()
        else:
            step()
        made.append([t.clone() for t in (s.cache.k_pages, s.cache.v_pages, s.cache.k_scales, s.cache.v_scales, out, *back)])
    for a, b in zip(*made):
        assert torch.equal(a, b)
    assert awq.awq_device_error() == 0
