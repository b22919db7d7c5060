"""awq_kv_attention on the GPU against the float64 oracle."""

import numpy as np
import pytest
import torch

import weight_only_int4_gemv_b200 as awq
from kv_util import DT, Setup, check, i32, to64

pytestmark = pytest.mark.gpu


def queries(rng, tokens, heads, dim, dtype, pad=0):
    """[tokens, heads, dim] as a slice of wider rows (pad extra values each)."""
    x = torch.from_numpy(rng.standard_normal((tokens, heads * dim + pad)) * 1.5).cuda().to(DT[dtype])
    return x[:, :heads * dim].view(tokens, heads, dim) if not pad else \
        x.as_strided((tokens, heads, dim), (heads * dim + pad, dim, 1))


def run(s, lens, new, heads, dtype, window=0, sinks=0, scale=None, max_q_len=None, extra=0, pad=0, tag="", wide=False):
    q = queries(s.rng, sum(new) + extra, heads, s.dim, dtype, pad)
    s.poison(lens)
    want, tol = s.expect(to64(q)[:sum(new)], lens, new, scale, window, sinks)
    out = torch.full(q.shape, 5.0, dtype=q.dtype, device="cuda")
    got = awq.awq_kv_attention(q, s.cache, s.batch(lens, new, max_q_len, wide=wide), scale=scale, window=window,
                               sinks=sinks, out=out)
    assert got is out
    assert awq.awq_device_error() == 0
    assert (out[sum(new):] == 5.0).all(), "rows behind the last sequence"
    check(out[:sum(new)], want, tol, tag)
    return q, out


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("group", [1, 3, 8, 16])
def test_single_tokens(dim, fmt, dtype, group):
    lens = [1, 2, 15, 16, 17, 64, 65, 200, 333]
    s = Setup(lens, 2, dim, 32, fmt, seed=group)
    run(s, lens, [1] * len(lens), 2 * group, dtype, max_q_len=1, extra=2, pad=8)


@pytest.mark.parametrize("dtype,fmt", [("fp16", "int8"), ("bf16", "e4m3")])
@pytest.mark.parametrize("new", [[5, 0, 33, 64], [1, 2, 130, 7], [200, 1, 1, 16]])
@pytest.mark.parametrize("dim,group", [(128, 4), (64, 1), (128, 7), (64, 16)])
@pytest.mark.parametrize("wide", [False, True])
def test_several_tokens(dtype, fmt, new, dim, group, wide):
    lens = [new[0], 90, 150, new[3] + 1]
    s = Setup(lens, 2, dim, 48, fmt, seed=sum(new))
    run(s, lens, new, 2 * group, dtype, max_q_len=max(new), extra=1, pad=8 * (group == 7), wide=wide)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (16, 4), (17, 16), (40, 33), (7, 300), (1000, 4)])
@pytest.mark.parametrize("new", [[1, 1, 1], [3, 40, 1], [150, 20, 9]])
@pytest.mark.parametrize("dim,fmt", [(128, "int8"), (64, "e4m3")])
@pytest.mark.parametrize("wide", [False, True])
def test_window_and_sinks(window, sinks, new, dim, fmt, wide):
    lens = [250, 64, 9]
    s = Setup(lens, 2, dim, 16, fmt, seed=window + sinks)
    run(s, lens, new, 6, "fp16", window=window, sinks=sinks, wide=wide)


def test_rows_that_see_nothing():
    """Padded entries (length 0), sequences shorter than their rows, no rows at all."""
    lens, new = [0, 3, 0, 40, 5], [1, 5, 0, 2, 9]
    s = Setup([max(n, 1) for n in lens], 2, 128, 16, "int8", seed=11)
    for group in (1, 4, 40):
        for wide in (False, True):
            _, out = run(s, lens, new, 2 * group, "fp16", wide=wide)
            assert (out[0] == 0).all() and (out[1:3] == 0).all()


@pytest.mark.parametrize("lens,heads,group", [([5000], 1, 4), ([3000, 1, 17, 2900], 2, 8), ([9000, 9001], 1, 1)])
def test_long_sequences_are_split(lens, heads, group):
    s = Setup(lens, heads, 128, 64, "int8", seed=12)
    run(s, lens, [1] * len(lens), heads * group, "fp16", max_q_len=1)
    run(s, lens, [min(3, n) for n in lens], heads * group, "bf16")


@pytest.mark.parametrize("dtype,fmt,dim", [("fp16", "int8", 128), ("bf16", "e4m3", 64)])
def test_many_rows_over_a_long_past_are_split(dtype, fmt, dim):
    lens, new = [3000, 700, 140], [70, 33, 140]
    s = Setup(lens, 1, dim, 64, fmt, seed=22)
    run(s, lens, new, 3, dtype, wide=True)
    run(s, lens, new, 3, dtype, window=300, sinks=130, wide=True)


def test_many_rows_are_reproducible():
    lens, new = [900, 260], [150, 260]
    s = Setup(lens, 2, 128, 16, "int8", seed=23)
    q = queries(s.rng, sum(new), 8, 128, "fp16")
    batch = s.batch(lens, new, wide=True)
    n = awq.awq_kv_attention_workspace_bytes(s.cache, batch, sum(new), 8)
    first = awq.awq_kv_attention(q, s.cache, batch)
    for fill in (0, 255):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(3):
            assert torch.equal(awq.awq_kv_attention(q, s.cache, batch, workspace=ws), first)


def test_split_is_reproducible_and_workspace_free_of_state():
    lens = [700, 5, 2100, 33]
    s = Setup(lens, 2, 128, 16, "int8", seed=13)
    batch = s.batch(lens, [1] * 4, 1)
    q = queries(s.rng, 4, 8, 128, "fp16")
    n = awq.awq_kv_attention_workspace_bytes(s.cache, batch, 4, 8)
    first = awq.awq_kv_attention(q, s.cache, batch)
    for fill in (0, 255):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(awq.awq_kv_attention(q, s.cache, batch, workspace=ws), first)
        assert torch.equal(awq.awq_kv_attention(q, s.cache, batch, workspace=ws), first)


def test_scales_far_apart():
    """Blocks whose value scales differ by many powers of two, zero blocks and
    loud keys: the weights stay accurate."""
    lens = [160, 64]
    s = Setup(lens, 2, 128, 16, "int8", seed=14)
    for w in range(2):
        f = 2.0 ** s.rng.integers(-14, 6, s.ref.scales[w].shape) if w else 2.0 ** s.rng.integers(-4, 2, s.ref.scales[0].shape)
        s.ref.scales[w] = (s.ref.scales[w] * f).astype(np.float32)
    zero = int(s.table[0, 2])
    s.ref.scales[1][zero] = 2.0 ** -60
    s.ref.codes[1][zero] = 128
    for t, a in ((s.cache.k_scales, s.ref.scales[0]), (s.cache.v_scales, s.ref.scales[1]),
                 (s.cache.v_pages, s.ref.codes[1])):
        t.copy_(torch.from_numpy(a))
    run(s, lens, [20, 1], 8, "fp16")
    run(s, lens, [40, 30], 8, "bf16", wide=True)
    run(s, lens, [1, 1], 2, "bf16", max_q_len=1)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3])
def test_other_logit_scales(scale):
    s = Setup([77, 31], 2, 64, 16, "int8", seed=15)
    run(s, [77, 31], [9, 31], 4, "fp16", scale=scale)
    run(s, [77, 31], [70, 31], 4, "fp16", scale=scale, wide=True)
    run(s, [77, 31], [70, 31], 4, "bf16", scale=scale, window=20, sinks=3, wide=True)


def test_tiny_and_large_queries():
    """bf16 queries whose magnitudes fp16 does not have."""
    s = Setup([50], 1, 128, 16, "int8", seed=16)
    for size in (2.0 ** -40, 2.0 ** 30, 0.0):
        q = (queries(s.rng, 2, 4, 128, "bf16").double() * size).to(torch.bfloat16)
        scale = 0.1 / size if size else 1.0
        want, tol = s.expect(to64(q), [50], [2], scale)
        check(awq.awq_kv_attention(q, s.cache, s.batch([50], [2]), scale=scale), want, tol, str(size))
        # the many-row kernel, rows that see nothing among them
        q = (queries(s.rng, 45, 4, 128, "bf16").double() * size).to(torch.bfloat16)
        want, tol = s.expect(to64(q), [40], [45], scale)
        check(awq.awq_kv_attention(q, s.cache, s.batch([40], [45], wide=True), scale=scale), want, tol, str(size))


def test_shared_pages_and_many_sequences():
    """Sequences that share their first pages; more sequences than threads."""
    n = 400
    s = Setup([40] + [17] * 3, 1, 64, 16, "int8", seed=17)
    table = np.zeros((n, 3), np.int32)
    table[:, 0] = s.table[0, 0]
    table[:, 1] = s.table[1 + np.arange(n) % 3, 1]
    lens = [17 + b % 9 for b in range(n)]
    s.table = table
    q = queries(s.rng, n, 2, 64, "fp16")
    want, tol = s.expect(to64(q), lens, [1] * n)
    check(awq.awq_kv_attention(q, s.cache, s.batch(lens, [1] * n, 1)), want, tol)


def test_bad_pages_are_recorded():
    s = Setup([100, 40], 2, 128, 16, "e4m3", seed=18)
    table = s.table.copy()
    table[0, 3] = s.n_pages + 7
    table[0, 4] = -9
    q = queries(s.rng, 2, 8, 128, "fp16")
    awq.awq_device_error()
    out = awq.awq_kv_attention(q, s.cache, s.batch([100, 40], [1, 1], table=table))
    assert awq.awq_device_error() == 16
    want, tol = s.expect(to64(q), [100, 40], [1, 1])
    check(out[1:], want[1:], tol[1:], "the other sequence")
    awq.awq_kv_attention(q, s.cache, awq.KvBatch(torch.from_numpy(s.table).cuda(), i32([2 ** 30, -4]), i32([0, 5, 3])))
    assert awq.awq_device_error() == 16
    # the many-row kernel
    q = queries(s.rng, 70, 8, 128, "fp16")
    out = awq.awq_kv_attention(q, s.cache, s.batch([100, 40], [40, 30], table=table, wide=True))
    assert awq.awq_device_error() == 16
    want, tol = s.expect(to64(q), [100, 40], [40, 30])
    check(out[40:], want[40:], tol[40:], "the other sequence")
    bad = s.batch([100, 40], [40, 30], wide=True)
    awq.awq_kv_attention(q, s.cache, awq.KvBatch(bad.block_table, i32([2 ** 30, -4]), i32([-3, 200, 50])))
    assert awq.awq_device_error() == 16


def test_cache_past_two_gigabytes():
    """Page offsets that pass 32 bits."""
    page, heads, dim = 64, 8, 128
    n = (1 << 31) // (page * heads * dim) + 40
    s = Setup([100], heads, dim, page, "int8", seed=19)
    big = awq.KvCache.allocate(n, heads, page, dim)
    move = {int(s.table[0, 0]): n - 1, int(s.table[0, 1]): n - 2}
    for src, dst in move.items():
        big.k_pages[dst], big.v_pages[dst] = s.cache.k_pages[src], s.cache.v_pages[src]
        big.k_scales[dst], big.v_scales[dst] = s.cache.k_scales[src], s.cache.v_scales[src]
    table = i32([[n - 1, n - 2]])
    q = queries(s.rng, 1, 16, dim, "fp16")
    want, tol = s.expect(to64(q), [100], [1])
    batch = awq.KvBatch(table, i32([100]), i32([0, 1]), 1)
    check(awq.awq_kv_attention(q, big, batch), want, tol)
    rows = torch.from_numpy(s.rng.standard_normal((2, 1, heads, dim))).cuda().half()
    awq.awq_kv_append(rows[0], rows[1], big, batch)
    for w in range(2):
        s.ref.append(w, s.table[0], 99, to64(rows[w]))
    want, tol = s.expect(to64(q), [100], [1])
    check(awq.awq_kv_attention(q, big, batch), want, tol)


def test_graph_replays_as_the_sequences_grow():
    """append and attention captured once, replayed with growing lengths; on a
    stream of its own; the replay's results are the eager ones."""
    s = Setup([80, 80, 80], 2, 128, 16, "int8", seed=20)
    start = [3, 40, 60]
    lens = i32(start)
    batch = awq.KvBatch(torch.from_numpy(s.table).cuda(), lens, i32([0, 1, 2, 3]), 1)
    rows = torch.zeros(3, 12, 128, dtype=torch.float16, device="cuda")
    q, k, v = rows.split((8, 2, 2), 1)
    from test_gpu_kv_cache import rope_table
    rope = torch.from_numpy(rope_table(80, 128)).cuda()
    ws = torch.empty(awq.awq_kv_attention_workspace_bytes(s.cache, batch, 3, 8), dtype=torch.uint8, device="cuda")
    out = torch.zeros(3, 8, 128, dtype=torch.float16, device="cuda")

    def step():
        turned = awq.awq_kv_append(k, v, s.cache, batch, q=q, rope=rope)
        awq.awq_kv_attention(turned, s.cache, batch, out=out, workspace=ws)

    keep = [t.clone() for t in (s.cache.k_pages, s.cache.v_pages, s.cache.k_scales, s.cache.v_scales)]
    inputs = [torch.from_numpy(s.rng.standard_normal((3, 12, 128))).cuda().half() for _ in range(6)]
    eager = []
    for x in inputs:
        rows.copy_(x)
        lens += 1
        step()
        eager.append(out.clone())
    for t, u in zip((s.cache.k_pages, s.cache.v_pages, s.cache.k_scales, s.cache.v_scales), keep):
        t.copy_(u)
    lens.copy_(i32(start))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        for x, want in zip(inputs, eager):
            rows.copy_(x)
            lens += 1
            graph.replay()
            assert torch.equal(out, want)
    torch.cuda.current_stream().wait_stream(side)


def test_two_streams_at_once():
    s = Setup([2000, 1500], 2, 128, 16, "int8", seed=21)
    batch = s.batch([2000, 1500], [1, 1], 1)
    qs = [queries(s.rng, 2, 8, 128, "fp16") for _ in range(2)]
    want = [awq.awq_kv_attention(q, s.cache, batch) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(awq.awq_kv_attention(qs[i], s.cache, batch))
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            assert torch.equal(y, want[i])


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("which", ["k_scales", "v_scales"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,fmt", [("fp16", "int8"), ("bf16", "e4m3")])
def test_a_spoilt_block_stays_with_the_rows_that_see_it(dtype, fmt, value, which, wide):
    """A block whose scale is not finite, in the same tiles as rows that do not see it: because they come before it,
    because the window has left it, because they belong to another head."""
    new = [45, 50] if wide else [10, 8]
    lens = [300, 84]                         # block 5 (positions 80 .. 95) is spoilt
    window, heads = 200, 8
    s = Setup(lens, 2, 128, 16, fmt, seed=22)
    for b in range(2):
        getattr(s.cache, which)[int(s.table[b, 5]), 0] = value
    q = queries(s.rng, sum(new), heads, 128, dtype)
    want, tol = s.expect(to64(q), lens, new, window=window)
    got = awq.awq_kv_attention(q, s.cache, s.batch(lens, new, wide=wide), window=window)
    assert awq.awq_device_error() == 0
    p = np.concatenate([np.arange(n - a, n) for n, a in zip(lens, new)])
    sees = (p >= 80) & (p - window < 95)
    assert sees.any() and not sees.all()
    half = heads // 2
    check(got[:, half:], want[:, half:], tol[:, half:], "the other head")
    clean = np.flatnonzero(~sees)
    check(got[torch.from_numpy(clean).cuda(), :half], want[clean, :half], tol[clean, :half], "rows that do not see it")
    if value != value:
        assert not torch.isfinite(got[torch.from_numpy(np.flatnonzero(sees)).cuda(), :half]).any()


def test_many_short_prompts():
    """More sequences than a warp has lanes, of more than 64 rows each, among them empty ones and one of many tiles of
    rows: the many-row kernel's schedule."""
    rng = np.random.default_rng(23)
    new = [int(n) for n in rng.integers(0, 20, 75)]
    new[3], new[40], new[41], new[74] = 700, 0, 19, 18
    lens = [n + int(e) for n, e in zip(new, rng.integers(-3, 60, 75))]
    lens = [max(n, 0) for n in lens]
    s = Setup(lens, 1, 64, 16, "int8", seed=24)
    run(s, lens, new, 4, "fp16", wide=True)


def test_two_graphs_share_a_workspace():
    """A chunk of prompt (many-row kernel) and single tokens (split over CTAs), captured apart, with one workspace,
    replayed in turn."""
    lens = [900, 700]
    s = Setup(lens, 2, 128, 16, "int8", seed=25)
    calls = [(s.batch(lens, [150, 90], wide=True), queries(s.rng, 240, 8, 128, "bf16")),
             (s.batch(lens, [1, 1], 1), queries(s.rng, 2, 8, 128, "bf16"))]
    want = [awq.awq_kv_attention(q, s.cache, b) for b, q in calls]
    n = max(awq.awq_kv_attention_workspace_bytes(s.cache, b, q.shape[0], 8) for b, q in calls)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.zeros_like(y) for y in want], []
    for (b, q), out in zip(calls, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            awq.awq_kv_attention(q, s.cache, b, out=out, workspace=ws)
        graphs.append(graph)
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for out in outs:
            out.fill_(7.0)
        for i in order:
            graphs[i].replay()
        for i in set(order):
            assert torch.equal(outs[i], want[i])
    assert awq.awq_device_error() == 0
