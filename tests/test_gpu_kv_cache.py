"""awq_kv_append and awq_kv_dequant on the GPU against the float64 oracle."""

import numpy as np
import pytest
import torch

import weight_only_int4_gemv_b200 as awq
from kv_util import DT, Setup, i32, to64
from oracle import kv_oracle as K

pytestmark = pytest.mark.gpu


def rope_table(n, rot, base=10000.0):
    f = base ** (-np.arange(rot // 2) / (rot // 2))
    a = np.arange(n)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def make_rows(rng, tokens, hq, hk, dim, dtype):
    """q, k, v as slices of one fused row matrix."""
    x = torch.from_numpy(rng.standard_normal((tokens, (hq + 2 * hk) * dim))).cuda().to(DT[dtype])
    return x, x.view(tokens, hq + 2 * hk, dim).split((hq, hk, hk), 1)


def same_codes(got, want, quotient, fmt, exact, tag):
    """Codes equal; where x was computed in fp32 (exact False), a neighbour is
    right too when the quotient lies within the arithmetic's error of the
    border: |x| <= sqrt 2 max|x|, three roundings of 2^-24 each of terms up
    to the block's range R, and one of the scale: 6 * 2^-24 R < 2^-21 R."""
    got, want = got.astype(np.int64), want.astype(np.int64)
    bad = got != want
    if exact or not bad.any():
        assert not bad.any(), f"{tag}: {bad.sum()} codes differ"
        return
    a, b = K.decode(got[bad].astype(np.uint8), fmt), K.decode(want[bad].astype(np.uint8), fmt)
    off = np.abs(quotient[bad] - (a + b) / 2)
    assert (off <= 2.0 ** -21 * K.TOP[fmt]).all(), f"{tag}: codes differ by {off.max()} from the border"


def check_cache(s, quotients, exact, tag):
    """Device pages against the oracle's: every page, touched or not."""
    for w, (pages, scales) in enumerate(((s.cache.k_pages, s.cache.k_scales), (s.cache.v_pages, s.cache.v_scales))):
        sc, ref = scales.cpu().numpy(), s.ref.scales[w]
        if exact or w == 1:
            assert np.array_equal(sc, ref, equal_nan=True), f"{tag}: scales"
        else:
            np.testing.assert_allclose(sc, ref, rtol=2.0 ** -21, err_msg=tag)
        codes = pages.cpu().numpy()
        same_codes(codes, s.ref.codes[w], quotients[w], s.fmt, exact or w == 1, f"{tag} {'kv'[w]}")


CASES = [
    # lens, new, heads, dim, page, dtype, fmt, rot, interleaved
    ([1], [1], (1, 1), 64, 16, "fp16", "int8", 64, False),
    ([5, 33, 48], [5, 33, 48], (4, 2), 128, 16, "bf16", "int8", 128, False),
    ([17, 100, 31], [1, 1, 1], (8, 8), 128, 64, "fp16", "e4m3", 64, True),
    ([40, 70, 129, 16], [3, 0, 40, 16], (6, 3), 64, 48, "bf16", "e4m3", 32, False),
    ([300, 7], [260, 6], (3, 1), 128, 32, "fp16", "int8", 16, True),
    ([64, 65], [17, 18], (5, 5), 64, 128, "fp16", "e4m3", 0, False),
    ([2, 0, 9], [4, 3, 9], (2, 1), 128, 16, "bf16", "int8", 128, False),      # rows without a position
]


@pytest.mark.parametrize("lens,new,heads,dim,page,dtype,fmt,rot,inter", CASES)
def test_append_and_read_back(lens, new, heads, dim, page, dtype, fmt, rot, inter):
    hq, hk = heads
    s = Setup([max(n, 1) for n in lens], hk, dim, page, fmt, seed=3, layers=2)
    tokens = sum(new) + 3                                # three rows behind the last sequence
    x, (q, k, v) = make_rows(s.rng, tokens, hq, hk, dim, dtype)
    before = x.clone()
    table = rope_table(max(lens), rot) if rot else None
    batch = s.batch(lens, new)
    out = torch.full((tokens, hq, dim), 7.0, dtype=DT[dtype], device="cuda")
    got = awq.awq_kv_append(k, v, s.cache, batch, q=q, rope=None if table is None else torch.from_numpy(table).cuda(),
                            interleaved=inter, q_out=out)
    assert got is out
    quotients = [np.zeros(c.shape) for c in s.ref.codes]
    want_q, has = np.full((tokens, hq, dim), 7.0), np.zeros(tokens, bool)
    at = 0
    for b, (n, a) in enumerate(zip(lens, new)):
        past = n - a
        skip = max(0, -past)
        rows = slice(at + skip, at + a)
        pos = np.arange(past + skip, n)
        at += a
        if not len(pos):
            continue
        has[rows] = True
        kk, qq = to64(k[rows]), to64(q[rows])
        if rot:
            cs = table[pos, :rot // 2], table[pos, rot // 2:]
            kk, qq = K.rotate(kk, *cs, inter), K.rotate(qq, *cs, inter)
        want_q[rows] = qq
        for w, y in ((0, kk), (1, to64(v[rows]))):
            t = s.ref.append(w, s.table[b], past + skip, y)
            quotients[w][s.table[b][pos // page], :, pos % page] = t
    check_cache(s, quotients, rot == 0, "append")
    # q: one rounding of fp32 values that are 3 roundings of terms <= sqrt 2 |pair| off
    err = np.abs(to64(out) - want_q)
    half = torch.finfo(DT[dtype]).eps / 2
    assert (err <= half * np.abs(want_q) + 2.0 ** -21 * np.abs(want_q).max() + 2.0 ** -25).all()
    assert torch.equal(x, before)
    assert awq.awq_device_error() == 0

    # read back: one rounding of the held value; rows without a token stay
    keys = [torch.full((tokens, hk, dim), 9.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
    awq.awq_kv_dequant(s.cache, batch, tokens, DT[dtype], *keys)
    scales = [s.cache.k_scales.cpu().numpy(), s.cache.v_scales.cpu().numpy()]
    codes = [s.cache.k_pages.cpu().numpy(), s.cache.v_pages.cpu().numpy()]
    held = K.Cache(codes[0], codes[1], scales[0], scales[1], fmt)
    for w in range(2):
        want, at = np.full((tokens, hk, dim), 9.0), 0
        for b, (n, a) in enumerate(zip(lens, new)):
            skip = max(0, a - n)
            if a > skip:
                want[at + skip:at + a] = held.values(w, s.table[b], n - a + skip, n)
            at += a
        exact = torch.from_numpy(want).float().to(DT[dtype])     # s * code is exact in fp32: 24 + 8 bits rounded once
        err = np.abs(to64(keys[w]) - want)
        assert (err <= (half + 2.0 ** -24) * np.abs(want) + 2.0 ** -25).all()
        assert torch.equal(keys[w].cpu()[~torch.from_numpy(has)], exact[~torch.from_numpy(has)])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_token_by_token_growth(fmt, dtype):
    """40 single tokens, each louder than the one before: every append raises
    its block's scale and rescales the codes before it."""
    s = Setup([48], 2, 64, 16, fmt, seed=5, filled=False)
    lens = i32([0])
    batch = awq.KvBatch(torch.from_numpy(s.table).cuda(), lens, i32([0, 1]), 1)
    for step in range(40):
        rows = torch.from_numpy(s.rng.standard_normal((2, 1, 2, 64)) * 1.07 ** step).cuda().to(DT[dtype])
        lens += 1
        awq.awq_kv_append(rows[0], rows[1], s.cache, batch)
        for w in range(2):
            s.ref.append(w, s.table[0], step, to64(rows[w]))
    check_cache(s, [np.zeros(c.shape) for c in s.ref.codes], True, "growth")


def test_appending_again_changes_nothing():
    s = Setup([90, 33], 2, 128, 32, "int8", seed=6)
    _, (q, k, v) = make_rows(s.rng, 30, 4, 2, 128, "fp16")
    rope = torch.from_numpy(rope_table(90, 128)).cuda()
    batch = s.batch([90, 33], [25, 5])
    first = awq.awq_kv_append(k, v, s.cache, batch, q=q, rope=rope)
    state = [t.clone() for t in (s.cache.k_pages, s.cache.v_pages, s.cache.k_scales, s.cache.v_scales)]
    second = awq.awq_kv_append(k, v, s.cache, batch, q=q, rope=rope)
    assert torch.equal(first, second)
    for a, b in zip(state, (s.cache.k_pages, s.cache.v_pages, s.cache.k_scales, s.cache.v_scales)):
        assert torch.equal(a, b)
    # q in place
    q2 = q.clone()
    awq.awq_kv_append(k, v, s.cache, batch, q=q2, rope=rope, q_out=q2)
    assert torch.equal(q2, first)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_zeros_and_extremes(fmt):
    """Zero blocks get the smallest scale and codes of zero; the type's largest values survive."""
    s = Setup([48], 2, 64, 16, fmt, seed=7, filled=False)
    x = torch.zeros(2, 48, 2, 64, device="cuda", dtype=torch.float16)
    x[:, 16:32] = 65504.0
    x[:, 20:24] = -65504.0
    x[:, 32:48] = 2.0 ** -24
    batch = s.batch([48], [48])
    awq.awq_kv_append(x[0], x[1], s.cache, batch)
    k, v = awq.awq_kv_dequant(s.cache, batch, 48)
    for y in (k, v):
        assert (y[:16] == 0).all()
        # s = fp32(65504 / R), times R: within two roundings of 2^-24, so fp16 gives it back
        assert torch.equal(y[16:32].float(), x[0][16:32].float())
        assert torch.equal(y[32:], x[0][32:])


def test_bad_tables_are_recorded_and_skipped():
    s = Setup([64, 64], 2, 64, 16, "int8", seed=8)
    table = s.table.copy()
    table[0, 1] = s.n_pages          # past the cache
    table[1, 0] = -1
    state = [t.clone() for t in (s.cache.k_pages, s.cache.v_pages)]
    _, (q, k, v) = make_rows(s.rng, 128, 2, 2, 64, "fp16")
    awq.awq_device_error()
    awq.awq_kv_append(k, v, s.cache, s.batch([64, 64], [64, 64], table=table))
    assert awq.awq_device_error() == 16
    assert awq.awq_device_error() == 0
    used = {int(p) for p in table.ravel() if 0 <= p < s.n_pages}
    for a, b in zip(state, (s.cache.k_pages, s.cache.v_pages)):
        for p in set(range(s.n_pages)) - used:
            assert torch.equal(a[p], b[p])
    # lengths and offsets out of range, positions past the rotation's table
    awq.awq_kv_append(k, v, s.cache, awq.KvBatch(torch.from_numpy(s.table).cuda(), i32([65, -5]), i32([0, 64, 128])))
    assert awq.awq_device_error() == 16
    awq.awq_kv_append(k, v, s.cache, awq.KvBatch(torch.from_numpy(s.table).cuda(), i32([64, 64]), i32([-7, 90, 20])))
    assert awq.awq_device_error() == 16
    awq.awq_kv_append(k, v, s.cache, s.batch([64, 64], [64, 64]), rope=torch.zeros(50, 64, device="cuda"))
    assert awq.awq_device_error() == 16
    awq.awq_kv_dequant(s.cache, s.batch([64, 64], [64, 64], table=table), 128)
    assert awq.awq_device_error() == 16


def test_many_sequences():
    """More sequences than a block has threads, most with nothing to write."""
    n = 1500
    lens = [1 + (i * 7) % 23 for i in range(n)]
    new = [1 if i % 5 == 0 else 0 for i in range(n)]
    s = Setup(lens, 1, 64, 32, "int8", seed=9)
    x = torch.from_numpy(s.rng.standard_normal((2, sum(new), 1, 64))).cuda().half()
    awq.awq_kv_append(x[0], x[1], s.cache, s.batch(lens, new, 1))
    at = 0
    for b in range(n):
        if new[b]:
            for w in range(2):
                s.ref.append(w, s.table[b], lens[b] - 1, to64(x[w, at:at + 1]))
            at += 1
    check_cache(s, [np.zeros(c.shape) for c in s.ref.codes], True, "many")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_non_finite_rows_spoil_their_block_alone(fmt, dtype):
    """A NaN or an infinity shows in its block's scale, leaves the other blocks and heads as they would be, and is gone
    when the block is written again from its first token."""
    s = Setup([100], 2, 64, 16, fmt, seed=9)
    batch = s.batch([100], [100])
    tensors = (s.cache.k_pages, s.cache.v_pages, s.cache.k_scales, s.cache.v_scales)
    rows = torch.from_numpy(s.rng.standard_normal((2, 100, 2, 64))).cuda().to(DT[dtype])
    awq.awq_kv_append(rows[0], rows[1], s.cache, batch)
    clean = [t.clone() for t in tensors]
    bad = rows.clone()
    spoilt = [(0, 20, 0, float("nan")), (0, 99, 1, float("-inf")), (1, 40, 1, float("inf")), (1, 64, 0, float("nan"))]
    for w, token, head, value in spoilt:
        bad[w, token, head, 7 * (token % 9)] = value
    awq.awq_kv_append(bad[0], bad[1], s.cache, batch)
    for w in range(2):
        keep = torch.ones(clean[2 + w].shape, dtype=torch.bool, device="cuda")
        for _, token, head, _ in (e for e in spoilt if e[0] == w):
            at = int(s.table[0, token // 16]), head, 0
            assert not torch.isfinite(tensors[2 + w][at]), (w, token)
            keep[at] = False
        assert torch.equal(tensors[2 + w][keep], clean[2 + w][keep])
        codes = [t[w].view(t[w].shape[0], 2, 1, 16, 64) for t in (tensors, clean)]
        assert torch.equal(codes[0][keep], codes[1][keep])
    held = awq.awq_kv_dequant(s.cache, batch, 100, DT[dtype])
    for w, token, head, value in spoilt:
        assert not torch.isfinite(held[w][token, head, 7 * (token % 9)]), (w, token)
    awq.awq_kv_append(rows[0], rows[1], s.cache, batch)
    for a, b in zip(tensors, clean):
        assert torch.equal(a, b)
