"""Refusals of the KV-cache entry points, without a GPU: every call below is
rejected (or has no work) before any CUDA call, so the addresses passed are
never dereferenced."""

import ctypes

import numpy as np
import pytest
import torch

import weight_only_int4_gemv_b200 as awq
from oracle import kv_oracle as K

OK, NULL, SHAPE, ALIGN, UNSUP, CUDA, WS = range(7)
A, MIS, ODD = 0x10000, 0x10008, 0x10001


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(awq.LIB_PATH):
        from weight_only_int4_gemv_b200 import build
        build.build()
    return awq.lib()


def cache(**kw):
    d = dict(k_pages=A, v_pages=A, k_scales=A, v_scales=A, n_pages=10, page_stride=2 * 32 * 128, scale_stride=4,
             n_kv_heads=2, head_dim=128, page_size=32, format=0)
    d.update(kw)
    return awq.KvCacheArgs(**d)


def batch(**kw):
    d = dict(block_table=A, seq_lens=A, q_indptr=A, table_stride=4, n_seqs=3, max_pages=4, max_q_len=1)
    d.update(kw)
    return awq.KvBatchArgs(**d)


def rope(**kw):
    d = dict(table=A, row_stride=128, n_positions=100, rot_dim=128, interleaved=0)
    d.update(kw)
    return awq.KvRopeArgs(**d)


def ref(s):
    return None if s is None else ctypes.addressof(s)


def append(L, c, b, n=3, dtype=0, k=A, ks=256, v=A, vs=256, q=A, qs=512, hq=4, r=None, o=A, os_=512):
    return L.awq_kv_append(ref(c), ref(b), n, dtype, k, ks, v, vs, q, qs, hq, ref(r), o, os_, None)


def dequant(L, c, b, n=3, dtype=0, k=A, v=A):
    return L.awq_kv_dequant(ref(c), ref(b), n, dtype, k, v, None)


def attend(L, c, b, n=3, dtype=0, q=A, qs=512, hq=4, scale=1.0, window=0, sinks=0, o=A, os_=512, ws=None, wb=0):
    return L.awq_kv_attention(ref(c), ref(b), n, dtype, q, qs, hq, scale, window, sinks, o, os_, ws, wb, None)


CACHE_FAULTS = [
    (dict(format=2), UNSUP), (dict(format=-1), UNSUP), (dict(head_dim=96), UNSUP), (dict(head_dim=0), UNSUP),
    (dict(n_kv_heads=0), SHAPE), (dict(n_kv_heads=2000), SHAPE), (dict(n_pages=-1), SHAPE),
    (dict(n_pages=2 ** 31), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=24), SHAPE),
    (dict(page_size=1 << 17), SHAPE), (dict(page_stride=2 * 32 * 128 - 16), SHAPE),
    (dict(page_stride=2 * 32 * 128 + 8), SHAPE), (dict(page_stride=1 << 40), SHAPE), (dict(scale_stride=3), SHAPE),
]
BATCH_FAULTS = [
    (dict(n_seqs=-1), SHAPE), (dict(max_pages=-1), SHAPE), (dict(table_stride=3), SHAPE), (dict(max_q_len=-1), SHAPE),
    (dict(max_pages=1 << 27, table_stride=1 << 27), SHAPE), (dict(n_seqs=(1 << 24) + 1), SHAPE),
]
POINTER_FAULTS = [
    (dict(k_pages=None), {}, NULL), (dict(v_pages=None), {}, NULL), (dict(k_scales=None), {}, NULL),
    (dict(v_scales=None), {}, NULL), (dict(k_pages=MIS), {}, ALIGN), (dict(v_pages=ODD), {}, ALIGN),
    (dict(k_scales=ODD), {}, ALIGN), ({}, dict(block_table=None), NULL), ({}, dict(seq_lens=None), NULL),
    ({}, dict(q_indptr=None), NULL), ({}, dict(seq_lens=ODD), ALIGN), ({}, dict(block_table=ODD), ALIGN),
]


@pytest.mark.parametrize("call", [append, dequant, attend])
def test_cache_and_batch_checks(L, call):
    assert call(L, None, batch()) == NULL
    assert call(L, cache(), None) == NULL
    for kw, want in CACHE_FAULTS:
        assert call(L, cache(**kw), batch()) == want, kw
    for kw, want in BATCH_FAULTS:
        assert call(L, cache(), batch(**kw)) == want, kw
    for ckw, bkw, want in POINTER_FAULTS:
        assert call(L, cache(**ckw), batch(**bkw)) == want, (ckw, bkw)
    assert call(L, cache(), batch(), n=-1) == SHAPE
    assert call(L, cache(), batch(), dtype=2) == UNSUP
    # no rows or no sequences: nothing to do, whatever the pointers
    assert call(L, cache(k_pages=None), batch(block_table=None), n=0) == OK
    assert call(L, cache(k_pages=None), batch(n_seqs=0)) == OK


def test_append_checks(L):
    c, b = cache(), batch()
    assert append(L, c, b, k=None) == NULL
    assert append(L, c, b, v=None) == NULL
    assert append(L, c, b, q=None) == NULL                 # q_out without q
    assert append(L, c, b, o=None) == NULL                 # q without q_out
    assert append(L, c, b, ks=248) == SHAPE                # rows overlap
    assert append(L, c, b, ks=260) == SHAPE                # stride not a multiple of 8
    assert append(L, c, b, k=MIS) == ALIGN
    assert append(L, c, b, v=MIS) == ALIGN
    assert append(L, c, b, q=MIS) == ALIGN
    assert append(L, c, b, os_=504) == SHAPE
    assert append(L, c, b, hq=0) == SHAPE
    for kw, want in [(dict(rot_dim=24), SHAPE), (dict(rot_dim=0), SHAPE), (dict(rot_dim=144, row_stride=144), SHAPE),
                     (dict(row_stride=64), SHAPE), (dict(n_positions=-1), SHAPE), (dict(interleaved=2), UNSUP),
                     (dict(table=None), NULL), (dict(table=ODD), ALIGN)]:
        assert append(L, c, b, r=rope(**kw)) == want, kw


def test_dequant_checks(L):
    assert dequant(L, cache(), batch(), k=None) == NULL
    assert dequant(L, cache(), batch(), v=MIS) == ALIGN


def test_attention_checks(L):
    c, b = cache(), batch()
    assert attend(L, c, b, q=None) == NULL
    assert attend(L, c, b, o=None) == NULL
    assert attend(L, c, b, q=MIS) == ALIGN
    assert attend(L, c, b, qs=504) == SHAPE
    assert attend(L, c, b, hq=3) == SHAPE                  # not a multiple of the key / value heads
    assert attend(L, c, b, hq=0) == SHAPE
    assert attend(L, c, b, window=-1) == SHAPE
    assert attend(L, c, b, sinks=-1) == SHAPE
    assert attend(L, c, b, scale=float("nan")) == SHAPE
    assert attend(L, c, b, scale=float("inf")) == SHAPE
    n = ctypes.c_size_t(7)
    assert L.awq_kv_attention_workspace_bytes(ref(c), ref(b), 3, 4, None) == NULL
    assert L.awq_kv_attention_workspace_bytes(ref(c), ref(b), 3, 5, ctypes.byref(n)) == SHAPE
    assert L.awq_kv_attention_workspace_bytes(ref(cache(head_dim=80)), ref(b), 3, 4, ctypes.byref(n)) == UNSUP
    assert L.awq_kv_attention_workspace_bytes(ref(c), ref(b), 0, 4, ctypes.byref(n)) == OK and n.value == 0


def test_logit_scales_that_overflow_in_log2_units(L):
    """A finite scale whose multiple by log2(e) and e4m3's 2^8 is not: refused, where the kernels would give NaN."""
    for scale in (3e38, -3e38, 2.0 ** 119, -2.0 ** 119):
        assert attend(L, cache(), batch(), scale=scale) == SHAPE, scale


def tensors(n=4, h=2, page=32, d=64):
    p = [torch.zeros(n, h, page, d, dtype=torch.uint8) for _ in range(2)]
    s = [torch.zeros(n, h, page // 16) for _ in range(2)]
    return p + s


def test_binding_checks():
    k, v, ks, vs = tensors()
    awq.KvCache(k, v, ks, vs)
    with pytest.raises(ValueError):
        awq.KvCache(k, v, ks, vs, "int4")
    with pytest.raises(TypeError):
        awq.KvCache(k.float(), v, ks, vs)
    with pytest.raises(TypeError):
        awq.KvCache(k, v, ks.half(), vs)
    with pytest.raises(TypeError):
        awq.KvCache(k, v, None, vs)
    with pytest.raises(ValueError):
        awq.KvCache(k[0], v, ks, vs)
    with pytest.raises(ValueError):
        awq.KvCache(k, v[:2], ks, vs)
    with pytest.raises(ValueError):
        awq.KvCache(k, v, ks[..., :1], vs[..., :1])
    with pytest.raises(ValueError):
        awq.KvCache(k.transpose(1, 2), v.transpose(1, 2), ks, vs)       # not dense within a page
    with pytest.raises(ValueError):
        awq.KvCache(k, torch.zeros(8, 2, 32, 64, dtype=torch.uint8)[::2], ks, vs)   # other stride than the keys'
    with pytest.raises(ValueError):
        awq.KvCache.allocate(3, 2, 20, 64, device="cpu")
    c = awq.KvCache(k, v, ks, vs)
    table, lens, ptr = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), \
        torch.zeros(4, dtype=torch.int32)
    b = awq.KvBatch(table, lens, ptr)
    with pytest.raises(TypeError):
        awq.KvBatch(table.long(), lens, ptr)
    with pytest.raises(TypeError):
        awq.KvBatch(table, [1, 2, 3], ptr)
    with pytest.raises(ValueError):
        awq.KvBatch(table, lens, ptr[:3])
    with pytest.raises(ValueError):
        awq.KvBatch(table[:, 0], lens, ptr)
    with pytest.raises(ValueError):
        awq.KvBatch(table[0].expand(3, 4), lens, ptr)
    with pytest.raises(ValueError):
        awq.KvBatch(table.t(), lens[:4], ptr)
    for bad in (0, -1, 2 ** 31):
        with pytest.raises(ValueError):
            awq.KvBatch(table, lens, ptr, bad)
    rows = torch.zeros(3, 2, 64, dtype=torch.float16)
    for call in (lambda: awq.awq_kv_append(rows, rows, c, b), lambda: awq.awq_kv_attention(rows, c, b)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        awq.awq_kv_attention(rows.float(), c, b)
    with pytest.raises(TypeError):
        awq.awq_kv_dequant(c, b, 3, torch.float32)


def test_block_tables_of_one_page_may_have_any_column_stride():
    """The stride of a dimension of one element means nothing."""
    lens, ptr = torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    table = torch.arange(3, dtype=torch.int32)[None].t()
    assert table.shape == (3, 1) and table.stride() == (1, 3)
    b = awq.KvBatch(table, lens, ptr)
    assert (b._args.table_stride, b._args.max_pages) == (1, 1)
    with pytest.raises(ValueError):
        awq.KvBatch(torch.zeros(3, 4, dtype=torch.int32).t()[:, :2], torch.zeros(4, dtype=torch.int32),
                    torch.zeros(5, dtype=torch.int32))


def test_oracle_encodes_the_nearest_code():
    """The oracle against the definition: no code is nearer, ties go to even."""
    rng = np.random.default_rng(1)
    t = np.concatenate([rng.standard_normal(3000) * 100, K._MID, -K._MID, [0.0, 1e9, -1e9, 2.0 ** -11]])
    for fmt, every in (("int8", np.arange(1, 256).astype(np.uint8)),
                       ("e4m3", np.array([b for b in range(256) if b & 127 != 127], np.uint8))):
        c = K.encode(t, fmt)
        values, got = K.decode(every, fmt), K.decode(c, fmt)
        x = np.clip(t, -K.TOP[fmt], K.TOP[fmt])
        near = np.abs(values[None] - x[:, None]).min(1)
        assert (np.abs(got - x) == near).all()
        tie = (np.isclose(np.abs(values[None] - x[:, None]), near[:, None], rtol=0, atol=0)).sum(1) == 2
        tie &= near > 0
        assert ((c[tie] - (128 if fmt == "int8" else 0)) % 2 == 0).all()


def test_oracle_attention_by_hand():
    """Two keys of equal logits, then a window of one and a sink."""
    k = np.ones((3, 1, 1))
    v = np.array([1.0, 3.0, 8.0])[:, None, None]
    q = np.zeros((2, 1, 1))
    out, *_ = K.attention(q, k, v, 1, 1.0, top=np.ones((3, 1)))
    assert np.allclose(out[:, 0, 0], [2.0, 4.0])
    out, *_ = K.attention(q, k, v, 1, 1.0, 1, 0, top=np.ones((3, 1)))
    assert np.allclose(out[:, 0, 0], [3.0, 8.0])
    out, *_ = K.attention(q, k, v, 1, 1.0, 1, 1, top=np.ones((3, 1)))
    assert np.allclose(out[:, 0, 0], [2.0, 4.5])
