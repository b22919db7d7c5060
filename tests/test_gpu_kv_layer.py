"""The attention half of a decoder layer through the library, as it is used:
fused q, k, v product (awq_linear over awq_concat_rows), awq_kv_append,
awq_kv_attention, output product; a prompt, then single tokens. Every stage
is compared with the oracle on the inputs that the stage before it gave."""

import numpy as np
import pytest
import torch

import weight_only_int4_gemv_b200 as awq
from kv_util import Setup, check, i32, to64
from oracle import awq_oracle as O
from oracle import kv_oracle as K
from parity_util import assert_close, dev, oracle_layer
from test_gpu_kv_cache import rope_table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,zp,window,sinks", [("int8", True, 0, 0), ("e4m3", False, 24, 4)])
def test_prompt_then_tokens(fmt, zp, window, sinks):
    hq, hk, dim, width = 8, 2, 64, 512
    shapes = [(hq * dim, width, 1), (hk * dim, width, 2), (hk * dim, width, 3), (width, hq * dim, 4)]
    layers = [oracle_layer(n, k, 0.05, 0.0, zp, seed) for n, k, seed in shapes]
    packed = [tuple(dev(a) if a is not None else None for a in (q, s, z)) for _, q, s, z, _ in layers]
    qkv = awq.awq_concat_rows(packed[:3])
    w_qkv = np.concatenate([layers[i][4] for i in range(3)])
    rope = rope_table(64, dim)
    s = Setup([64, 64], hk, dim, 16, fmt, seed=31, filled=False)
    rng = np.random.default_rng(32)
    lens = [0, 0]
    for new in ([20, 13], [1, 1], [1, 1], [3, 1], [1, 1]):
        past = list(lens)
        lens = [a + n for a, n in zip(lens, new)]
        rows = sum(new)
        x = rng.standard_normal((rows, width)).astype(np.float16)
        y = awq.awq_linear(dev(x), *qkv, workspace=awq.alloc_workspace(rows, w_qkv.shape[0], width, zp))
        assert_close(y.cpu().numpy(), O.matmul_f64(x, w_qkv), "qkv")
        batch = s.batch(lens, new, max(new))
        q, k, v = y.view(rows, hq + 2 * hk, dim).split((hq, hk, hk), 1)
        turned = awq.awq_kv_append(k, v, s.cache, batch, q=q, rope=dev(rope))
        out = awq.awq_kv_attention(turned, s.cache, batch, window=window, sinks=sinks)
        # the oracle's cache takes what the device's holds (its own test compares the two), and attends
        at = 0
        for b in range(2):
            pos = np.arange(past[b], lens[b])
            kk = K.rotate(to64(k[at:at + new[b]]), rope[pos, :dim // 2], rope[pos, dim // 2:], False)
            s.ref.append(0, s.table[b], past[b], kk)
            s.ref.append(1, s.table[b], past[b], to64(v[at:at + new[b]]))
            at += new[b]
        np.testing.assert_array_equal(s.cache.v_scales.cpu().numpy(), s.ref.scales[1])
        np.testing.assert_allclose(s.cache.k_scales.cpu().numpy(), s.ref.scales[0], rtol=2.0 ** -21)
        s.ref.codes = [s.cache.k_pages.cpu().numpy(), s.cache.v_pages.cpu().numpy()]
        s.ref.scales = [s.cache.k_scales.cpu().numpy(), s.cache.v_scales.cpu().numpy()]
        want, tol = s.expect(to64(turned), lens, new, None, window, sinks)
        check(out, want, tol, "attention")
        flat = out.view(rows, hq * dim)
        o = awq.awq_linear(flat, *packed[3], workspace=awq.alloc_workspace(rows, width, hq * dim, zp))
        assert_close(o.cpu().numpy(), O.matmul_f64(flat.cpu().numpy(), layers[3][4]), "output product")
    assert awq.awq_device_error() == 0
