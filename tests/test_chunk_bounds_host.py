"""What the bounds on chunk attention over quantised middles can tell apart, on the
CPU: outputs computed as the kernel rounds them pass, outputs of a kernel that reads
a scale, a row or a block wrongly do not."""
import math

import numpy as np
import pytest

from decode_attention_pruned_gb300 import synth as S
from helpers import f64
from oracle import chunk as OC
from oracle import quant as OQ
from test_gpu_chunk_quantised import RMS, _bound, _rms

W = S.WORKLOADS[1].scaled(num_kv_heads=1, num_q_heads=4, batch=1, sink=16, local=64)
N, n = 850, 45                                        # 6 sealed blocks and a tail


def _bf16(x):
    """fp64 values to the nearest bf16, ties to even."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7fff + (u >> 16 & 1)) & 0xffff0000).astype(np.uint32).view(np.float32).astype(np.float64)


def _attend(q, K, V, kept, as_kernel):
    """Every query over its keys; as_kernel: weights and outputs rounded to bf16."""
    out = np.zeros(q.shape)
    beta = np.zeros(128)
    beta[kept] = 1
    for i in range(len(q)):
        t, p = np.arange(N + i + 1), N + i
        near = (t < W.sink) | (p - t < W.local)
        s = np.where(near, q[i] @ K[:p + 1].T, (q[i] * beta) @ K[:p + 1].T) / math.sqrt(128)
        w = np.exp(s - s.max(1, keepdims=True))
        o = (_bf16(w) if as_kernel else w) @ V[:p + 1] / w.sum(1, keepdims=True)
        out[i] = _bf16(o) if as_kernel else o
    return out


def _case(fmt, k, seed=0):
    r = np.random.default_rng(seed)
    key, v = (f64(x)[0, :N + n, 0] for x in S.make_kv(W, 0, N + n))
    q = _bf16(r.standard_normal((n, 4, 128)))
    kept = np.sort(r.choice(128, k, replace=False))
    blocks = OQ.middle_blocks(key, v, kept, N, W.sink, W.local, fmt)
    assert len(blocks) == 6
    K, V = key.copy(), v.copy()
    K[:N], V[:N] = OC.sealed_history(key[:N], v[:N], kept, 0, N, W.sink, W.local, fmt)
    return q, K, V, kept, blocks


def _ok(got, q, K, V, kept):
    o = _attend(q, K, V, kept, False)
    within = (np.abs(got - o) <= _bound(o, _attend(q, K, np.abs(V), kept, False))).all()
    return bool(within) and _rms(got, o) <= RMS


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("k", [32, 64, 96, 128])
def test_bounds_pass_the_right_outputs_and_no_wrong_ones(fmt, k):
    q, K, V, kept, blocks = _case(fmt, k)
    want = _attend(q, K, V, kept, False)
    assert np.abs(want - OC.chunk_head(q, K, V, 0, kept, N, W.sink, W.local, 0)).max() < 1e-12
    assert _ok(_attend(q, K, V, kept, True), q, K, V, kept)
    at = lambda j: slice(W.sink + 128 * j, W.sink + 128 * (j + 1))  # noqa: E731
    for j, (kc, ks, vc, vs) in enumerate(blocks):
        # one block's value scales a row late, and another's keys by the next channel's scale
        wrong = V.copy()
        wrong[at(j)] = OQ.dequantize_per_token(vc, np.roll(vs, 1), fmt)
        assert not _ok(_attend(q, K, wrong, kept, True), q, K, V, kept), ("value scales", j)
        wrong = K.copy()
        wrong[at(j), kept] = 0
        wrong[np.ix_(np.arange(at(j).start, at(j).stop), kept)] = OC.sealed_keys(kc, np.roll(ks, 1), fmt)
        assert not _ok(_attend(q, wrong, V, kept, True), q, K, V, kept), ("key scales", j)
        # a block left out, and two of its rows
        for rows in (at(j), slice(at(j).start + 40, at(j).start + 42)):
            wrong = V.copy()
            wrong[rows] = 0
            assert not _ok(_attend(q, K, wrong, kept, True), q, K, V, kept), ("rows", j, rows)
    # keys and values before their quantisation
    key, v = (f64(x)[0, :N + n, 0] for x in S.make_kv(W, 0, N + n))
    assert not _ok(_attend(q, key, v, kept, True), q, K, V, kept)


def test_sealed_keys_are_close_to_the_dequantised_ones():
    r = np.random.default_rng(3)
    for fmt in ("int8", "fp8"):
        x = r.standard_normal((128, 64)) * 2.0 ** r.integers(-12, 12, 64)
        codes, scales = OQ.quantize_per_channel(x, fmt)
        exact = OQ.dequantize_per_channel(codes, scales, fmt)
        got = OC.sealed_keys(codes, scales, fmt)
        # two roundings to 11 bits; f16's smallest step below them
        step = 2.0 ** -25 * 2.0 ** (math.floor(math.log2(float(scales.max()))) - 6)
        tol = 2.01 * 2.0 ** -11 * np.abs(exact) + (1 + np.abs(OQ.code_value(codes, fmt))) * step
        assert (np.abs(got - exact) <= tol).all()
        codes, scales = OQ.quantize_per_channel(np.zeros((128, 32)), fmt)
        assert not OC.sealed_keys(codes, scales, fmt).any()
