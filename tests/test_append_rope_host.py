"""Appends with a rotation, step_rope and the FP8_BLOCK format: what the host refuses
or counts, without a GPU."""
import ctypes
import os
import types

import numpy as np
import pytest
import torch

from decode_attention_pruned_gb300 import binding as lkb
from decode_attention_pruned_gb300 import synth as S
from oracle import quant as OQ
from test_chunk_calls_host import CUDA, AllOk, Allocations, NoCalls, OnGpu, Stream

CSRC = os.path.join(os.path.dirname(lkb.__file__), "csrc")


def test_null_arguments(lib):
    rope, c = lkb.Rope(), lkb.Chunk()
    c.n_max = 1
    p = ctypes.byref(c)
    assert lib.lk_append_rope(None, 0, rope._h, p, None, None, 0, None) == lkb.LK_ERR_ARG
    assert lib.lk_append_rope(None, 0, None, p, None, None, 0, None) == lkb.LK_ERR_ARG
    assert lib.lk_step_rope(None, 0, rope._h, p, None, None, None, 0, None) == lkb.LK_ERR_ARG


def test_format_bytes(lib):
    w = S.WORKLOADS[1]
    plan = lkb.Plan.for_workload(w, S.masks_with_counts(w, [32, 64, 96, 128] * 2), S.make_policies(w))
    B, cap = 2, 32768
    mid = cap - w.sink - w.local
    bf16, block = plan.cache_bytes(B, cap), plan.cache_bytes(B, cap, kv_format=lkb.KV_FP8_BLOCK)
    # sealed blocks of 128 (k + 128) codes and 16 bytes, and a 128-row bf16 tail
    expect = bf16 + sum(2 * B * (-mid * 2 * (k + 128) + mid // 128 * (128 * (k + 128) + 16) + 128 * 2 * (k + 128))
                        for k in (32, 64, 96, 128))
    assert abs(block - expect) < 1 << 16
    paged = plan.cache_bytes(B, cap, middle_tokens=B * mid, kv_format=lkb.KV_FP8_BLOCK)
    assert abs(paged - block) < 1 << 20
    assert block < plan.cache_bytes(B, cap, kv_format=lkb.KV_FP8)
    with pytest.raises(lkb.LeankError) as e:
        plan.cache_bytes(B, cap, kv_format=4)
    assert e.value.status == lkb.LK_ERR_ARG


def test_oracle_block_scales():
    """One scale for K's kept channels and one for V; its lower bound; codes as FP8's."""
    rng = np.random.default_rng(1)
    K, V = rng.standard_normal((400, 128)).astype(np.float32), rng.standard_normal((400, 128)).astype(np.float32)
    kept = np.arange(5, 69, 2)
    K[10 + 4, 6] = 1000.0                                    # a channel that is not kept
    (kc, ks, vc, vs), = OQ.middle_blocks(K, V, kept, 4 + 200, 4, 72, "fp8_block")
    k = K[4:132][:, kept]
    assert ks.shape == (32,) and np.all(ks == np.float32(np.abs(k).max()) / np.float32(448))
    assert vs.shape == (128,) and np.all(vs == np.float32(np.abs(V[4:132]).max()) / np.float32(448))
    assert np.abs(OQ.code_value(kc, "fp8") * ks.astype(np.float64) - k).max() <= 2.0 ** -4 * np.abs(k).max()
    (kc, ks, vc, vs), = OQ.middle_blocks(K * 0, V * np.float32(1e-30), kept, 204, 4, 72, "fp8_block")
    assert np.all(ks == np.float32(2.0 ** -64)) and np.all(vs == np.float32(2.0 ** -64))
    assert not (kc & 0x7f).any() and not (vc & 0x7f).any()      # (a zero keeps its sign)


def test_block_byte_order():
    """The order of the codes, as the header says it: a bijection, and a lane's word is
    16 bytes in a row."""
    def kbyte(k, r, c):
        return (r >> 4) * 16 * k + (c >> 5) * 512 + ((r & 7) * 4 + ((c >> 3) & 3)) * 16 + ((r >> 3) & 1) * 8 + (c & 7)

    def vbyte(r, c):
        return (r >> 4) * 2048 + ((c & 7) >> 1) * 512 + (((c >> 3) & 7) * 4 + ((r & 7) >> 1)) * 16 + (c & 1) * 8 + \
            (c >> 6) * 4 + ((r >> 3) & 1) * 2 + (r & 1)

    for k in (32, 64, 96, 128):
        assert sorted(kbyte(k, r, c) for r in range(128) for c in range(k)) == list(range(128 * k))
        for s, u, g, t in ((0, 0, 0, 0), (3, k // 32 - 1, 5, 2), (7, 0, 7, 3)):
            at = 16 * k * s + 512 * u + 16 * (4 * g + t)
            assert [kbyte(k, 16 * s + g + 8 * i, 32 * u + 8 * t + j) for i in (0, 1) for j in range(8)] == \
                list(range(at, at + 16))
    assert sorted(vbyte(r, c) for r in range(128) for c in range(128)) == list(range(128 * 128))
    for s, u, g, t in ((0, 0, 0, 0), (6, 3, 4, 1), (7, 1, 7, 3)):
        at = 2048 * s + 512 * u + 16 * (4 * g + t)
        rows = [16 * s + 2 * t + i for i in (0, 1, 8, 9)]
        assert [vbyte(r, 8 * g + 2 * u + i + h) for i in (0, 1) for h in (0, 64) for r in rows] == list(range(at, at + 16))
    text = open(os.path.join(CSRC, "lk_block.h")).read()
    assert "(r >> 4) * 16 * k + (c >> 5) * 512" in text and "(r >> 4) * 2048 + ((c & 7) >> 1) * 512" in text


# ------------------------------------------------------------ the Python side
def _rows(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _cache(B, Hq, H):
    c = object.__new__(lkb.Cache)
    c._h, c.batch, c.buffer = None, B, OnGpu(torch.zeros(1))
    c.plan = types.SimpleNamespace(num_q_heads=Hq, num_kv_heads=H, _h=None)
    return c


def _rope(axes=()):
    r = object.__new__(lkb.Rope)
    r._h, r.axes = None, axes
    return r


def _ints(*shape):
    return OnGpu(torch.zeros(shape, dtype=torch.int32))


def test_binding_refusals(monkeypatch):
    monkeypatch.setattr(lkb, "_lib", NoCalls())
    monkeypatch.setattr(lkb, "_stream", lambda stream=None: None)
    c, r, r3 = _cache(2, 4, 2), _rope(), _rope((3,))
    q, k = OnGpu(_rows(2, 5, 4, 128)), OnGpu(_rows(2, 5, 2, 128))
    q1, k1 = OnGpu(_rows(2, 4, 128)), OnGpu(_rows(2, 2, 128))
    far = OnGpu(_rows(2, 5, 2, 128))
    far.device = torch.device("cuda", 1)
    bad = [
        lambda: c.append_rope(0, r, k, OnGpu(_rows(2, 4, 2, 128))),
        lambda: c.append_rope(0, r, k, k, q=OnGpu(_rows(2, 5, 5, 128))),
        lambda: c.append_rope(0, r, k, k, q=q1),
        lambda: c.append_rope(0, r, OnGpu(_rows(3, 5, 2, 128)), OnGpu(_rows(3, 5, 2, 128))),
        lambda: c.append_rope(0, r, OnGpu(torch.zeros(2, 5, 2, 128)), k),                      # fp32
        lambda: c.append_rope(0, r, OnGpu(_rows(2, 5, 2, 64)), k),
        lambda: c.append_rope(0, r, OnGpu(_rows(2, 1, 2, 128).expand(2, 5, 2, 128)), k),        # tokens share rows
        lambda: c.append_rope(0, r, k, k, q_out=q),
        lambda: c.append_rope(0, r, k, k, q=q, q_out=OnGpu(_rows(2, 4, 4, 128))),
        lambda: c.append_rope(0, r, k, k, positions=_ints(2, 4)),
        lambda: c.append_rope(0, r, k, k, positions=_ints(3, 2, 5)),
        lambda: c.append_rope(0, r3, k, k, positions=_ints(2, 5)),
        lambda: c.append_rope(0, r3, k1, k1, positions=_ints(2)),
        lambda: c.append_rope(0, r, k, k, positions=OnGpu(torch.zeros(2, 5, dtype=torch.int64))),
        lambda: c.append_rope(0, r, k, k, ids=_ints(5, 2)),
        lambda: c.append_rope(0, r, k, k, lens=[1, 2, 3]),
        lambda: c.append_rope(0, r, far, k),
        lambda: c.append_rope(0, r, OnGpu(_rows(2, 128)), k),
        lambda: c.step_rope(0, r, q, k, k),
        lambda: c.step_rope(0, r, q1, k1, k1, positions=_ints(2, 1)),
        lambda: c.step_rope(0, r, q1, k1, k1, o=OnGpu(torch.zeros(2, 4, 64))),
    ]
    for call in bad:
        with pytest.raises((ValueError, TypeError)):
            call()


@pytest.mark.parametrize("given", [False, True], ids=["current", "given"])
def test_new_tensors_belong_to_the_stream_of_the_call(monkeypatch, given):
    made = Allocations(monkeypatch)
    monkeypatch.setattr(lkb, "_lib", AllOk())
    monkeypatch.setattr(lkb, "_stream", lambda stream=None: None)
    monkeypatch.setattr(OnGpu, "numel", lambda self: 1, raising=False)
    s = Stream() if given else None
    c = _cache(2, 4, 2)
    c.workspace, c.device = OnGpu(torch.zeros(1)), CUDA
    q1, k1 = OnGpu(_rows(2, 4, 128)), OnGpu(_rows(2, 2, 128))
    for n, call in ((1, lambda: c.append_rope(0, _rope(), k1, k1, q=q1, stream=s)),
                    (0, lambda: c.append_rope(0, _rope(), k1, k1, stream=s)),
                    (1, lambda: c.step_rope(0, _rope(), q1, k1, k1, stream=s))):
        made.made.clear()
        call()
        assert made.made == [s] * n
