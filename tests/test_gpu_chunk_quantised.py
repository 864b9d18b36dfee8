"""Chunk attention over INT8 / FP8 middles, as exactly as its roundings allow.

The oracle takes sealed keys as the kernel does (scales and products to f16, as
oracle.chunk.sealed_keys says) and everything else in fp64.  What remains of an
output o = sum p v, with A = sum p |v|:

  each value:  2^-8 |o| (its rounding to bf16) + 2^-8 A (p rounded to bf16; over
      sealed blocks p times the value's scale to f16, 2^-11) + 2^-12 A (fp32 scores
      of up to 128 products, exponentials)
      and, for weights so small that f16 holds them in steps of 2^-24: a row's
      weights are p = 2^(s - m) with m <= max s + log2(c) - 6, c the largest scale of
      a value, so l = sum p >= 2^6 / c; half a step, 2^-25, times a code of at most
      max |v| / c, is 2^-31 max |v| of l for each of the N tokens held

  all values of a head together, root mean square relative to the outputs': a
      rounding to bf16 is off by a uniform share of half a step, on average over
      mantissas 2^-8 / sqrt(3) * sqrt(3 / (8 ln 2)) = 1.66e-3; once for o, once for
      the weights, whose errors are independent and meet independent values:
      sqrt(2) * 1.66e-3 = 2.35e-3, and a fifth more for heads of a few thousand
      outputs.

Against keys in fp64 instead, f16's 2^-11 of scale and product each add at most
sqrt(2) * 2^-11 / sqrt(3) * 0.735 = 0.3e-3 times the size of a score, sqrt(sum q^2
k^2 / 128): 0.06e-3 more for scores of about one."""
import math

import numpy as np
import pytest
import torch

from decode_attention_pruned_gb300 import binding as lkb
from decode_attention_pruned_gb300 import synth as S
from helpers import Case, f64
from oracle import chunk as OC
from oracle import quant as OQ
from test_gpu_chunk import _chunk, _fill, _queries

pytestmark = pytest.mark.gpu

TINY = S.WORKLOADS[0]
LLAMA = S.WORKLOADS[1]
FASTGEN = S.WORKLOADS[4]
FORMATS = [lkb.KV_INT8, lkb.KV_FP8]
FORMAT_IDS = ["int8", "fp8"]
RMS = 1.2 * 2.35e-3


def _bound(o, A):
    return 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -12) * A


def _expected(case, q, held, lens, history=OC.sealed_history):
    """{(b, h): (o, bound)} fp64 [lens[b], G, 128]."""
    k, v = case.history(0)
    w, G, out = case.w, case.w.group, {}
    for b in range(w.batch):
        N, n = int(held[b]), int(lens[b])
        if n == 0:
            continue
        for h in range(w.num_kv_heads):
            pol = int(case.policies[0, h])
            kept = np.nonzero(case.masks[0, h])[0] if pol == S.POLICY_FULL else np.arange(0)
            K, V = f64(k[b, :N + n, h]), f64(v[b, :N + n, h])
            if case.kv_format != lkb.KV_BF16:
                K[:N], V[:N] = history(K[:N], V[:N], kept, pol, N, w.sink, w.local,
                                       fmt=lkb.KV_FORMAT_NAMES[case.kv_format])
            args = (pol, kept, N, w.sink, w.local, w.local_only_window, case.flags[b][:N + n])
            Q = f64(q[b, :n, h * G:(h + 1) * G])
            o, A = OC.chunk_head(Q, K, V, *args), OC.chunk_head(Q, K, np.abs(V), *args)
            sealed = case.kv_format != lkb.KV_BF16 and len(kept) > 0
            tiny = 2.0 ** -31 * N * np.abs(V[:N]).max(initial=0.0) if sealed else 0.0
            out[b, h] = o, _bound(o, A) + tiny
    return out


def _rms(got, o):
    return math.sqrt(((got - o) ** 2).sum() / max((o ** 2).sum(), 1e-300))


def _attend(case, held, n, lens=None, q=None, **kw):
    q = _queries(case, n) if q is None else q
    k, v, ids = _chunk(case, 0, held, n)
    full = [n] * case.w.batch if lens is None else lens
    got = f64(case.cache.chunk_attn(0, q, k, v, lens=lens, ids=ids))
    case.cache.check()
    G = case.w.group
    for (b, h), (o, tol) in _expected(case, q, held, full, **kw).items():
        x = got[b, :full[b], h * G:(h + 1) * G]
        bad = np.abs(x - o) > tol + 1e-30
        assert not bad.any(), (b, h, int(bad.sum()), np.argwhere(bad)[:4].tolist())
        if o.size >= 1024:
            assert _rms(x, o) <= RMS, (b, h, _rms(x, o))


@pytest.mark.parametrize("fmt", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("k", [32, 64, 96, 128])
@pytest.mark.parametrize("n", [3, 60])
def test_outputs_are_as_exact_as_their_roundings(cuda, fmt, k, n):
    """Against the dequantised values themselves: keys are not what limits o."""
    w = TINY.scaled(num_kv_heads=2, num_q_heads=8, batch=2, sink=4, local=64)
    case = Case(w, total=1600, masks=S.masks_with_counts(w, (k, k)), kv_format=fmt)
    held = [1500, 1111]
    _fill(case, held)
    q = _queries(case, n)
    key, v, _ = _chunk(case, 0, held, n)
    got = f64(case.cache.chunk_attn(0, q, key, v))
    for (b, h), (o, _) in _expected(case, q, held, [n, n], history=OQ.quantized_history).items():
        assert _rms(got[b, :, h * 4:h * 4 + 4], o) <= RMS, (b, h)


@pytest.mark.parametrize("fmt", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("n", [4, 50])
def test_keys_and_queries_of_any_size(cuda, fmt, n):
    """Keys far outside f16's range, met by queries that bring the scores back; rows
    of q of very different sizes side by side; blocks of very different sizes one
    after the other; a block of zeros."""
    w = TINY.scaled(num_kv_heads=4, num_q_heads=16, batch=3, sink=4, local=64)
    case = Case(w, total=900, masks=S.masks_with_counts(w, (32, 64, 96, 128)), kv_format=fmt)
    held = [800, 517, 68 + 256]
    k, v = case.history(0)
    by = torch.tensor([2.0 ** 60, 2.0 ** -60, 2.0 ** 17], device="cuda")
    k *= by[:, None, None, None].to(torch.bfloat16)
    k[:, 196:324] *= 2.0 ** -9
    k[:, 324:400, :, ::2] *= 2.0 ** 6
    k[1, 68:196] = 0
    _fill(case, held)
    q = _queries(case, n)
    q *= (1 / by)[:, None, None, None].to(torch.bfloat16)
    q[:, 1] *= 2.0 ** -30                          # scores of about nothing
    q[:, 2, ::3] *= 2.0 ** 3
    q[:, 3, 5] = 0
    _attend(case, held, n, q=q)


@pytest.mark.parametrize("fmt", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("held", [[67, 68], [69, 195], [196, 197], [323, 324], [325, 451], [452, 60]], ids=str)
@pytest.mark.parametrize("n", [1, 2, 40, 130])
def test_open_blocks_of_every_size(cuda, fmt, held, n):
    """Middles that end on, before and behind a block's border, where rows that no
    block has sealed, rows that leave the window and the chunk's own follow one
    another in the same tiles."""
    w = TINY.scaled(num_kv_heads=4, num_q_heads=8, batch=2, sink=4, local=64)
    case = Case(w, total=600, masks=S.masks_with_counts(w, (32, 128, 96, 0)), kv_format=fmt)
    _fill(case, held)
    _attend(case, held, n)


@pytest.mark.parametrize("fmt", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "paged"])
def test_middles_of_every_width(cuda, fmt, paged):
    w = LLAMA.scaled(num_kv_heads=5, num_q_heads=20, batch=2, sink=16, local=64)
    case = Case(w, total=900, masks=S.masks_with_counts(w, (0, 32, 64, 96, 128)), kv_format=fmt,
                middle_tokens=1800 if paged else None)
    held = [850, 208]                 # 6 blocks and a tail; exactly one block
    _fill(case, held)
    _attend(case, held, 45)
    _attend(case, held, 3, lens=[3, 1])


@pytest.mark.parametrize("fmt", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("n", [3, 60])
def test_policies(cuda, fmt, n):
    w = FASTGEN.scaled(num_layers=1, batch=2, context=700, policy_counts=(2, 2, 4))
    case = Case(w, total=800, kv_format=fmt)
    held = [700, 301]
    _fill(case, held)
    _attend(case, held, n, lens=[n, n - 2])


@pytest.mark.parametrize("fmt", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("n", [1, 16, 17, 100])
def test_wide_tiles_then_sealed_ones(cuda, fmt, n):
    w = TINY.scaled(num_kv_heads=6, num_q_heads=48, batch=3, sink=130, local=400)
    case = Case(w, total=2200, masks=S.masks_with_counts(w, (96, 96, 128, 32, 0, 96)), kv_format=fmt)
    held = [2100, 700, 1313]
    _fill(case, held)
    _attend(case, held, n)


@pytest.mark.parametrize("fmt", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("n", [1, 3, 40])
def test_one_item_over_every_block(cuda, fmt, n):
    w = TINY.scaled(num_kv_heads=1, num_q_heads=8, batch=1, sink=4, local=64)
    case = Case(w, total=60050, masks=S.masks_with_counts(w, (64,)), gen_device="cuda", kv_format=fmt)
    _fill(case, [60000])
    _attend(case, [60000], n)


@pytest.mark.parametrize("fmt", FORMATS, ids=FORMAT_IDS)
def test_stale_rows_behind_an_open_block(cuda, fmt):
    """A slot's last request left NaN in the rows behind the next one's."""
    w = TINY.scaled(num_kv_heads=2, num_q_heads=8, batch=2, sink=4, local=40)
    case = Case(w, total=600, masks=S.masks_with_counts(w, (32, 96)), kv_format=fmt)
    bad = torch.full((600, 2, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    for b in range(2):
        case.cache.prefill_sequence(0, b, bad, bad)
        case.cache.release(b)
    held = [233, 75]
    k, v = case.history(0)
    for b in range(2):
        case.cache.prefill_sequence(0, b, k[b, :held[b]].contiguous(), v[b, :held[b]].contiguous())
    _attend(case, held, 7)
    _attend(case, held, 50)


@pytest.mark.parametrize("fmt", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("held, n, counts", [([460, 460], 150, (128, 96)), ([200, 330], 40, (128, 96)),
                                             ([330, 200], 150, (96, 64, 128)), ([460] * 8, 70, (128, 96)),
                                             ([460] * 8, 150, (128, 96))], ids=str)
def test_blocks_with_nothing_to_do(cuda, fmt, held, n, counts):
    """Little work a block: some blocks start where the next one does, at an item's
    first tile, and have nothing to do.  Inside an item no two start at one tile."""
    H = len(counts)
    w = TINY.scaled(num_kv_heads=H, num_q_heads=4 * H, batch=len(held), sink=4, local=64)
    case = Case(w, total=max(held) + n, masks=S.masks_with_counts(w, counts), kv_format=fmt)
    _fill(case, held)
    _attend(case, held, n)
    torch.cuda.synchronize()
    ctas = min(torch.cuda.get_device_properties(0).multi_processor_count, 160)
    starts = case.cache.chunk_workspace[:8 * (ctas + 2)].view(torch.int32).view(-1, 2).tolist()
    blocks = starts[ctas + 1][0]
    starts = [tuple(x) for x in starts[:blocks + 1]]
    assert 1 < blocks <= ctas and starts[0] == (0, 0) and starts == sorted(starts)
    same = [x for x, y in zip(starts, starts[1:]) if x == y]
    assert same and all(tile == 0 for _, tile in same)


@pytest.mark.parametrize("fmt", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("n", [4, 50, 130])
def test_values_of_any_size(cuda, fmt, n):
    """Values whose scales differ by far from block to block and from row to row, a
    block of zeros, values near fp32's ends of what sums hold."""
    w = TINY.scaled(num_kv_heads=4, num_q_heads=16, batch=4, sink=4, local=64)
    case = Case(w, total=1030, masks=S.masks_with_counts(w, (32, 64, 96, 128)), kv_format=fmt)
    held = [900, 517, 68 + 256, 700]
    k, v = case.history(0)
    by = torch.tensor([1.0, 2.0 ** 40, 2.0 ** -40, 2.0 ** 7], device="cuda")
    v *= by[:, None, None, None].to(torch.bfloat16)
    v[:, 68:196] *= 2.0 ** -12
    v[:, 196:324] *= 2.0 ** 9
    v[:, 200:300:7] *= 2.0 ** -18
    v[1, 324:452] = 0
    v[3, 324:452] *= 2.0 ** 30
    _fill(case, held)
    _attend(case, held, n)


@pytest.mark.parametrize("fmt", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("k", [32, 128])
@pytest.mark.parametrize("n", [3, 60])
def test_sealed_values_cost_no_precision(cuda, fmt, k, n):
    """Where nearly every weight is a sealed block's, o is as exact as its own
    rounding: 1.66e-3 in the root mean square, and a fifth of P's 11 bits' 0.2e-3
    and of the near tokens' bf16 weights."""
    w = TINY.scaled(num_kv_heads=2, num_q_heads=8, batch=1, sink=0, local=8)
    case = Case(w, total=6200, masks=S.masks_with_counts(w, (k, k)), kv_format=fmt)
    held = [6100]
    _fill(case, held)
    q = _queries(case, n, scale=0.3)
    key, v, _ = _chunk(case, 0, held, n)
    got = f64(case.cache.chunk_attn(0, q, key, v))
    for (b, h), (o, _) in _expected(case, q, held, [n]).items():
        assert _rms(got[b, :, h * 4:h * 4 + 4], o) <= 1.2 * 1.66e-3, (b, h)
