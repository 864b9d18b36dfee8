"""Weights over sealed blocks with a reference of their own, and sums that meet in
shared memory: decode and chunks over KV_FP8_BLOCK caches (chunks over INT8 and FP8
too) where full-width rows and blocks, or one block and the next, differ by far more
than f16's range, and segments long enough that sums are flushed several times.

Bounds of decode (fp32 out; A = sum p |v|).  Keys are multiples of 1/4 up to 7/4 and
queries of +-1 (their codes times +-1 in blocks), so a score's products and sums are exact
in fp32.  Then in units of 2^-24, y a score in log2 units and j a block's value exponent:
the factor of y is rounded twice, y + j once, m and the difference once each: 3 |y| +
3 |y + j| + 64 <= 3 * 40 + 3 * 80 + 64 < 430 in the cases below, 2.6e-5 ln 2 = 1.8e-5 of a
weight.  Exponentials, three rescalings' among them, are off by 2^-22 each, 1e-6; the sums
by less than 64 roundings, 3.9e-6; P by 2^-22.  Together a weight is off by less than
2^-15.4, and a normalised one by twice that: 2^-14 A.

Chunks (bf16 out): 2^-8 |o| for o, 2^-8 A for P in bf16 or f16, 2^-12 A for the rest; INT8 and
FP8 take keys' scales and products to 11 bits: 2 * 2^-12 of sum |q k| / sqrt(128) <= 64 * 7/4 /
11.3 = 9.9, a weight's 4.9e-3, a normalised one's 9.7e-3 A."""
import numpy as np
import pytest
import torch

from decode_attention_pruned_gb300 import binding as lkb
from decode_attention_pruned_gb300 import synth as S
from helpers import Case, f64
from oracle import attention as OA
from oracle import quant as OQ

pytestmark = pytest.mark.gpu

TINY = S.WORKLOADS[0]
FMT = lkb.KV_FP8_BLOCK
COMMON = 64                                        # channels on which the queries agree
LOG2 = 1.4426950408889634 / 128 ** 0.5             # of a score, per q.k
SINK, LOCAL = 4, 32


def _case(G, N, counts=(32, 128), fmt=FMT, batch=1, local=LOCAL):
    """Keys that are 0 on the common channels and small multiples of 1/4 on the others, the
    kept ones among them; each block has a key of 7/4."""
    H = len(counts)
    w = TINY.scaled(num_q_heads=H * G, num_kv_heads=H, sink=SINK, local=local, batch=batch)
    masks = np.zeros((1, H, 128), np.uint8)
    for h, c in enumerate(counts):
        masks[0, h, 128 - c:] = 1
    case = Case(w, total=N, masks=masks, kv_format=fmt)
    rs = np.random.default_rng(3)
    k = rs.choice([-1.0, -0.5, -0.25, 0.0, 0.25, 0.5, 1.0, 1.75], (1, N, H, 128))
    k[..., :COMMON] = 0
    k[:, SINK::128, :, -1] = 1.75
    v = rs.standard_normal((1, N, H, 128))
    return case, k, v


def _queries(case, shape=()):
    """+-1; on the common channels +1."""
    q = torch.from_numpy(np.random.default_rng(9).choice([-1.0, 1.0], (1, *shape, case.w.num_q_heads, 128)))
    q[..., :COMMON] = 1
    return q.to(torch.bfloat16).cuda()


def _history(case, k, v):
    case.hist[0] = tuple(torch.from_numpy(x).to(torch.bfloat16).cuda() for x in (k, v))
    for x, y in zip(case.hist[0], (k, v)):
        assert bool(x.isfinite().all()), y
    return case.hist[0]


def _expected(case, q, N, held):
    """(o, A) of queries [Hq, 128] that see N tokens, of which blocks were sealed when `held` were there."""
    w, G, o, A = case.w, case.w.group, [], []
    k, v = case.history(0)
    for h in range(w.num_kv_heads):
        kept = np.nonzero(case.masks[0, h])[0]
        K, V = f64(k[0, :N, h]), f64(v[0, :N, h])
        K[:held], V[:held] = OQ.quantized_history(K, V, kept, 0, held, w.sink, w.local,
                                                  lkb.KV_FORMAT_NAMES[case.kv_format])
        args = (0, kept, N, w.sink, w.local, 0, case.flags[0])
        o.append(OA.decode_head(f64(q[h * G:(h + 1) * G]), K, V, *args))
        A.append(OA.decode_head(f64(q[h * G:(h + 1) * G]), K, np.abs(V), *args))
    return np.concatenate(o), np.concatenate(A)


def _check(got, o, A, tol):
    off = np.abs(f64(got) - o)
    assert np.all(off <= tol), (float((off / np.maximum(A, 1e-300)).max()), float((off / np.maximum(tol, 1e-300)).max()))


def _decode(case, N, ctas=0):
    case.prefill(0, N)
    case.cache.set_decode_ctas(ctas)
    q = _queries(case)
    got = case.cache.decode(0, q)
    case.cache.check()
    o, A = _expected(case, q[0], N, N)
    _check(got[0], o, A, 2.0 ** -14 * A)


@pytest.mark.parametrize("ctas", [1, 0])
@pytest.mark.parametrize("gap", [0, 16, 24, 28, 32])
@pytest.mark.parametrize("G", [4, 7])
def test_rows_that_score_far_above_the_blocks(cuda, G, gap, ctas):
    """Sinks that take nearly all of the softmax and have no value: o is what the middle
    and the window give, however small their weights."""
    N = SINK + LOCAL + 128 * 6 + 50
    case, k, v = _case(G, N)
    k[:, :SINK, :, :COMMON] = gap / 8                  # 8.16 log2 units for each
    v[:, :SINK] = 0
    v[:, -LOCAL:] /= 256                               # (so that the middle is most of o)
    _history(case, k, v)
    _decode(case, N, ctas)


@pytest.mark.parametrize("ctas", [0, 50, 5, 1])
@pytest.mark.parametrize("G", [3, 6])
def test_parts_whose_references_fell_far(cuda, G, ctas):
    """Parts of an entry that hold a few rows and a block of zeros, for which m falls by 76, beside
    one with sinks 2^56 above them: what they hold is still there when they meet.  (|y| <=
    66 and |y + j| <= 140: 2.8e-5 instead of the 1.8e-5 above, 2^-13 A in all.)"""
    N = 843
    for counts in ((64, 64, 64), (32, 64, 128), (128, 32, 96)):
        case, k, v = _case(G, N, counts=counts, local=200)
        k[:, :SINK, :, :COMMON] = 7
        v[:, :SINK] = 0
        v[:, SINK:SINK + 128] = 0
        _history(case, k, v)
        case.prefill(0, N)
        case.cache.set_decode_ctas(ctas)
        q = _queries(case)
        got = case.cache.decode(0, q)
        case.cache.check()
        for h in range(3):                             # head by head, so that none hides behind another's size
            o, A = _expected(case, q[0], N, N)
            rows = slice(h * G, (h + 1) * G)
            _check(got[0, rows], o[rows], A[rows], 2.0 ** -13 * A[rows])


@pytest.mark.parametrize("gap", [20, 30])
@pytest.mark.parametrize("G", [4, 7])
def test_a_first_block_of_far_larger_values(cuda, G, gap):
    """The oldest block's values are 2^gap times the others', and its scores as far below
    them, beside rows that score as the others do."""
    N = SINK + LOCAL + 128 * 6 + 50
    case, k, v = _case(G, N, counts=(128, 128))
    k[:, SINK:SINK + 128, :, :COMMON] = -gap / 8
    v[:, SINK:SINK + 128] *= 2.0 ** gap
    _history(case, k, v)
    _decode(case, N)


@pytest.mark.parametrize("G", [4, 7])
def test_a_first_block_of_zeros_and_rows_of_huge_values(cuda, G):
    """What rows before it gave stays inside fp32's range."""
    N = SINK + LOCAL + 128 * 3 + 50
    case, k, v = _case(G, N)
    v[:, SINK:SINK + 128] = 0
    v[:, :SINK] *= 2.0 ** 90
    v[:, -LOCAL:] *= 2.0 ** 90
    _history(case, k, v)
    _decode(case, N)


@pytest.mark.parametrize("values", [0, 30, -30])
@pytest.mark.parametrize("G", [4, 7])
def test_maxima_that_move_after_sums_were_flushed(cuda, G, values):
    """One thread block, 48 blocks of a head: keys that score more and more, by 31 log2
    units in steps, and values whose size changes by 2^values on the way."""
    N = SINK + LOCAL + 128 * 48 + 70
    case, k, v = _case(G, N, counts=(128, 128))
    k[..., :COMMON] = np.floor(np.linspace(0, 31, N))[None, :, None, None] / 8
    v *= 2.0 ** np.round(np.linspace(0, values, N))[None, :, None, None]
    _history(case, k, v)
    _decode(case, N, ctas=1)


def test_weights_over_rows_keep_24_bits(cuda):
    """100 rows of one value, one of each 16 (a warp's) of weight 1 and the others of the same
    weight p: o is that value whatever p is, but for what P's three bf16 numbers and some 30
    roundings leave, 30 * 2^-24.  Two bf16 numbers would leave out up to 2^-17 of p, in 93 of
    the 100 rows: the key is one for which they leave most."""
    bf = lambda x: float(torch.tensor(x, dtype=torch.float64).to(torch.bfloat16))  # noqa: E731
    tol = 30 * 2.0 ** -24

    def left(key):
        p = 2.0 ** (-key * LOG2)
        hi = bf(p)
        return abs(p - hi - bf(p - hi)) / p
    key = max((x / 16 for x in range(16, 256)), key=left)
    p = 2.0 ** (-key * LOG2)
    assert left(key) * 93 * p / (7 + 93 * p) > 2 * tol
    for G in (4, 7):
        w = TINY.scaled(num_q_heads=G, num_kv_heads=1, sink=4, local=200)
        case = Case(w, total=100, masks=S.masks_with_counts(w, (32,)), kv_format=FMT)
        k, v = np.zeros((1, 100, 1, 128)), np.full((1, 100, 1, 128), 1.25)
        k[..., 0] = -key
        k[:, ::16, :, 0] = 0
        _history(case, k, v)
        case.prefill(0, 100)
        q = torch.zeros(1, G, 128, dtype=torch.bfloat16, device="cuda")
        q[..., 0] = 1
        o = f64(case.cache.decode(0, q))
        case.cache.check()
        assert np.abs(o / 1.25 - 1).max() <= tol, (G, np.abs(o / 1.25 - 1).max())


@pytest.mark.parametrize("G", [4, 7])
def test_long_sums_are_as_exact_as_short_ones(cuda, G):
    """131,072 tokens of one value through one thread block, with scores that rise by 36 log2 units:
    o is that value.  The products' accumulators drop bits towards zero, up to 2^-23 of what
    they hold with each product; they take 8 stages of 3 blocks (twice, with G > 4), half of
    that on average: 24.5 * 2^-23.  A warp adds 64 such sums, and l's, 32 roundings each on average
    where their sizes are alike: 64 * 2^-24; its 24 weights of a stage to l: 12 * 2^-24; merges and
    the rest 30 * 2^-24.  In one accumulator the 2000 products would drop some 2^-14."""
    N, V = 131072, 1.75
    w = TINY.scaled(num_q_heads=G, num_kv_heads=1, sink=4, local=64)
    case = Case(w, total=N, masks=S.masks_with_counts(w, (32,)), kv_format=FMT)
    kept = int(np.nonzero(case.masks[0, 0])[0][0])
    k = torch.zeros(1, N, 1, 128, dtype=torch.bfloat16, device="cuda")
    k[0, :, 0, kept] = (torch.arange(N, device="cuda") * 9 // N).to(torch.bfloat16) * 32
    case.hist[0] = (k, torch.full_like(k, V))
    case.prefill(0, N)
    case.cache.set_decode_ctas(1)
    q = torch.zeros(1, G, 128, dtype=torch.bfloat16, device="cuda")
    q[..., kept] = 1
    for sharp in (0.0, 2.0 ** -6, 1.0):                # flat, a little, all
        o = f64(case.cache.decode(0, q * sharp))
        case.cache.check()
        off = np.abs(o / V - 1).max()
        assert off <= 24.5 * 2.0 ** -23 + 106 * 2.0 ** -24, (sharp, off)


def test_a_stream_of_its_own(cuda):
    """A decode on a stream that the current one does not wait for, and its output read
    once it is done."""
    N = 1500
    case, k, v = _case(4, N)
    _history(case, k, v)
    case.prefill(0, N)
    q = _queries(case)
    want = case.cache.decode(0, q).clone()
    s, o = torch.cuda.Stream(), torch.full_like(want, 3.0)
    s.wait_stream(torch.cuda.current_stream())
    case.cache.decode(0, q, o, stream=s)
    new = case.cache.decode(0, q, stream=s)
    s.synchronize()
    assert torch.equal(o, want) and torch.equal(new, want)
    case.cache.check()


# ------------------------------------------------------------------------------ chunks
COPIES = 80                                        # sequences: more items than there are SMs


def _chunk(case, k, v, held, n):
    """A chunk of n tokens on every one of COPIES sequences that hold the same: next to no item
    is cut, so that one softmax sees the sinks and the blocks."""
    kd, vd = (x.expand(COPIES, -1, -1, -1).contiguous() for x in _history(case, k, v))
    case.cache.prefill(0, kd[:, :held].contiguous(), vd[:, :held].contiguous())
    q = _queries(case, (n,)).expand(COPIES, -1, -1, -1).contiguous()
    got = case.cache.chunk_attn(0, q, kd[:, held:].contiguous(), vd[:, held:].contiguous())
    case.cache.check()
    keys = 0.0 if case.kv_format == FMT else 9.7e-3
    for i in range(0, n, 1 if n < 8 else 7):
        o, A = _expected(case, q[0, i], held + i + 1, held)
        _check(got[:, i], o, A, 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -12 + keys) * A)


@pytest.mark.parametrize("fmt", [FMT, lkb.KV_FP8, lkb.KV_INT8], ids=["fp8_block", "fp8", "int8"])
@pytest.mark.parametrize("gap", [0, 16, 24, 28, 32, 48])
@pytest.mark.parametrize("n", [2, 40])
def test_chunks_whose_sinks_score_far_above_the_blocks(cuda, n, gap, fmt):
    held = SINK + LOCAL + 128 * 6 + 50
    case, k, v = _case(4, held + n, fmt=fmt, batch=COPIES)
    k[:, :SINK, :, :COMMON] = gap / 8
    v[:, :SINK] = 0
    v[:, held - LOCAL:] /= 256
    _chunk(case, k, v, held, n)


@pytest.mark.parametrize("fmt", [FMT, lkb.KV_FP8, lkb.KV_INT8], ids=["fp8_block", "fp8", "int8"])
@pytest.mark.parametrize("zeros", [False, True], ids=["tiny", "zeros"])
@pytest.mark.parametrize("n", [2, 40])
def test_chunks_over_a_block_of_zeros_beside_huge_values(cuda, n, zeros, fmt):
    held = SINK + LOCAL + 128 * 3 + 50
    case, k, v = _case(4, held + n, fmt=fmt, batch=COPIES)
    v[:, SINK:SINK + 128] *= 0.0 if zeros else 2.0 ** -50
    v[:, :SINK] *= 2.0 ** 90
    v[:, held - LOCAL:] *= 2.0 ** 90
    _chunk(case, k, v, held, n)


@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("batch", [1, 7])
def test_chunks_in_parts_whose_references_fell_far(cuda, n, batch):
    """The same for items that are cut between thread blocks."""
    held = 843
    for counts in ((64, 64, 64), (32, 64, 128), (128, 32, 96)):
        case, k, v = _case(2, held + n, counts=counts, local=200, batch=batch)
        k[:, :SINK, :, :COMMON] = 7
        v[:, :SINK] = 0
        v[:, SINK:SINK + 128] = 0
        kd, vd = (x.expand(batch, -1, -1, -1).contiguous() for x in _history(case, k, v))
        case.cache.prefill(0, kd[:, :held].contiguous(), vd[:, :held].contiguous())
        q = _queries(case, (n,)).expand(batch, -1, -1, -1).contiguous()
        got = case.cache.chunk_attn(0, q, kd[:, held:].contiguous(), vd[:, held:].contiguous())
        case.cache.check()
        for i in range(n):
            o, A = _expected(case, q[0, i], held + i + 1, held)
            _check(got[:, i], o, A, 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -12) * A)
