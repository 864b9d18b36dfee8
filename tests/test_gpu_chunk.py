"""Attention of a chunk of new tokens, and the chunk's append, on the GPU.

The oracle of query i is the decode step's over the tokens 0 .. N + i, in fp64
(quantised middles: over the values the cache holds when the chunk arrives).

Bound of an output o = sum p v against it, with A = sum p |v|:
  2^-8 |o|       its rounding to bf16
  2^-8 A         p rounded to bf16 before p.V
  2^-12 A        fp32: scores of 128 products and their exponential
and where sealed blocks are read, 2 D A with D = 2^-8 max_t sum_c |q_c k_c| /
sqrt(128): the key's dequantised channels rounded to bf16 move a score by at
most D, a weight by e^D - 1, and so the normalised weights by about 2 D."""
import math

import numpy as np
import pytest
import torch

from decode_attention_pruned_gb300 import binding as lkb
from decode_attention_pruned_gb300 import synth as S
from helpers import Case, f64
from oracle import chunk as OC
from oracle import quant as OQ

pytestmark = pytest.mark.gpu

TINY = S.WORKLOADS[0]
LLAMA = S.WORKLOADS[1]
FASTGEN = S.WORKLOADS[4]


def _queries(case, n, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(977 + seed)
    q = torch.randn((case.w.batch, n, case.w.num_q_heads, 128), generator=g) * scale
    return q.to(torch.bfloat16).cuda()


def _chunk(case, layer, held, n):
    """k, v, ids [B, n, ...] of the tokens that follow held[b]."""
    k, v = case.history(layer)
    B = case.w.batch
    at = torch.as_tensor(held, device=k.device)[:, None] + torch.arange(n, device=k.device)
    at = at.clamp(max=k.shape[1] - 1)
    b = torch.arange(B, device=k.device)[:, None]
    ids = case.ids[b, at].contiguous() if len(case.is_special) else None
    return k[b, at].contiguous(), v[b, at].contiguous(), ids


def _expected(case, layer, q, held, lens, special_capacity=None):
    """(o, bound) fp64 [B, n, Hq, 128]; rows past lens are 0."""
    k, v = case.history(layer)
    w, G = case.w, case.w.group
    quant = case.kv_format != lkb.KV_BF16
    o = np.zeros(q.shape)
    tol = np.zeros(q.shape)
    for b in range(w.batch):
        N, n = int(held[b]), int(lens[b])
        if n == 0:
            continue
        for h in range(w.num_kv_heads):
            pol = int(case.policies[layer, h])
            kept = np.nonzero(case.masks[layer, h])[0] if pol == S.POLICY_FULL else np.arange(0)
            K, V = f64(k[b, :N + n, h]), f64(v[b, :N + n, h])
            flags = case.flags[b][:N + n].copy()
            if special_capacity is not None:
                flags[np.nonzero(flags)[0][special_capacity:]] = False
            Qh = f64(q[b, :n, h * G:(h + 1) * G])
            extra = 0.0
            if quant and pol == S.POLICY_FULL:
                K[:N], V[:N] = OQ.quantized_history(K[:N], V[:N], kept, pol, N, w.sink, w.local,
                                                    fmt=lkb.KV_FORMAT_NAMES[case.kv_format])
                extra = 2 * 2.0 ** -8 * np.abs(Qh).reshape(-1, 128).dot(np.abs(K).T).max(1).reshape(n, G, 1) / math.sqrt(128)
            args = (pol, kept, N, w.sink, w.local, w.local_only_window, flags)
            out = OC.chunk_head(Qh, K, V, *args)
            A = OC.chunk_head(Qh, K, np.abs(V), *args)
            o[b, :n, h * G:(h + 1) * G] = out
            tol[b, :n, h * G:(h + 1) * G] = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2.0 ** -12 + extra) * A
    return o, tol


def _check(got, want):
    ref, tol = want
    err = np.abs(got.double().cpu().numpy() - ref)
    bad = err > tol + 1e-30
    assert not bad.any(), (int(bad.sum()), float(err.max()), np.argwhere(bad)[:4].tolist())


def _fill(case, held, layer=0):
    """The first held[b] tokens of every sequence."""
    k, v = case.history(layer)
    top = max(held)
    ids = case.ids[:, :top].contiguous() if len(case.is_special) else None
    case.cache.prefill_ragged(layer, k[:, :top].contiguous(), v[:, :top].contiguous(), held, ids)


def _attend(case, held, n, lens=None, layer=0, seed=0, scale=1.0, special_capacity=None):
    q = _queries(case, n, seed, scale)
    k, v, ids = _chunk(case, layer, held, n)
    o = case.cache.chunk_attn(layer, q, k, v, lens=lens, ids=ids)
    case.cache.check()
    full = [n] * case.w.batch if lens is None else lens
    ref, tol = _expected(case, layer, q, held, full, special_capacity)
    for b, m in enumerate(full):
        _check(o[b, :m], (ref[b, :m], tol[b, :m]))
    return o


# ------------------------------------------------------------------ attention

# the tiny layer: S = 4, W = 64; the window starts to move at 68 tokens
@pytest.mark.parametrize("N, n", [(0, 1), (0, 2), (0, 4), (0, 5), (0, 68), (0, 69), (0, 200), (1, 1), (3, 3), (4, 64),
                                  (5, 64), (67, 1), (68, 1), (69, 130), (100, 31), (127, 33), (131, 129), (195, 64),
                                  (196, 65), (197, 257), (300, 16), (333, 7), (513, 128)])
def test_tiny_lengths(cuda, N, n):
    case = Case(TINY, total=N + n, masks=S.masks_with_counts(TINY, (0, 64)))
    _fill(case, [N])
    before = case.cache.buffer.clone()
    _attend(case, [N], n)
    assert torch.equal(before, case.cache.buffer)              # the cache is only read


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "paged"])
def test_group_sizes_and_widths(cuda, G, paged):
    w = TINY.scaled(num_kv_heads=5, num_q_heads=5 * G, batch=2, sink=16, local=100)
    case = Case(w, total=520, masks=S.masks_with_counts(w, (0, 32, 64, 96, 128)), middle_tokens=900 if paged else None)
    _fill(case, [467, 130])
    _attend(case, [467, 130], 53)


@pytest.mark.parametrize("sink, local", [(0, 1), (0, 128), (1, 300), (130, 7), (128, 128), (16, 129)])
def test_sinks_and_windows(cuda, sink, local):
    w = TINY.scaled(sink=sink, local=local)
    for N, n in ((0, 150), (sink + local, 140), (400, 99)):
        case = Case(w, total=N + n, masks=S.masks_with_counts(w, (96, 0)))
        _fill(case, [N])
        _attend(case, [N], n)


@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "paged"])
def test_ragged_padded_batch(cuda, paged):
    """Sequences of several lengths, some without new tokens; what lies past a
    sequence's length is NaN and is neither read nor written."""
    w = LLAMA.scaled(num_kv_heads=3, num_q_heads=12, batch=6, sink=16, local=80)
    case = Case(w, total=700, masks=S.masks_with_counts(w, (32, 0, 128)), middle_tokens=3000 if paged else None)
    held, lens, n = [500, 0, 96, 97, 333, 224], [37, 70, 0, 1, 64, 33], 70
    _fill(case, held)
    q = _queries(case, n)
    k, v, _ = _chunk(case, 0, held, n)
    for b, m in enumerate(lens):
        q[b, m:] = k[b, m:] = v[b, m:] = math.nan
    o = torch.full((w.batch, n, w.num_q_heads, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    assert case.cache.chunk_attn(0, q, k, v, lens=lens, o=o) is o
    ref, tol = _expected(case, 0, q, held, lens)
    for b, m in enumerate(lens):
        _check(o[b, :m], (ref[b, :m], tol[b, :m]))
        assert bool((o[b, m:] == 7.0).all())


@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "paged"])
def test_stale_rows_of_released_slots(cuda, paged):
    """A slot's last request left infinities and NaN behind; the next one is shorter."""
    w = TINY.scaled(num_kv_heads=2, num_q_heads=8, batch=2, sink=4, local=40)
    case = Case(w, total=600, masks=S.masks_with_counts(w, (32, 96)), middle_tokens=1200 if paged else None)
    bad = torch.full((600, 2, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    bad[::2] = math.inf
    for b in range(2):
        case.cache.prefill_sequence(0, b, bad, bad)
        case.cache.release(b)
    held = [150, 21]
    k, v = case.history(0)
    for b in range(2):
        case.cache.prefill_sequence(0, b, k[b, :held[b]].contiguous(), v[b, :held[b]].contiguous())
    _attend(case, held, 50)


@pytest.mark.parametrize("fmt", [lkb.KV_INT8, lkb.KV_FP8], ids=["int8", "fp8"])
@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "paged"])
def test_quantised_middles(cuda, fmt, paged):
    w = LLAMA.scaled(num_kv_heads=5, num_q_heads=20, batch=2, sink=16, local=64)
    case = Case(w, total=900, masks=S.masks_with_counts(w, (0, 32, 64, 96, 128)), kv_format=fmt,
                middle_tokens=1800 if paged else None)
    held = [850, 208]                 # 6 blocks and a tail; exactly one block
    _fill(case, held)
    _attend(case, held, 45)
    _attend(case, held, 3, lens=[3, 1], seed=1)


@pytest.mark.parametrize("n", [1, 40, 200])
def test_policies(cuda, n):
    w = FASTGEN.scaled(num_layers=2, batch=3, context=600, policy_counts=(6, 4, 6))
    case = Case(w, total=900)
    held = [600, 255, 0]
    for layer in range(2):
        _fill(case, held, layer)
        _attend(case, held, n, lens=[n, max(1, n - 9), n], layer=layer)


def test_special_tokens_run_out_of_rows(cuda):
    w = FASTGEN.scaled(num_layers=1, batch=2, num_q_heads=8, num_kv_heads=2, policy_counts=(0, 2, 0))
    case = Case(w, total=700, special_capacity=20)
    held = [300, 0]
    top = case.flags[0][:300].sum()
    assert top < 20 < case.flags[0][:700].sum()
    _fill(case, held)
    _attend(case, held, 400, special_capacity=20)


def test_no_special_token_gives_zero(cuda):
    w = FASTGEN.scaled(num_layers=1, batch=1, num_q_heads=4, num_kv_heads=1, policy_counts=(0, 1, 0))
    case = Case(w, total=64)
    q = _queries(case, 40)
    k, v, _ = _chunk(case, 0, [0], 40)
    plain = int(np.nonzero(case.is_special == 0)[0][0])
    special = int(np.nonzero(case.is_special)[0][0])
    ids = torch.full((1, 40), plain, dtype=torch.int32, device="cuda")
    assert not case.cache.chunk_attn(0, q, k, v).any()                       # no ids: no special token
    assert not case.cache.chunk_attn(0, q, k, v, ids=ids).any()
    ids[0, 33] = special                                                     # queries 33.. see that one token
    ids[0, 39] = -5
    o = case.cache.chunk_attn(0, q, k, v, ids=ids)
    assert not o[0, :33].any()
    assert torch.equal(o[0, 33:], v[0, 33, 0].expand(7, 4, 128))


@pytest.mark.parametrize("scale", [6.0, 40.0])
def test_peaky_scores(cuda, scale):
    """Large scores: the running maximum moves from tile to tile, and one
    weight takes nearly all."""
    w = TINY.scaled(num_kv_heads=2, num_q_heads=8)
    case = Case(w, total=1500, masks=S.masks_with_counts(w, (64, 128)))
    k, _ = case.history(0)
    k *= torch.linspace(0.2, 2.0, 1500, device="cuda")[None, :, None, None].to(torch.bfloat16)
    _fill(case, [1300])
    _attend(case, [1300], 200, scale=scale)


def test_one_token_equals_the_decode_step(cuda):
    w = LLAMA.scaled(context=1500, batch=2)
    case = Case(w, total=1501, masks=S.masks_with_counts(w, [0, 32, 64, 96, 128, 32, 0, 64]))
    _fill(case, [1500, 1100])
    q = _queries(case, 1)
    k, v, _ = _chunk(case, 0, [1500, 1100], 1)
    o = case.cache.chunk_attn(0, q, k, v)
    step = case.cache.step(0, q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous())
    ref, tol = _expected(case, 0, q, [1500, 1100], [1, 1])
    _check(o, (ref, tol))
    assert float((o[:, 0].float() - step).abs().max()) <= float(tol.max()) + 2e-3


def test_fused_projection_rows(cuda):
    """q, k and v as views of one projection's rows give the dense result bit for bit."""
    w = TINY.scaled(num_kv_heads=2, num_q_heads=14, batch=2)
    case = Case(w, total=400, masks=S.masks_with_counts(w, (32, 128)))
    held, n = [300, 77], 60
    _fill(case, held)
    q, (k, v, _) = _queries(case, n), _chunk(case, 0, held, n)
    rows = torch.cat([q, k, v], 2)
    dense = case.cache.chunk_attn(0, q, k, v)
    views = case.cache.chunk_attn(0, rows[:, :, :14], rows[:, :, 14:16], rows[:, :, 16:])
    assert torch.equal(dense, views)
    other = Case(w, total=400, masks=S.masks_with_counts(w, (32, 128)))
    _fill(other, held)
    case.cache.append_chunk(0, k, v)
    other.cache.append_chunk(0, rows[:, :, 14:16], rows[:, :, 16:])
    torch.cuda.synchronize()
    assert torch.equal(case.cache.buffer, other.cache.buffer)


def test_many_sequences(cuda):
    """More sequences than one launch takes."""
    w = TINY.scaled(num_kv_heads=1, num_q_heads=2, batch=300, sink=2, local=8)
    case = Case(w, total=40, masks=S.masks_with_counts(w, (32,)))
    held = [b % 30 for b in range(300)]
    lens = [b % 4 for b in range(300)]
    _fill(case, held)
    _attend(case, held, 3, lens=lens)
    k, v, _ = _chunk(case, 0, held, 3)
    case.cache.append_chunk(0, k, v, lens=lens)
    case.check_layout(0, np.array(held) + np.array(lens))


def test_long_cache(cuda):
    """A chunk far into a long sequence: the keys are split over many blocks."""
    w = LLAMA.scaled(num_kv_heads=2, num_q_heads=8, context=20000)
    case = Case(w, total=20010, masks=S.masks_with_counts(w, (32, 0)), gen_device="cuda")
    _fill(case, [20000])
    _attend(case, [20000], 5)
    _attend(case, [20000], 10, lens=[9], seed=3)


def test_graph_replays_and_streams(cuda):
    w = TINY.scaled(num_kv_heads=2, num_q_heads=8, batch=2)
    case = Case(w, total=500, masks=S.masks_with_counts(w, (32, 96)))
    held, n = [400, 170], 20
    _fill(case, held)
    q, (k, v, _) = _queries(case, n), _chunk(case, 0, held, n)
    ref = case.cache.chunk_attn(0, q, k, v, lens=[20, 11])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o = torch.zeros_like(ref)
    case.cache.chunk_attn(0, q, k, v, lens=[20, 11], o=o, stream=s)
    s.synchronize()
    assert torch.equal(o[0], ref[0]) and torch.equal(o[1, :11], ref[1, :11]) and not o[1, 11:].any()
    # two captured calls share the cache's workspace; the lengths are theirs
    graphs, outs = [], []
    for lens in ([20, 11], [3, 20]):
        out = torch.zeros_like(ref)
        g = torch.cuda.CUDAGraph()
        lens_host = list(lens)
        with torch.cuda.graph(g):
            case.cache.chunk_attn(0, q, k, v, lens=lens_host, o=out)
        graphs.append(g)
        outs.append(out)
    want = case.cache.chunk_attn(0, q, k, v, lens=[3, 20])
    for g in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], ref[0]) and torch.equal(outs[0][1, :11], ref[1, :11]) and not outs[0][1, 11:].any()
    assert torch.equal(outs[1][0, :3], want[0, :3]) and torch.equal(outs[1][1], want[1]) and not outs[1][0, 3:].any()


def test_calls_repeat_bit_for_bit(cuda):
    w = LLAMA.scaled(num_kv_heads=4, num_q_heads=16, context=5000, batch=2)
    case = Case(w, total=5100, masks=S.masks_with_counts(w, (32, 0, 64, 128)))
    _fill(case, [5000, 2000])
    q, (k, v, _) = _queries(case, 90), _chunk(case, 0, [5000, 2000], 90)
    a = case.cache.chunk_attn(0, q, k, v)
    for _ in range(3):
        assert torch.equal(a, case.cache.chunk_attn(0, q, k, v))


# --------------------------------------------------------------------- append

def _append_both(whole, steps, held, lens, layer=0):
    """The chunk at once on one cache, token by token on the other."""
    n = max(lens)
    k, v, ids = _chunk(whole, layer, held, n)
    whole.cache.append_chunk(layer, k, v, lens=lens, ids=ids)
    B = whole.w.batch
    assert len(set(lens)) == 1 or B == 1
    for t in range(n):
        steps.cache.append(layer, k[:, t].contiguous(), v[:, t].contiguous(),
                           None if ids is None else ids[:, t].contiguous())


@pytest.mark.parametrize("fmt", [lkb.KV_BF16, lkb.KV_INT8, lkb.KV_FP8], ids=["bf16", "int8", "fp8"])
@pytest.mark.parametrize("chunks", [[1, 2, 3, 4], [64, 64, 64], [68, 1], [300], [5, 200, 131, 128], [130, 257, 129, 127]],
                         ids=str)
def test_append_equals_single_appends(cuda, fmt, chunks):
    w = TINY.scaled(num_kv_heads=5, num_q_heads=5, batch=2)
    masks = S.masks_with_counts(w, (0, 32, 64, 96, 128))
    whole, steps = (Case(w, total=sum(chunks), masks=masks, kv_format=fmt) for _ in range(2))
    N = 0
    for n in chunks:
        _append_both(whole, steps, [N, N], [n, n])
        N += n
        whole.cache.check()
        steps.cache.check()
        torch.cuda.synchronize()
        assert torch.equal(whole.cache.buffer, steps.cache.buffer), (n, N)
    assert list(whole.cache.lengths(0)) == [N, N]
    whole.check_layout(0, N)


@pytest.mark.parametrize("fmt", [lkb.KV_BF16, lkb.KV_FP8], ids=["bf16", "fp8"])
def test_paged_append(cuda, fmt):
    w = TINY.scaled(num_kv_heads=3, num_q_heads=3, batch=3, sink=4, local=30)
    case = Case(w, total=700, masks=S.masks_with_counts(w, (32, 0, 96)), kv_format=fmt, middle_tokens=1500)
    N = np.zeros(3, np.int64)
    for lens in ([200, 33, 0], [1, 130, 500], [162, 128, 7], [300, 129, 100]):
        k, v, _ = _chunk(case, 0, N, max(lens))
        case.cache.append_chunk(0, k, v, lens=lens)
        N += lens
        case.check_layout(0, N)
        case.cache.check()
    used = sum(-(-max(0, int(n) - 34) // 128) if fmt == lkb.KV_BF16 else max(0, int(n) - 34) // 128 for n in N)
    for width in (32, 96):
        total, free = case.cache.pages(width)
        assert total - free == used
    case.cache.release(1)
    case.cache.prefill_sequence(0, 1, k[0, :0], v[0, :0])
    N[1] = 0
    k, v, _ = _chunk(case, 0, N, 290)
    case.cache.append_chunk(0, k, v, lens=[0, 290, 0])
    N[1] = 290
    case.check_layout(0, N)


def test_append_policies_and_special_rows(cuda):
    w = FASTGEN.scaled(num_layers=1, batch=2, policy_counts=(3, 2, 3))
    whole, steps = (Case(w, total=900, special_capacity=30) for _ in range(2))
    N = 0
    for n in (1, 255, 2, 300, 342):
        _append_both(whole, steps, [N, N], [n, n])
        N += n
        torch.cuda.synchronize()
        assert torch.equal(whole.cache.buffer, steps.cache.buffer), N
    # the special heads overflowed on both
    for c in (whole, steps):
        with pytest.raises(lkb.LeankError) as e:
            c.cache.check()
        assert e.value.status == lkb.LK_ERR_CAPACITY


def test_append_flags_a_bad_id(cuda):
    w = FASTGEN.scaled(num_layers=1, batch=1, policy_counts=(2, 3, 3))
    case = Case(w, total=20)
    k, v, ids = _chunk(case, 0, [0], 10)
    ids[0, 4] = w.vocab
    case.cache.append_chunk(0, k, v, ids=ids)
    with pytest.raises(lkb.LeankError) as e:
        case.cache.check()
    assert e.value.status == lkb.LK_ERR_ARG
    assert case.cache.length(0) == 10


def test_append_skips_released_slots(cuda):
    w = TINY.scaled(batch=2)
    case = Case(w, total=100)
    _fill(case, [50, 40])
    case.cache.release(1)
    k, v, _ = _chunk(case, 0, [50, 40], 9)
    q = _queries(case, 9)
    o = torch.full((2, 9, w.num_q_heads, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    case.cache.extend(0, q, k, v, o=o)
    assert list(case.cache.lengths(0)) == [59, 0]
    assert bool((o[1] == 3.0).all())
    ref, tol = _expected(case, 0, q, [50, 40], [9, 0])
    _check(o[:1], (ref[:1], tol[:1]))


# ------------------------------------------------------------------- together

@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "paged"])
def test_prompt_in_chunks_then_decode(cuda, paged):
    """A serving program: rotary positions, a prompt in odd chunks through
    extend, drafts verified without being appended, the accepted ones
    appended, then a decode step."""
    w = LLAMA.scaled(num_kv_heads=4, num_q_heads=16, batch=2, sink=16, local=128)
    T = 700
    case = Case(w, total=T + 20, masks=S.masks_with_counts(w, (0, 32, 64, 128)), middle_tokens=1500 if paged else None)
    rope = lkb.Rope(base=5e5)
    k_raw, v = case.history(0)
    pos = torch.arange(T + 20, dtype=torch.int32, device="cuda").expand(2, -1).contiguous()
    q_raw = _queries(case, T + 20)
    q, k = rope.apply(q_raw, k_raw, pos)
    case.hist[0] = (k, v)
    cut = lambda x, a, b: x[:, a:b].contiguous()  # noqa: E731
    at = 0
    for n in (1, 130, 200, 69, 300):
        o = case.cache.extend(0, cut(q, at, at + n), cut(k, at, at + n), cut(v, at, at + n))
        _check(o, _expected(case, 0, cut(q, at, at + n), [at, at], [n, n]))
        at += n
    assert at == T
    o = case.cache.chunk_attn(0, cut(q, T, T + 6), cut(k, T, T + 6), cut(v, T, T + 6))
    _check(o, _expected(case, 0, cut(q, T, T + 6), [T, T], [6, 6]))
    case.cache.append_chunk(0, cut(k, T, T + 6), cut(v, T, T + 6), lens=[6, 2])      # what was accepted
    N = np.array([T + 6, T + 2])
    case.check_layout(0, N)
    b = torch.arange(2, device="cuda")
    nxt = torch.as_tensor(N, device="cuda")
    qn, kn, vn = q[b, nxt].contiguous(), k[b, nxt].contiguous(), v[b, nxt].contiguous()
    step = case.cache.step(0, qn, kn, vn)
    case.cache.check()
    assert np.abs(f64(step) - case.expected(0, qn, N + 1)).max() <= 2e-3


def test_chunks_equal_one_prefill(cuda):
    """The cache after a chunked prompt is the one that lk_prefill builds."""
    w = TINY.scaled(num_kv_heads=4, num_q_heads=4, batch=2)
    masks = S.masks_with_counts(w, (0, 32, 96, 128))
    for fmt in (lkb.KV_BF16, lkb.KV_INT8):
        a, b = (Case(w, total=500, masks=masks, kv_format=fmt) for _ in range(2))
        k, v = a.history(0)
        b.cache.prefill(0, k, v)
        for i in range(0, 500, 77):
            a.cache.append_chunk(0, k[:, i:i + 77].contiguous(), v[:, i:i + 77].contiguous())
        torch.cuda.synchronize()
        assert torch.equal(a.cache.buffer, b.cache.buffer)


# ------------------------------------------------------------------- refusals

def test_refusals(cuda):
    w = TINY.scaled(batch=2)
    case = Case(w, total=100, masks=S.masks_with_counts(w, (32, 64)), middle_tokens=10)
    _fill(case, [70, 60])
    c = case.cache
    q, (k, v, _) = _queries(case, 8), _chunk(case, 0, [70, 60], 8)
    before = c.buffer.clone()

    def refused(status, call, *args, **kw):
        with pytest.raises(lkb.LeankError) as e:
            call(*args, **kw)
        assert e.value.status == status, str(e.value)

    refused(lkb.LK_ERR_ARG, c.chunk_attn, 1, q, k, v)
    refused(lkb.LK_ERR_ARG, c.append_chunk, -1, k, v)
    refused(lkb.LK_ERR_ARG, c.chunk_attn, 0, q, k, v, lens=[9, 1])
    refused(lkb.LK_ERR_ARG, c.extend, 0, q, k, v, lens=[-1, 1])
    kk = k.repeat(1, 5, 1, 1)
    refused(lkb.LK_ERR_CAPACITY, c.append_chunk, 0, kk, kk)                  # 70 + 40 > 100
    refused(lkb.LK_ERR_CAPACITY, c.extend, 0, q.repeat(1, 5, 1, 1), kk, kk)
    with pytest.raises(ValueError):
        c.chunk_attn(0, q, k, v, lens=[1])
    with pytest.raises(ValueError):
        c.chunk_attn(0, q[:, :4], k, v)
    with pytest.raises(ValueError):
        c.chunk_attn(0, q.float(), k, v)
    with pytest.raises(ValueError):
        c.chunk_attn(0, q, k, v, o=torch.empty_like(q).float())
    with pytest.raises(ValueError):
        c.append_chunk(0, k[..., :64], v)
    ch, lens = c._chunk(q, k, v, None, None)
    o = torch.empty_like(q)
    import ctypes
    call = lambda o=o.data_ptr(), ws=c.chunk_workspace.data_ptr(), n=c.chunk_workspace.numel(): \
        lkb._lib.lk_chunk_attn(c._h, 0, ctypes.byref(ch), o, ws, n, None)  # noqa: E731
    assert call(o=None) == lkb.LK_ERR_ARG
    assert call(o=o.data_ptr() + 2) == lkb.LK_ERR_ALIGN
    assert call(ws=None) == lkb.LK_ERR_ARG
    assert call(ws=c.chunk_workspace.data_ptr() + 16) == lkb.LK_ERR_ALIGN
    assert call(n=0) == lkb.LK_ERR_CAPACITY
    for field, value, status in (("q", None, lkb.LK_ERR_ARG), ("k", k.data_ptr() + 2, lkb.LK_ERR_ALIGN),
                                 ("q_stride", 64, lkb.LK_ERR_ARG), ("v_stride", 260, lkb.LK_ERR_ARG),
                                 ("k_stride", 1 << 40, lkb.LK_ERR_ARG), ("n_max", -1, lkb.LK_ERR_ARG),
                                 ("reserved", 1, lkb.LK_ERR_ARG)):
        old = getattr(ch, field)
        setattr(ch, field, value)
        assert call() == status, field
        setattr(ch, field, old)
    torch.cuda.synchronize()
    assert torch.equal(before, c.buffer) and list(c.lengths(0)) == [70, 60]
    # nothing to do is no error
    assert c.chunk_attn(0, q[:, :0], k[:, :0], v[:, :0]).shape == (2, 0, w.num_q_heads, 128)
    c.append_chunk(0, k, v, lens=[0, 0])
    assert list(c.lengths(0)) == [70, 60]


def test_too_few_pages(cuda):
    w = TINY.scaled(batch=2)
    case = Case(w, total=900, masks=S.masks_with_counts(w, (32, 64)), middle_tokens=10)     # 3 pages a head
    k, v, _ = _chunk(case, 0, [0, 0], 400)
    q = _queries(case, 400)
    free = case.cache.pages(32)
    for call in (lambda: case.cache.append_chunk(0, k, v), lambda: case.cache.extend(0, q, k, v)):
        with pytest.raises(lkb.LeankError) as e:
            call()
        assert e.value.status == lkb.LK_ERR_CAPACITY
    assert case.cache.pages(32) == free and list(case.cache.lengths(0)) == [0, 0]
    case.cache.append_chunk(0, k, v, lens=[400, 0])
    case.check_layout(0, np.array([400, 0]))
