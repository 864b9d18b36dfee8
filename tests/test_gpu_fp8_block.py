"""Caches whose sealed blocks have one scale for the keys and one for the values
(KV_FP8_BLOCK), against the fp64 oracle over the dequantised cache: sealing, decode,
chunks.

Bounds.  With A = sum p |v| of an output o = sum p v:
  decode (fp32 out): a weight is off by what its score is, sums of 128 products of
    magnitude up to sum |q k| / sqrt(128) each rounded 2^-24 of what stands in the
    accumulator, 2^-19 with room for both regions' factors and the exponential, times
    max_t sum |q k| / sqrt(128) =: D; P is held in two bf16 numbers hi + lo (|p - hi| <=
    2^-8 p, and lo is off by 2^-8 of that: 2^-16 p), or two f16 ones.  The normalised
    weights are off by twice that: 2 A (2^-19 (1 + D) + 2^-16).
  chunks (bf16 out): 2^-8 |o| for o, 2^-8 A for P in bf16, 2^-12 A for the rest."""
import numpy as np
import pytest
import torch

import test_gpu_quantized as TQ
from decode_attention_pruned_gb300 import binding as lkb
from decode_attention_pruned_gb300 import synth as S
from helpers import Case, f64
from oracle import attention as OA
from oracle import quant as OQ

pytestmark = pytest.mark.gpu

TINY, LLAMA, SERVING, FASTGEN = S.WORKLOADS[0], S.WORKLOADS[1], S.WORKLOADS[2], S.WORKLOADS[4]
FMT = lkb.KV_FP8_BLOCK


def _head(case, layer, b, h, N):
    k, v = case.history(layer)
    kept = np.nonzero(case.masks[layer, h])[0]
    return (*OQ.quantized_history(f64(k[b, :N, h]), f64(v[b, :N, h]), kept, int(case.policies[layer, h]), N,
                                  case.w.sink, case.w.local, "fp8_block"), kept)


def _check_decode(case, layer, q, o, held):
    w, G = case.w, case.w.group
    worst = 0.0
    for b in range(w.batch):
        N = int(held[b])
        for h in range(w.num_kv_heads):
            K, V, kept = _head(case, layer, b, h, N)
            qh, got = f64(q[b, h * G:(h + 1) * G]), f64(o[b, h * G:(h + 1) * G])
            args = (int(case.policies[layer, h]), kept, N, w.sink, w.local, w.local_only_window, case.flags[b])
            ref, A = OA.decode_head(qh, K, V, *args), OA.decode_head(qh, K, np.abs(V), *args)
            D = np.abs(qh) @ np.abs(K).T / np.sqrt(128.0) if N else np.zeros((G, 1))
            tol = 2 * A * (2.0 ** -19 * (1 + D.max(1, keepdims=True)) + 2.0 ** -16)
            off = float((np.abs(got - ref) / np.maximum(tol, 1e-300)).max())
            assert np.all(np.abs(got - ref) <= tol), (b, h, N, off)
            worst = max(worst, off)
    return worst


def _filled(w, masks, held, total=None, **kw):
    case = Case(w, total=total or max(max(held), 1), masks=masks, kv_format=FMT, **kw)
    k, v = case.history(0)
    n = max(max(held), 1)
    ids = case.ids[:, :n].contiguous() if len(case.is_special) else None
    case.cache.prefill_ragged(0, k[:, :n].contiguous(), v[:, :n].contiguous(), np.array(held, np.int32), ids)
    return case


# ------------------------------------------------ what holds for every quantised format
@pytest.mark.parametrize("counts", [(0, 64), (64, 64), None], ids=["k0-64", "k64-64", "seeded"])
def test_tiny_seal_during_appends(cuda, counts):
    TQ.test_tiny_seal_during_appends(cuda, FMT, counts)


def test_llama_layer_all_widths(cuda):
    TQ.test_llama_layer_all_widths(cuda, FMT)


@pytest.mark.parametrize("ctas", [1, 7, 0])
def test_split_invariance(cuda, ctas):
    TQ.test_split_invariance(cuda, FMT, ctas)


def test_prefill_equals_appends_byte_for_byte(cuda):
    TQ.test_prefill_equals_appends_byte_for_byte(cuda, FMT)


def test_fastgen_policy_mix_two_layers(cuda):
    TQ.test_fastgen_policy_mix_two_layers(cuda, FMT)


def test_paged_release_and_refill(cuda):
    TQ.test_paged_release_and_refill(cuda, FMT)


def test_all_layers_in_one_launch(cuda):
    TQ.test_all_layers_in_one_launch(cuda, FMT)


# ------------------------------------------------------------------------- sealing
@pytest.mark.parametrize("mag", [1.0, 1e-12, 1e-25, 3e34], ids=["one", "small", "below the least scale", "large"])
def test_sealed_bytes_of_edge_values(cuda, mag):
    """Codes and scales against the oracle's, byte for byte: ties between e4m3 values,
    neighbours of ties, zeros of both signs, blocks of zeros, values that the least
    scale leaves no code for."""
    w = TINY.scaled(num_q_heads=2, num_kv_heads=1, context=4 + 64 + 384)
    masks = S.masks_with_counts(w, (32,))
    N = w.context
    case = Case(w, total=N, masks=masks, kv_format=FMT)
    kept = np.nonzero(masks[0, 0])[0]
    rs = np.random.default_rng(5)
    grid = OQ.e4m3_value(np.arange(0x7F))
    ties = (grid[:-1] + grid[1:]) / 2
    edge = np.concatenate([ties, -ties, ties * (1 + 2.0 ** -7), ties * (1 - 2.0 ** -7), [0.0, -0.0, 448.0, -448.0]])
    k, v = torch.randn(1, N, 1, 128), torch.randn(1, N, 1, 128)
    scale = 2.0 ** np.round(np.log2(mag / 448))
    mid = slice(w.sink, w.sink + 384)
    kb, vb = rs.choice(edge, (384, len(kept))), rs.choice(edge, (384, 128))
    kb[0, 3] = vb[200, 100] = 448.0
    kb[128:256] = 0.0                                    # a block of zeros
    vb[256:] *= -0.0
    kk = k[0, mid, 0].numpy().astype(np.float64) * 1e30 if mag < 1 else k[0, mid, 0].numpy().astype(np.float64)
    kk[:, kept] = kb * scale
    k[0, mid, 0], v[0, mid, 0] = torch.from_numpy(kk), torch.from_numpy(vb * scale)
    case.hist[0] = (k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda())
    case.prefill(0, N)
    case.cache.check()
    case.check_layout(0, N)


def test_codes_of_every_significand(cuda):
    """A block for every significand that its largest value may have, with values of every
    significand: the codes are those of the correctly rounded quotients, byte for byte."""
    w = TINY.scaled(batch=8, num_q_heads=2, num_kv_heads=1, context=4 + 64 + 16 * 128)
    masks = S.masks_with_counts(w, (32,))
    N = w.context
    case = Case(w, total=N, masks=masks, kv_format=FMT)
    rs = np.random.default_rng(11)
    k, v = (rs.integers(128, 256, (8, N, 1, 128)) * 2.0 ** rs.integers(-18, -7, (8, N, 1, 128)) *
            rs.choice([-1.0, 1.0], (8, N, 1, 128)) for _ in range(2))
    for b in range(8):
        for j in range(16):
            rows = slice(w.sink + 128 * j, w.sink + 128 * (j + 1))
            top = (128 + 16 * b + j) * 2.0 ** -7
            for x in (k, v):
                x[b, rows] = np.clip(x[b, rows], -top, top)
                x[b, rows.start + 37, 0] = top
    case.hist[0] = tuple(torch.from_numpy(x).to(torch.bfloat16).cuda() for x in (k, v))
    case.prefill(0, N)
    case.cache.check()
    case.check_layout(0, N)


@pytest.mark.parametrize("paged", [False, True], ids=["flat", "paged"])
def test_every_way_in_gives_the_same_bytes(cuda, paged):
    """Prefill, chunks and single tokens seal the same blocks; every policy."""
    w = FASTGEN.scaled(num_layers=1, batch=2, context=900, policy_counts=(2, 2, 4), sink=4, local=40,
                       local_only_window=24)
    cases = [Case(w, total=700, kv_format=FMT, middle_tokens=1400 if paged else None) for _ in range(3)]
    k, v = cases[0].history(0)
    cases[0].prefill(0, 700)
    at = 0
    for n in (30, 200, 1, 300, 169):
        ids = cases[1].ids[:, at:at + n].contiguous()
        cases[1].cache.append_chunk(0, k[:, at:at + n].contiguous(), v[:, at:at + n].contiguous(), ids=ids)
        at += n
    cases[2].prefill(0, 160)
    for t in range(160, 700):
        cases[2].append(0, t)
    for c in cases:
        c.cache.check()
        c.check_layout(0, 700)
    torch.cuda.synchronize()
    if not paged:
        assert torch.equal(cases[0].cache.buffer, cases[1].cache.buffer)
        assert torch.equal(cases[0].cache.buffer, cases[2].cache.buffer)


# -------------------------------------------------------------------------- decode
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8])
def test_groups_and_widths(cuda, G):
    w = LLAMA.scaled(num_q_heads=6 * G, num_kv_heads=6, batch=3, sink=4, local=100)
    masks = S.masks_with_counts(w, (0, 32, 64, 96, 128, 32))
    held = [1030, 333, 700]
    case = _filled(w, masks, held)
    q = case.q(0, 1030)
    o = case.cache.decode(0, q)
    case.cache.check()
    _check_decode(case, 0, q, o, held)


@pytest.mark.parametrize("sink, local", [(0, 1), (4, 64), (16, 17)])
def test_lengths_around_every_border(cuda, sink, local):
    """Empty sequences, one token, the sinks, the window and a block, and one either
    side of each; the last slab of each region full or not."""
    c = sink + local
    held = [0, 1, sink, sink + 1, c - 1, c, c + 1, c + 15, c + 16, c + 17, c + 127, c + 128, c + 129, c + 144, c + 255,
            c + 256, c + 385, 5]
    w = TINY.scaled(batch=len(held), num_q_heads=6, num_kv_heads=2, sink=sink, local=local)
    case = _filled(w, S.masks_with_counts(w, (32, 96)), held)
    q = case.q(0, 300)
    o = case.cache.decode(0, q)
    case.cache.check()
    _check_decode(case, 0, q, o, held)
    assert bool((o[0] == 0).all())


@pytest.mark.parametrize("ctas", [1, 2, 3, 50, 0])
def test_ctas_and_pages(cuda, ctas):
    """However the line is cut: within the bounds, and the same bits in every call."""
    w = SERVING.scaled(num_layers=1, batch=5, num_q_heads=8, num_kv_heads=4, sink=16, local=64)
    held = [3000, 1500, 2999, 40, 0]
    case = _filled(w, S.masks_with_counts(w, (32, 0, 64, 128)), held, middle_tokens=7600)
    case.cache.set_decode_ctas(ctas)
    q = case.q(0, 3000)
    o = case.cache.decode(0, q).clone()
    case.cache.check()
    _check_decode(case, 0, q, o, held)
    for _ in range(3):
        assert torch.equal(case.cache.decode(0, q), o)


def test_many_entries(cuda):
    """More entries than a block has threads, most of them short."""
    w = TINY.scaled(batch=170, num_q_heads=8, num_kv_heads=2, sink=2, local=8)
    held = [(37 * i) % 300 for i in range(170)]
    case = _filled(w, S.masks_with_counts(w, (32, 64)), held)
    q = case.q(0, 300)
    o = case.cache.decode(0, q)
    case.cache.check()
    _check_decode(case, 0, q, o, held)


@pytest.mark.parametrize("batch", [2, 11], ids=["heads", "heads and lengths"])
def test_more_heads_and_lengths_than_shared_memory_keeps(cuda, batch):
    """All layers in one launch: 56 (layer, head) descriptors and up to 616 lengths, of
    which places are kept for 48 and 512."""
    w = TINY.scaled(num_layers=7, batch=batch, num_q_heads=8, num_kv_heads=8, sink=2, local=8)
    case = Case(w, total=300, masks=S.masks_with_counts(w, np.resize([32, 64, 0, 96, 128], 56)), kv_format=FMT)
    held = [[(97 * b + 41 * layer) % 300 for b in range(batch)] for layer in range(7)]
    for layer in range(7):
        k, v = case.history(layer)
        case.cache.prefill_ragged(layer, k, v, np.array(held[layer], np.int32))
    q = torch.stack([case.q(layer, 300) for layer in range(7)]).contiguous()
    o = case.cache.decode_layers(0, q)
    case.cache.check()
    for layer in range(7):
        _check_decode(case, layer, q[layer], o[layer], held[layer])


@pytest.mark.parametrize("shift", [0, 40, -40], ids=["alike", "growing", "shrinking"])
def test_scales_that_differ_between_blocks(cuda, shift):
    """Values, and keys, whose size changes by 2^shift from the window to the oldest
    block: the running maximum follows scores times scales."""
    w = TINY.scaled(num_q_heads=8, num_kv_heads=2, sink=4, local=32)
    N = 36 + 128 * 6 + 50
    case = Case(w, total=N, masks=S.masks_with_counts(w, (64, 128)), kv_format=FMT)
    k, v = (x.clone() for x in case.history(0))
    step = torch.linspace(1, 0, N, device="cuda") * shift
    v = (v.float() * torch.exp2(step.round())[None, :, None, None]).to(torch.bfloat16)
    k = (k.float() * torch.exp2((step / 20).round())[None, :, None, None]).to(torch.bfloat16)
    case.hist[0] = (k, v)
    case.prefill(0, N)
    q = case.q(0, N)
    o = case.cache.decode(0, q)
    case.cache.check()
    _check_decode(case, 0, q, o, [N])


@pytest.mark.parametrize("size", [2.0 ** -20, 1.0, 30.0])
def test_sharp_and_flat_scores(cuda, size):
    """From weights that are all alike to one that is all; q far below 1 and above."""
    w = TINY.scaled(num_q_heads=8, num_kv_heads=2, batch=2)
    held = [900, 333]
    case = _filled(w, S.masks_with_counts(w, (32, 64)), held)
    q = (case.q(0, 900).float() * size).to(torch.bfloat16)
    o = case.cache.decode(0, q)
    case.cache.check()
    _check_decode(case, 0, q, o, held)


def test_rows_that_hold_nothing_are_not_read(cuda):
    """NaN in rows behind a sequence's last, as a request before may have left them."""
    w = TINY.scaled(batch=3, num_q_heads=8, num_kv_heads=2, sink=4, local=100)
    held = [50, 104 + 128 + 5, 7]
    case = _filled(w, S.masks_with_counts(w, (64, 96)), held, total=600)
    for b in range(3):
        for h in range(2):
            r = case.cache.region(0, b, h)
            n = min(held[b], 104)
            for at in (r.k_a_offset, r.v_a_offset):
                case.cache.rows(at, r.rows_a, 128)[n:] = float("nan")
            n = max(held[b] - 104, 0) % 128
            case.cache.rows(r.k_b_offset, r.rows_b, r.n_kept)[n:] = float("nan")
            case.cache.rows(r.v_b_offset, r.rows_b, 128)[n:] = float("nan")
    q = case.q(0, 300)
    o = case.cache.decode(0, q)
    case.cache.check()
    _check_decode(case, 0, q, o, held)


def test_offsets_past_32_bits(cuda):
    """The last head of the last sequence lies beyond 4 GB of blocks."""
    w = TINY.scaled(batch=2, num_q_heads=8, num_kv_heads=8, sink=4, local=64)
    case = Case(w, total=700, masks=S.masks_with_counts(w, (128,) * 8), capacity=1_300_000, kv_format=FMT)
    k, v = case.history(0)
    case.cache.prefill_ragged(0, k, v, [700, 600])
    q = case.q(0, 700)
    o = case.cache.decode(0, q)
    case.cache.check()
    _check_decode(case, 0, q, o, [700, 600])


def test_graph_streams_and_the_static_form(cuda):
    w = LLAMA.scaled(num_q_heads=8, num_kv_heads=2, batch=2, sink=4, local=64)
    case = _filled(w, S.masks_with_counts(w, (32, 64)), [2000, 1500], total=2010)
    q = case.q(0, 2000)
    o = case.cache.decode(0, q).clone()
    out = torch.zeros_like(o)
    assert torch.equal(case.cache.decode_static(0, q, out), o)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert torch.equal(case.cache.decode(0, q, stream=s), o) or s.synchronize()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        case.cache.decode(0, q, out)
    q.copy_(case.q(0, 2000, step=3))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, case.cache.decode(0, q))
    # a step is an append and a decode, from host memory too
    k1, v1 = (x[:, 2000].contiguous() for x in case.history(0))
    other = _filled(w, S.masks_with_counts(w, (32, 64)), [2000, 1500], total=2010)
    assert not other.cache.step_is_fused()
    a = other.cache.step(0, q, k1, v1)
    case.cache.append(0, k1, v1)
    assert torch.equal(case.cache.decode(0, q), a)
    assert torch.equal(case.cache.buffer, other.cache.buffer)
    pin = [x.cpu().pin_memory() for x in (q, k1, v1)]
    host = torch.zeros(2, 8, 128).pin_memory()
    other.cache.step_host(0, *pin, None, host)
    case.cache.append(0, k1, v1)
    want = case.cache.decode(0, q)
    torch.cuda.synchronize()
    assert torch.equal(host, want.cpu())


def test_resident_bytes(cuda):
    w = SERVING.scaled(num_layers=1, batch=2, sink=16, local=64)
    case = _filled(w, S.masks_with_counts(w, (0, 32, 64, 96, 128, 32, 0, 64)), [2000, 100])
    want = sum(OQ.resident_bytes_quantized(0, int(case.masks[0, h].sum()), n, 16, 64, 0, fmt="fp8_block")
               if case.masks[0, h].sum() < 128 else
               min(n, 80) * 512 + (max(n - 80, 0) // 128) * (128 * 256 + 16) + max(n - 80, 0) % 128 * 512
               for n in (2000, 100) for h in range(8))
    assert case.cache.resident_bytes(0) == want


# -------------------------------------------------------------------------- chunks
def _check_chunk(case, q, o, held, lens):
    w, G = case.w, case.w.group
    k, v = case.history(0)
    for b in range(w.batch):
        N, n = int(held[b]), int(lens[b])
        assert bool((o[b, n:] == 3.0).all())
        for h in range(w.num_kv_heads):
            kept = np.nonzero(case.masks[0, h])[0]
            pol = int(case.policies[0, h])
            K, V = f64(k[b, :N + n, h]), f64(v[b, :N + n, h])
            K[:N], V[:N], _ = _head(case, 0, b, h, N)
            for i in range(n):
                qh = f64(q[b, i, h * G:(h + 1) * G])
                args = (pol, kept, N + i + 1, w.sink, w.local, w.local_only_window, case.flags[b])
                ref, A = OA.decode_head(qh, K, V, *args), OA.decode_head(qh, K, np.abs(V), *args)
                err = np.abs(f64(o[b, i, h * G:(h + 1) * G]) - ref)
                tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * A
                assert np.all(err <= tol), (b, h, i, float((err / np.maximum(tol, 1e-300)).max()))


def _chunk_case(w, masks, held, n, lens=None, **kw):
    total = max(held) + n
    case = Case(w, total=total, masks=masks, kv_format=FMT, **kw)
    k, v = case.history(0)
    ids = case.ids if len(case.is_special) else None
    case.cache.prefill_ragged(0, k, v, np.array(held, np.int32), ids)
    at = torch.as_tensor(held, device="cuda")[:, None] + torch.arange(n, device="cuda")
    b = torch.arange(w.batch, device="cuda")[:, None]
    q = torch.randn(w.batch, n, w.num_q_heads, 128, generator=torch.Generator().manual_seed(5))
    q, k1, v1 = q.to(torch.bfloat16).cuda(), k[b, at].contiguous(), v[b, at].contiguous()
    id1 = case.ids[b, at].contiguous() if ids is not None else None

    def call():
        o = torch.full((w.batch, n, w.num_q_heads, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        return case.cache.chunk_attn(0, q, k1, v1, lens=lens, ids=id1, o=o)
    o = call()
    case.cache.check()
    _check_chunk(case, q, o, held, [n] * w.batch if lens is None else lens)
    return case, call, o


@pytest.mark.parametrize("G", [1, 4, 7, 8])
@pytest.mark.parametrize("n", [1, 5, 40])
def test_chunks_over_every_width(cuda, n, G):
    w = LLAMA.scaled(num_q_heads=6 * G, num_kv_heads=6, batch=2, sink=4, local=60)
    _chunk_case(w, S.masks_with_counts(w, (0, 32, 64, 96, 128, 32)), [900, 333], n)


def test_chunks_ragged_paged_and_policies(cuda):
    w = FASTGEN.scaled(num_layers=1, batch=3, policy_counts=(2, 2, 4), sink=4, local=40, local_only_window=24)
    _chunk_case(w, None, [800, 100, 0], 30, lens=[30, 0, 17], middle_tokens=1400)


def test_long_chunks(cuda):
    w = TINY.scaled(num_q_heads=4, num_kv_heads=1, sink=4, local=60)
    for k in (32, 96, 128):
        _chunk_case(w, S.masks_with_counts(w, (k,)), [1500], 130)


@pytest.mark.parametrize("shift", [30, -30])
def test_chunks_over_scales_that_differ(cuda, shift):
    w = TINY.scaled(num_q_heads=8, num_kv_heads=2, sink=4, local=32)
    held, n = 36 + 128 * 5 + 20, 4
    case = Case(w, total=held + n, masks=S.masks_with_counts(w, (64, 128)), kv_format=FMT)
    k, v = case.history(0)
    step = torch.linspace(1, 0, held + n, device="cuda") * shift
    case.hist[0] = k, v = k, (v.float() * torch.exp2(step.round())[None, :, None, None]).to(torch.bfloat16)
    case.cache.prefill(0, k[:, :held].contiguous(), v[:, :held].contiguous())
    q = torch.randn(1, n, 8, 128, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    o = case.cache.chunk_attn(0, q, k[:, held:].contiguous(), v[:, held:].contiguous())
    case.cache.check()
    _check_chunk(case, q, o, [held], [n])


@pytest.mark.parametrize("n", [1, 17, 40])
def test_chunks_wide_tiles_then_blocks(cuda, n):
    """Several full-width tiles before those made of blocks, for items that follow one
    another in a thread block; blocks that come in pages."""
    w = TINY.scaled(num_kv_heads=4, num_q_heads=32, batch=3, sink=130, local=400)
    _chunk_case(w, S.masks_with_counts(w, (96, 128, 32, 0)), [2000, 700, 1313], n, middle_tokens=4000)


@pytest.mark.parametrize("paged", [False, True], ids=["flat", "paged"])
@pytest.mark.parametrize("n", [2, 60])
def test_chunk_waits_that_run_out(cuda, n, paged):
    """With a limit of 0, and with ones that run out on the way, a call ends and leaves
    nothing behind: the next one, with no synchronisation between, is as before."""
    w = TINY.scaled(num_kv_heads=4, num_q_heads=16, batch=2, sink=4, local=30)
    masks = S.masks_with_counts(w, (32, 96, 0, 128))
    case, call, want = _chunk_case(w, masks, [1300, 801], n, **(dict(middle_tokens=2400) if paged else {}))
    case.cache.set_wait_limit(0)
    call()
    with pytest.raises(lkb.LeankError) as e:
        case.cache.check()
    assert e.value.status == lkb.LK_ERR_TIMEOUT
    case.cache.check()
    for limit in (0, 1, 300, 1000, 3000, 10000) * 2:
        outs = []
        for _ in range(3):
            case.cache.set_wait_limit(limit)
            call()
            case.cache.set_wait_limit(10 ** 9)
            outs.append(call())
        for o in outs:
            assert torch.equal(o, want), limit
        try:
            case.cache.check()
        except lkb.LeankError as e:
            assert e.status == lkb.LK_ERR_TIMEOUT
    assert torch.equal(call(), want)
    case.cache.check()


def test_calls_overlap_on_two_streams(cuda):
    """Decodes and chunks over one cache, each with its own workspace, at once."""
    w = TINY.scaled(num_kv_heads=4, num_q_heads=16, batch=2, sink=4, local=30)
    case, call, want = _chunk_case(w, S.masks_with_counts(w, (32, 96, 64, 128)), [1300, 801], 9)
    q = case.q(0, 1300)
    first = case.cache.decode(0, q).clone()
    other = torch.zeros_like(case.cache.workspace)
    lib, s = lkb.load(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs, chunks = [torch.empty_like(first) for _ in range(20)], []
    for o in outs:
        st = lib.lk_decode_attn(case.cache._h, 0, q.data_ptr(), o.data_ptr(), other.data_ptr(), other.numel(),
                                s.cuda_stream)
        assert st == lkb.LK_OK
        chunks.append(call())
        assert torch.equal(case.cache.decode(0, q), first)
    torch.cuda.synchronize()
    case.cache.check()
    assert all(torch.equal(o, first) for o in outs) and all(torch.equal(o, want) for o in chunks)


def test_prompt_steps_and_verification_together(cuda):
    """As a server uses them: a prompt enters turned, steps follow, a chunk of drafts is
    turned, attended with and partly appended, steps follow."""
    w = LLAMA.scaled(num_q_heads=8, num_kv_heads=2, batch=2, sink=4, local=60)
    masks = S.masks_with_counts(w, (32, 96))
    case = Case(w, total=520, masks=masks, kv_format=FMT, middle_tokens=1000)
    rope = lkb.Rope(axes=[24, 20, 20], axis_order=lkb.ROPE_AXES_CYCLIC)
    raw = [x.clone() for x in case.history(0)]
    pos = torch.randint(0, 3000, (3, 2, 520), dtype=torch.int32, device="cuda")
    turned = rope.apply(None, raw[0], pos)[1]
    case.hist[0] = (turned, raw[1])                      # what the cache has to hold
    k, v = raw
    at = lambda i, j: pos[:, :, i:j].contiguous()  # noqa: E731
    held = np.array([400, 300], np.int32)
    case.cache.append_rope(0, rope, k[:, :400].contiguous(), v[:, :400].contiguous(), positions=at(0, 400), lens=held)
    b = torch.arange(2, device="cuda")
    for step in range(30):
        i = torch.from_numpy(held.astype(np.int64)).cuda()
        q = case.q(0, 400, step=step)
        p = pos[:, b, i].contiguous()
        o = case.cache.step_rope(0, rope, q, k[b, i].contiguous(), v[b, i].contiguous(), positions=p)
        held += 1
        if step % 9 == 0:
            qt = rope.apply(q, None, p)[0]
            _check_decode(case, 0, qt, o, held)
    n = 5
    i = torch.from_numpy(held.astype(np.int64)).cuda()[:, None] + torch.arange(n, device="cuda")
    q = torch.randn(2, n, 8, 128, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).cuda()
    qt, kt = rope.apply(q, k[b[:, None], i].contiguous(), pos[:, b[:, None], i].contiguous())
    o = case.cache.chunk_attn(0, qt, kt, v[b[:, None], i].contiguous())
    _check_chunk(case, qt, o, held, [n, n])
    case.cache.append_chunk(0, kt, v[b[:, None], i].contiguous(), lens=[3, 0])
    held += np.array([3, 0], np.int32)
    case.cache.check()
    case.check_layout(0, held)


@pytest.mark.parametrize("paged", [False, True], ids=["flat", "paged"])
def test_waits_that_run_out(cuda, paged):
    """With a limit of 0 every wait of a decode that is not complete at once runs
    out: the call ends and says so, and with the limit back and the workspace
    zeroed the next one is right."""
    w = TINY.scaled(num_kv_heads=4, num_q_heads=16, batch=3, sink=4, local=30)
    held = [1400, 1, 260]
    case = _filled(w, S.masks_with_counts(w, (32, 64, 96, 128)), held, **(dict(middle_tokens=4000) if paged else {}))
    q = case.q(0, max(held))
    want = case.cache.decode(0, q).clone()
    case.cache.check()
    for ctas in (1, 4, 0):
        case.cache.set_decode_ctas(ctas)
        case.cache.set_wait_limit(0)
        case.cache.decode(0, q)
        with pytest.raises(lkb.LeankError) as e:
            case.cache.check()
        assert e.value.status == lkb.LK_ERR_TIMEOUT
        case.cache.check()
        case.cache.set_wait_limit(10 ** 9)
        case.cache.workspace_init()
        o = case.cache.decode(0, q)
        case.cache.check()
        _check_decode(case, 0, q, o, held)
    assert torch.equal(o, want)
