"""Chunk attention and its append where they are most likely to go wrong: key
tiles of every width in turn, waits that run out, captured appends, offsets
past 32 bits, overlapping calls, rows beside rows with large scores.

Bounds against the fp64 oracle: those derived in test_gpu_chunk.py."""
import ctypes
import math

import numpy as np
import pytest
import torch

from decode_attention_pruned_gb300 import binding as lkb
from decode_attention_pruned_gb300 import synth as S
from helpers import Case
from test_gpu_chunk import _attend, _check, _chunk, _expected, _fill, _queries

pytestmark = pytest.mark.gpu

TINY = S.WORKLOADS[0]
FASTGEN = S.WORKLOADS[4]
FORMATS = [lkb.KV_BF16, lkb.KV_INT8, lkb.KV_FP8]
FORMAT_IDS = ["bf16", "int8", "fp8"]


@pytest.mark.parametrize("fmt", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("n", [1, 16, 17, 100])
def test_wide_tiles_then_kept_ones(cuda, fmt, n):
    """Several full-width tiles before those on 96 channels, for items that
    follow one another in a block (16 tokens of 8 heads fill one query tile)."""
    w = TINY.scaled(num_kv_heads=6, num_q_heads=48, batch=3, sink=130, local=400)
    case = Case(w, total=2200, masks=S.masks_with_counts(w, (96, 96, 128, 32, 0, 96)), kv_format=fmt)
    held = [2100, 700, 1313]
    _fill(case, held)
    _attend(case, held, n)


@pytest.mark.parametrize("fmt", [lkb.KV_INT8, lkb.KV_FP8], ids=["int8", "fp8"])
def test_stale_rows_behind_a_quantised_tail(cuda, fmt):
    """A slot's last request left NaN in the rows behind the next one's."""
    w = TINY.scaled(num_kv_heads=2, num_q_heads=8, batch=2, sink=4, local=40)
    case = Case(w, total=600, masks=S.masks_with_counts(w, (32, 96)), kv_format=fmt)
    bad = torch.full((600, 2, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    for b in range(2):
        case.cache.prefill_sequence(0, b, bad, bad)
        case.cache.release(b)
    held = [233, 75]                            # one block and a tail; a tail only
    k, v = case.history(0)
    for b in range(2):
        case.cache.prefill_sequence(0, b, k[b, :held[b]].contiguous(), v[b, :held[b]].contiguous())
    _attend(case, held, 7)
    _attend(case, held, 50)


@pytest.mark.parametrize("fmt", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("n", [2, 150])
def test_waits_that_run_out(cuda, fmt, n):
    """With a limit of 0 every wait that is not complete at once runs out: the
    call ends, says so, and leaves nothing behind that the next one meets."""
    w = TINY.scaled(num_kv_heads=4, num_q_heads=16, batch=2)
    case = Case(w, total=1500, masks=S.masks_with_counts(w, (32, 96, 0, 128)), kv_format=fmt)
    held = [1300, 801]
    _fill(case, held)
    q, (k, v, _) = _queries(case, n), _chunk(case, 0, held, n)
    case.cache.set_wait_limit(0)
    case.cache.chunk_attn(0, q, k, v)
    with pytest.raises(lkb.LeankError) as e:
        case.cache.check()
    assert e.value.status == lkb.LK_ERR_TIMEOUT
    case.cache.check()
    case.cache.set_wait_limit(10 ** 9)
    _attend(case, held, n)


@pytest.mark.parametrize("fmt", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("held, n", [([90, 20], 2), ([1300, 801], 5), ([90, 20], 150), ([1300, 801], 300)], ids=str)
def test_calls_right_behind_one_that_gave_up(cuda, fmt, held, n):
    """Where some of a block's waits run out, its other threads may be done with
    theirs: the block still ends only when its copies have landed, and what runs
    next, with no synchronisation between, is as if nothing had happened."""
    w = TINY.scaled(num_kv_heads=4, num_q_heads=16, batch=2)
    case = Case(w, total=1700, masks=S.masks_with_counts(w, (32, 96, 0, 128)), kv_format=fmt)
    _fill(case, held)
    q, (k, v, _) = _queries(case, n), _chunk(case, 0, held, n)
    want = _attend(case, held, n)
    torch.cuda.synchronize()
    for limit in (0, 1, 300, 1000, 3000, 10000) * 2:
        outs = []
        for _ in range(4):
            case.cache.set_wait_limit(limit)
            case.cache.chunk_attn(0, q, k, v)
            case.cache.set_wait_limit(10 ** 9)
            outs.append(case.cache.chunk_attn(0, q, k, v))
        for o in outs:
            assert torch.equal(o, want), limit
        if limit == 0:
            with pytest.raises(lkb.LeankError) as e:
                case.cache.check()
            assert e.value.status == lkb.LK_ERR_TIMEOUT
        else:
            try:
                case.cache.check()
            except lkb.LeankError as e:
                assert e.status == lkb.LK_ERR_TIMEOUT
    _attend(case, held, n)


def test_captured_extend_and_append(cuda):
    """A captured extend and append take the tokens at the lengths of the replay."""
    w = TINY.scaled(num_kv_heads=4, num_q_heads=8, batch=2, sink=4, local=30)
    masks = S.masks_with_counts(w, (32, 0, 96, 128))
    graphed, eager = (Case(w, total=400, masks=masks, middle_tokens=900) for _ in range(2))
    held, n = [150, 20], 9
    q, (k, v, _) = _queries(graphed, n), _chunk(graphed, 0, held, n)
    for c in (graphed, eager):
        _fill(c, held)
    out = torch.zeros_like(q)
    ref = [torch.zeros_like(q) for _ in range(3)]
    eager.cache.extend(0, q, k, v, lens=[9, 4], o=ref[0])
    graphed.cache.extend(0, q, k, v, lens=[9, 4], o=out)
    assert torch.equal(out, ref[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graphed.cache.extend(0, q, k, v, lens=[9, 4], o=out)
        graphed.cache.append_chunk(0, k, v, lens=[0, 7])
    for x in (1, 2):
        g.replay()
        eager.cache.extend(0, q, k, v, lens=[9, 4], o=ref[x])
        eager.cache.append_chunk(0, k, v, lens=[0, 7])
        torch.cuda.synchronize()
        assert torch.equal(out, ref[x]), x
        assert torch.equal(graphed.cache.buffer, eager.cache.buffer), x
    assert not torch.equal(ref[1], ref[2])


@pytest.mark.parametrize("fmt", [lkb.KV_BF16, lkb.KV_FP8], ids=["bf16", "fp8"])
def test_offsets_past_32_bits(cuda, fmt):
    """Rows more than 2^32 bytes into their pool, read and written."""
    w = TINY.scaled(num_kv_heads=8, num_q_heads=16, batch=2, sink=4, local=60)
    case = Case(w, total=700, masks=S.masks_with_counts(w, (128,) * 8), capacity=1_200_000, kv_format=fmt)
    held = [300, 650]
    _fill(case, held)
    if fmt == lkb.KV_BF16:
        assert case.cache.region(0, 1, 7).k_b_offset - case.cache.region(0, 0, 0).k_b_offset > 1 << 32
    else:                                       # 9374 blocks of 132 x 256 bytes for each of 15 before the last
        assert 15 * (1_200_000 - 64) // 128 * 132 * 256 > 1 << 32
    _attend(case, held, 30)
    _attend(case, held, 3)
    k, v, _ = _chunk(case, 0, held, 30)
    case.cache.append_chunk(0, k, v)
    case.check_layout(0, np.array(held) + 30)


def test_calls_overlap_on_two_streams(cuda):
    """Two calls at once on one cache, each with a workspace of its own."""
    w = TINY.scaled(num_kv_heads=4, num_q_heads=16, batch=2)
    case = Case(w, total=3000, masks=S.masks_with_counts(w, (32, 64, 0, 128)))
    held = [2900, 1500]
    _fill(case, held)
    cases = []
    for n, seed in ((5, 1), (90, 2)):
        q, (k, v, _) = _queries(case, n, seed), _chunk(case, 0, held, n)
        cases.append((q, k, v, case.cache.chunk_attn(0, q, k, v)))
    size = ctypes.c_size_t()
    assert lkb._lib.lk_chunk_workspace_bytes(case.plan._h, 2, 90, ctypes.byref(size)) == lkb.LK_OK
    spaces = [torch.empty(size.value, dtype=torch.uint8, device="cuda") for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.zeros_like(q) for q, _, _, _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for (q, k, v, _), ws, s, o in zip(cases, spaces, streams, outs):
            c, lens = case.cache._chunk(q, k, v, None, None)
            assert lkb._lib.lk_chunk_attn(case.cache._h, 0, ctypes.byref(c), o.data_ptr(), ws.data_ptr(), ws.numel(),
                                          s.cuda_stream) == lkb.LK_OK
    torch.cuda.synchronize()
    for (_, _, _, want), o in zip(cases, outs):
        assert torch.equal(o, want)


def test_layers_append_on_two_streams(cuda):
    """Appends to two layers that overlap: each layer's lengths advance by its own."""
    w = TINY.scaled(num_layers=2, num_kv_heads=4, num_q_heads=4, batch=2, sink=4, local=60)
    case = Case(w, total=900, masks=S.masks_with_counts(w, (32, 64, 0, 128) * 2))
    rows = [case.history(layer) for layer in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    sizes = ([7, 300, 2, 90, 1], [150, 3, 220, 8, 19])
    N = [0, 0]
    chunks = [[], []]
    for layer in range(2):
        for n in sizes[layer]:
            chunks[layer].append(tuple(t[:, N[layer]:N[layer] + n].contiguous() for t in rows[layer]))
            N[layer] += n
    torch.cuda.synchronize()
    for x in range(5):
        for layer in range(2):
            case.cache.append_chunk(layer, *chunks[layer][x], stream=streams[layer])
    torch.cuda.synchronize()
    for layer in range(2):
        case.check_layout(layer, N[layer])
    case.cache.check()


@pytest.mark.parametrize("G, n", [(4, 20), (3, 100), (8, 4)])
def test_rows_do_not_depend_on_each_other(cuda, G, n):
    w = TINY.scaled(num_kv_heads=2, num_q_heads=2 * G, batch=1)
    case = Case(w, total=1500, masks=S.masks_with_counts(w, (32, 128)))
    _fill(case, [1300])
    q, (k, v, _) = _queries(case, n), _chunk(case, 0, [1300], n)
    o = case.cache.chunk_attn(0, q, k, v)
    loud = q.clone()
    loud[:, 2] *= 60
    loud[:, 3, 1] = math.nan
    other = case.cache.chunk_attn(0, loud, k, v)
    rest = [i for i in range(n) if i not in (2, 3)]
    assert torch.equal(o[:, rest], other[:, rest])
    heads = [h for h in range(2 * G) if h != 1]
    assert torch.equal(o[:, 3][:, heads], other[:, 3][:, heads])
    ref, tol = _expected(case, 0, loud[:, :3], [1300], [3])
    _check(other[:, :3], (ref, tol))


def test_chunks_too_long(cuda):
    case = Case(TINY, total=64)
    _fill(case, [10])
    q, (k, v, _) = _queries(case, 4), _chunk(case, 0, [10], 4)
    o = case.cache.chunk_attn(0, q, k, v)
    c, _ = case.cache._chunk(q, k, v, None, None)
    ws = case.cache.chunk_workspace
    for n in ((1 << 28) + 1, 2 ** 31 - 1):
        c.n_max = n
        assert lkb._lib.lk_chunk_attn(case.cache._h, 0, ctypes.byref(c), o.data_ptr(), ws.data_ptr(), ws.numel(),
                                      None) == lkb.LK_ERR_UNSUPPORTED
        assert lkb._lib.lk_append_chunk(case.cache._h, 0, ctypes.byref(c), None) == lkb.LK_ERR_UNSUPPORTED


def test_tensors_of_another_device(cuda, monkeypatch):
    """Tensors that are not where the call runs are refused before any launch."""
    case = Case(TINY, total=64)
    _fill(case, [10])
    q, (k, v, _) = _queries(case, 4), _chunk(case, 0, [10], 4)
    for call in (lambda: case.cache.chunk_attn(0, q, k.cpu(), v), lambda: case.cache.append_chunk(0, k, v.cpu()),
                 lambda: case.cache.extend(0, q, k, v, o=torch.empty_like(q, device="cpu"))):
        with pytest.raises(ValueError):
            call()
    assert case.cache.length(0) == 10
    rope = lkb.Rope()
    pos = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    rope.apply(q, k, pos)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="cuda:0"):
        rope.apply(q, k, pos)
    with pytest.raises(ValueError):
        rope.apply(q[0, 0, 0], None, pos)


@pytest.mark.parametrize("n", [3, 60])
def test_policies_over_quantised_middles(cuda, n):
    w = S.WORKLOADS[4].scaled(num_layers=1, batch=2, context=700, policy_counts=(2, 2, 4))
    case = Case(w, total=800, kv_format=lkb.KV_FP8)
    held = [700, 301]
    _fill(case, held)
    _attend(case, held, n, lens=[n, n - 2])


@pytest.mark.parametrize("fmt", [lkb.KV_BF16, lkb.KV_INT8], ids=["bf16", "int8"])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_one_item_over_every_block(cuda, fmt, n):
    """One sequence, one kv head: its keys are cut into more partials than a warp has lanes."""
    w = TINY.scaled(num_kv_heads=1, num_q_heads=8, batch=1, sink=4, local=64)
    case = Case(w, total=60050, masks=S.masks_with_counts(w, (64,)), gen_device="cuda", kv_format=fmt)
    _fill(case, [60000])
    _attend(case, [60000], n)


def test_outputs_of_another_stream_are_its_own(cuda):
    """What the current stream has freed, and may still be using, is not handed
    to a call on another one."""
    w = TINY.scaled(num_kv_heads=2, num_q_heads=8, batch=2)
    case = Case(w, total=500, masks=S.masks_with_counts(w, (32, 96)))
    _fill(case, [400, 170])
    q, (k, v, _) = _queries(case, 20), _chunk(case, 0, [400, 170], 20)
    ref = case.cache.chunk_attn(0, q, k, v)
    rope, pos, one = lkb.Rope(), torch.zeros(2, 20, dtype=torch.int32, device="cuda"), q[:, 0].contiguous()
    sizes = {t.numel() * t.element_size() for t in (ref, q, one.float(), case.cache.chunk_workspace)}
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    spans = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in freed]
    del freed
    case.cache._chunk_tokens, spaces = 0, len(case.cache._chunk_workspaces)
    outs = [case.cache.chunk_attn(0, q, k, v, stream=s), rope.apply(q, None, pos, stream=s)[0],
            case.cache.decode(0, one, stream=s), case.cache._chunk_workspaces[-1]]
    assert len(case.cache._chunk_workspaces) == spaces + 1
    for t in outs:
        at, end = t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()
        assert all(end <= a or b <= at for a, b in spans)
    s.synchronize()
    assert torch.equal(outs[0], ref) and torch.equal(outs[1], q)


@pytest.mark.parametrize("k", [0, 32, 128])
@pytest.mark.parametrize("n", [3, 5, 60, 200])
def test_outputs_are_as_exact_as_two_roundings(cuda, k, n):
    """o and the weights are each rounded to bf16 once, off by a uniform share of half
    a step, 1.66e-3 of the value in the root mean square, and independently of one
    another: sqrt(2) times that over a head's outputs, and a fifth more for the few
    thousand of them here."""
    w = TINY.scaled(num_kv_heads=2, num_q_heads=8, batch=2, sink=4, local=64)
    case = Case(w, total=1700, masks=S.masks_with_counts(w, (k, k)))
    held = [1500, 1111]
    _fill(case, held)
    q, (key, v, _) = _queries(case, n), _chunk(case, 0, held, n)
    got = case.cache.chunk_attn(0, q, key, v).double().cpu().numpy()
    ref, _ = _expected(case, 0, q, held, [n, n])
    for b in range(2):
        for h in (slice(0, 4), slice(4, 8)):
            x, o = got[b, :, h], ref[b, :, h]
            assert math.sqrt(((x - o) ** 2).sum() / (o ** 2).sum()) <= 1.2 * 2.35e-3, (b, h)


@pytest.mark.parametrize("fmt", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("n", [1, 40, 150])
def test_windows_that_nothing_leaves(cuda, fmt, n):
    """Windows of 2^31 - 1 tokens: every token is near, and no sum passes an int32."""
    w = FASTGEN.scaled(num_layers=1, batch=2, num_q_heads=8, num_kv_heads=4, policy_counts=(2, 1, 1), sink=0,
                       local=2 ** 31 - 1, local_only_window=2 ** 31 - 1, context=400)
    masks = S.masks_with_counts(w, (32, 0, 96, 128))
    case = Case(w, total=600, masks=masks, kv_format=fmt)
    held = [400, 133]
    _fill(case, held)
    _attend(case, held, n)
    k, v, ids = _chunk(case, 0, held, n)
    case.cache.append_chunk(0, k, v, ids=ids)
    case.check_layout(0, np.array(held) + n)
    case.cache.check()
