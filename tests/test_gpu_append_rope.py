"""Appends that turn their keys on the way, and steps that do: the cache and the
queries have to be, bit for bit, what turning first and appending then gives (which
is tested against the oracle elsewhere)."""
import numpy as np
import pytest
import torch

from decode_attention_pruned_gb300 import binding as lkb
from decode_attention_pruned_gb300 import synth as S
from helpers import Case

pytestmark = pytest.mark.gpu

TINY, LLAMA, FASTGEN = S.WORKLOADS[0], S.WORKLOADS[1], S.WORKLOADS[4]
FORMATS = [lkb.KV_BF16, lkb.KV_INT8, lkb.KV_FP8, lkb.KV_FP8_BLOCK]
NAMES = [lkb.KV_FORMAT_NAMES[f] for f in FORMATS]
FULL_HEADS = (0, 32, 64, 96, 128, 32)


def _draw(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def _rope(kind):
    return {"plain": lambda: lkb.Rope(base=1e6),
            "part": lambda: lkb.Rope(rotary_dim=64, layout=lkb.ROPE_INTERLEAVED),
            "half-part": lambda: lkb.Rope(rotary_dim=48, base=5e5),
            "axes": lambda: lkb.Rope(axes=[16, 24, 24]),
            "axes-own": lambda: lkb.Rope(layout=lkb.ROPE_INTERLEAVED, axes=[24, 20, 20], axis_order=lkb.ROPE_AXES_CYCLIC,
                                         axis_spectrum=lkb.ROPE_SPECTRUM_OWN)}[kind]()


def _workload(batch, policies=False, **kw):
    """Six FULL heads of every width, or a mix of policies."""
    if policies:
        return FASTGEN.scaled(num_layers=1, batch=batch, policy_counts=(2, 2, 4), **kw), None
    w = LLAMA.scaled(num_q_heads=12, num_kv_heads=6, batch=batch, **kw)
    return w, S.masks_with_counts(w, FULL_HEADS)


def _twins(w, masks, total, fmt, paged=False):
    middle = w.batch * total if paged else None
    return [Case(w, total=total, masks=masks, kv_format=fmt, middle_tokens=middle) for _ in range(2)]


def _same_caches(a, b, layer=0):
    """All that the two caches hold of a layer is equal."""
    a.cache.check()
    b.cache.check()
    assert np.array_equal(a.cache.lengths(layer), b.cache.lengths(layer))
    torch.cuda.synchronize()
    if not a.cache.paged:
        assert torch.equal(a.cache.buffer, b.cache.buffer)
        return
    w = a.w
    for i in range(w.batch):
        n = int(a.cache.lengths(layer)[i])
        for h in range(w.num_kv_heads):
            r, s = a.cache.region(layer, i, h), b.cache.region(layer, i, h)
            for at in ("k_a_offset", "v_a_offset"):
                assert torch.equal(a.cache.rows(getattr(r, at), r.rows_a, 128), b.cache.rows(getattr(s, at), s.rows_a, 128))
            assert r.sealed_blocks == s.sealed_blocks
            for j in range(r.sealed_blocks):
                for x, y in zip(a.cache.block(layer, i, h, j), b.cache.block(layer, i, h, j)):
                    assert np.array_equal(x.view(np.uint8), y.view(np.uint8)), (i, h, j)
            if not r.n_kept:
                continue
            rows = max(n - w.sink - w.local, 0) - 128 * r.sealed_blocks
            m = torch.arange(rows, device="cuda")
            for at, width in (("k_b_offset", r.n_kept), ("v_b_offset", 128)):
                assert torch.equal(a.cache.middle_rows(r, getattr(r, at), width, m),
                                   b.cache.middle_rows(s, getattr(s, at), width, m)), (i, h, at)
    for width in (32, 64, 96, 128):
        assert a.cache.pages(width) == b.cache.pages(width)


def _run(w, masks, fmt, rope, chunks, paged=False, own_positions=False, ragged=False, fused=False, ids=True):
    """Chunks of the given lengths enter twin caches, turned on the way and before."""
    total = sum(chunks)
    a, b = _twins(w, masks, total, fmt, paged)
    B, Hq, H = w.batch, w.num_q_heads, w.num_kv_heads
    rng = np.random.default_rng(7)
    special = len(a.is_special) > 0 and ids
    for x, n in enumerate(chunks):
        row = _draw(100 + x, B, n, Hq + 2 * H, 128)
        q, k, v = row[:, :, :Hq], row[:, :, Hq:Hq + H], row[:, :, Hq + H:]
        if not fused:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        lens = rng.integers(0, n + 1, B).astype(np.int32) if ragged else None
        if own_positions:
            pos = torch.from_numpy(a.cache.lengths(0)).cuda()[:, None] + torch.arange(n, device="cuda")[None]
            pos = pos.to(torch.int32)
            pos = (pos.expand(3, B, n) if rope.axes else pos).contiguous()
        else:
            pos = torch.from_numpy(rng.integers(-9, 70000, (*rope.axes, B, n)).astype(np.int32)).cuda()
        tid = torch.from_numpy(rng.integers(0, w.vocab, (B, n)).astype(np.int32)).cuda() if special else None
        qt, kt = rope.apply(q, k, pos)
        b.cache.append_chunk(0, kt, v, lens=lens, ids=tid)
        out = torch.full_like(qt, 3.0)
        got = a.cache.append_rope(0, rope, k, v, positions=None if own_positions else pos, q=q, q_out=out, lens=lens,
                                  ids=tid)
        assert got is out
        for i in range(B):
            m = n if lens is None else int(lens[i])
            assert torch.equal(out[i, :m], qt[i, :m]) and bool((out[i, m:] == 3.0).all())
    _same_caches(a, b)
    return a, b


@pytest.mark.parametrize("fmt", FORMATS, ids=NAMES)
@pytest.mark.parametrize("kind", ["plain", "part", "half-part", "axes", "axes-own"])
def test_chunks_of_full_heads(cuda, fmt, kind):
    w, masks = _workload(2, sink=4, local=64)
    _run(w, masks, fmt, _rope(kind), [3, 100, 260, 1, 129, 1, 7])


@pytest.mark.parametrize("fmt", FORMATS, ids=NAMES)
@pytest.mark.parametrize("own", [False, True], ids=["given", "own"])
def test_pages_and_ragged_chunks(cuda, fmt, own):
    w, masks = _workload(3, sink=0, local=33)
    _run(w, masks, fmt, _rope("axes" if own else "plain"), [140, 1, 300, 2, 1, 515], paged=True, own_positions=own,
         ragged=True, fused=True)


@pytest.mark.parametrize("fmt", FORMATS, ids=NAMES)
def test_every_policy(cuda, fmt):
    w, masks = _workload(2, policies=True, context=900, sink=4, local=40, local_only_window=24)
    _run(w, masks, fmt, _rope("half-part"), [50, 1, 1, 300, 1, 90], ragged=True, own_positions=True)


@pytest.mark.parametrize("fmt", FORMATS, ids=NAMES)
@pytest.mark.parametrize("paged", [False, True], ids=["flat", "paged"])
def test_single_tokens_through_a_seal(cuda, fmt, paged):
    """One token at a time, past the window and past a sealed block (or a page)."""
    w, masks = _workload(3, sink=2, local=20)
    _run(w, masks, fmt, _rope("plain"), [140] + [1] * 30, paged=paged, own_positions=True, fused=True)


def test_long_prompt_takes_wide_runs(cuda):
    """More tokens than 16 for each SM: four to a block."""
    w, masks = _workload(2, sink=16, local=512)
    _run(w, masks, lkb.KV_BF16, _rope("plain"), [2049, 5], fused=True, own_positions=True)
    _run(w, masks, lkb.KV_FP8_BLOCK, _rope("axes"), [2050], paged=True)


@pytest.mark.parametrize("fmt", FORMATS, ids=NAMES)
def test_one_token_forms_agree(cuda, fmt):
    """[B, heads, 128] and [B, 1, heads, 128]; without queries; step_rope is append_rope
    and decode."""
    w, masks = _workload(2, sink=2, local=20)
    a, b = _twins(w, masks, 200, fmt)
    c, _ = _twins(w, masks, 200, fmt)
    rope = _rope("plain")
    B, Hq, H = w.batch, w.num_q_heads, w.num_kv_heads
    for x in (a, b, c):
        x.cache.append_rope(0, rope, _draw(1, B, 145, H, 128), _draw(2, B, 145, H, 128))
    for t in range(12):
        q, k, v = _draw(10 + t, B, Hq, 128), _draw(40 + t, B, H, 128), _draw(70 + t, B, H, 128)
        pos = torch.tensor([5 * t, 1000 + t], dtype=torch.int32, device="cuda")
        qa = a.cache.append_rope(0, rope, k, v, positions=pos, q=q)
        assert qa.shape == (B, Hq, 128)
        o = a.cache.decode(0, qa)
        qb = b.cache.append_rope(0, rope, k[:, None], v[:, None], positions=pos[:, None], q=q[:, None])
        assert torch.equal(qb[:, 0], qa)
        assert torch.equal(c.cache.step_rope(0, rope, q, k, v, positions=pos), o)
    _same_caches(a, b)
    _same_caches(a, c)


def test_released_slots_and_many_sequences(cuda):
    """More sequences than one launch group takes, one of them released."""
    w = TINY.scaled(batch=300, num_q_heads=2, num_kv_heads=1)
    masks = S.masks_with_counts(w, (32,))
    a, b = _twins(w, masks, 80, lkb.KV_FP8_BLOCK)
    rope = _rope("plain")
    for x in (a, b):
        x.cache.append_chunk(0, _draw(1, 300, 70, 1, 128), _draw(2, 300, 70, 1, 128))
        x.cache.release(299)
        x.cache.release(3)
    for n in (1, 2, 1):
        q, k, v = _draw(3, 300, n, 2, 128), _draw(4, 300, n, 1, 128), _draw(5, 300, n, 1, 128)
        pos = torch.from_numpy(a.cache.lengths(0)).cuda()[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)
        qt, kt = rope.apply(q, k, pos.to(torch.int32).contiguous())
        b.cache.append_chunk(0, kt, v)
        out = torch.full_like(qt, 3.0)
        a.cache.append_rope(0, rope, k, v, q=q, q_out=out)
        off = torch.zeros(300, dtype=torch.bool, device="cuda")
        off[[3, 299]] = True
        assert torch.equal(out[~off], qt[~off]) and bool((out[off] == 3.0).all())
    _same_caches(a, b)


def test_in_place_and_strided_outputs(cuda):
    w, masks = _workload(2, sink=2, local=20)
    a, b = _twins(w, masks, 60, lkb.KV_BF16)
    rope = _rope("part")
    B, Hq, H = w.batch, w.num_q_heads, w.num_kv_heads
    for n in (9, 1):
        row = _draw(n, B, n, Hq + 2 * H, 128)
        before = row.clone()
        q, k, v = row[:, :, :Hq], row[:, :, Hq:Hq + H], row[:, :, Hq + H:]
        want = b.cache.append_rope(0, rope, k, v, q=q)
        a.cache.append_rope(0, rope, k, v, q=q, q_out=q)
        assert torch.equal(q, want) and torch.equal(row[:, :, Hq:], before[:, :, Hq:])
    _same_caches(a, b)


def test_captured_steps_advance_by_themselves(cuda):
    """Positions left to the cache: replays of one captured step are steps."""
    w, masks = _workload(2, sink=2, local=20)
    for fmt in (lkb.KV_BF16, lkb.KV_FP8_BLOCK):
        a, b = _twins(w, masks, 200, fmt)
        rope = _rope("plain")
        B, Hq, H = w.batch, w.num_q_heads, w.num_kv_heads
        q, k, v = _draw(1, B, Hq, 128), _draw(2, B, H, 128), _draw(3, B, H, 128)
        o = torch.zeros(B, Hq, 128, device="cuda")
        for x in (a, b):
            x.cache.append_rope(0, rope, _draw(4, B, 147, H, 128), _draw(5, B, 147, H, 128))
            x.cache.step_rope(0, rope, q, k, v, o=o)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            a.cache.step_rope(0, rope, q, k, v, o=o)
        for t in range(6):
            q.copy_(_draw(20 + t, B, Hq, 128))
            k.copy_(_draw(40 + t, B, H, 128))
            v.copy_(_draw(60 + t, B, H, 128))
            g.replay()
            assert torch.equal(o, b.cache.step_rope(0, rope, q, k, v)), (fmt, t)
        a.cache.check()
        b.cache.check()
        torch.cuda.synchronize()
        assert torch.equal(a.cache.buffer, b.cache.buffer)


def test_side_stream(cuda):
    w, masks = _workload(2, sink=2, local=20)
    a, b = _twins(w, masks, 300, lkb.KV_FP8_BLOCK)
    rope = _rope("axes")
    B, H = w.batch, w.num_kv_heads
    pos = torch.randint(0, 999, (3, B, 200), dtype=torch.int32, device="cuda")
    k, v = _draw(1, B, 200, H, 128), _draw(2, B, 200, H, 128)
    b.cache.append_rope(0, rope, k, v, positions=pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a.cache.append_rope(0, rope, k, v, positions=pos, stream=s)
    s.synchronize()
    _same_caches(a, b)


def test_refusals(cuda):
    w, masks = _workload(2, sink=2, local=20)
    a, = _twins(w, masks, 40, lkb.KV_BF16)[:1]
    rope = _rope("plain")
    B, Hq, H = w.batch, w.num_q_heads, w.num_kv_heads
    k = _draw(1, B, 41, H, 128)
    before = a.cache.buffer.clone()
    with pytest.raises(lkb.LeankError) as e:
        a.cache.append_rope(0, rope, k, k)
    assert e.value.status == lkb.LK_ERR_CAPACITY
    with pytest.raises(lkb.LeankError) as e:
        a.cache.append_rope(0, rope, k[:, :5].contiguous(), k[:, :5].contiguous(), lens=[6, 0])
    assert e.value.status == lkb.LK_ERR_ARG
    with pytest.raises(lkb.LeankError) as e:
        a.cache.append_rope(1, rope, k[:, :5].contiguous(), k[:, :5].contiguous())
    assert e.value.status == lkb.LK_ERR_ARG
    wide = _draw(2, B, 5, 2 * Hq, 128)
    with pytest.raises(lkb.LeankError) as e:                                 # in place, another stride
        a.cache.append_rope(0, rope, k[:, :5].contiguous(), k[:, :5].contiguous(), q=wide[:, :, :Hq],
                            q_out=wide.view(-1)[:B * 5 * Hq * 128].view(B, 5, Hq, 128))
    assert e.value.status == lkb.LK_ERR_ARG
    torch.cuda.synchronize()
    assert torch.equal(a.cache.buffer, before) and a.cache.length(0) == 0
    q = _draw(3, B, Hq, 128)
    a.cache.append_rope(0, rope, k[:, :40].contiguous(), k[:, :40].contiguous())
    with pytest.raises(lkb.LeankError) as e:
        a.cache.step_rope(0, rope, q, k[:, 0].contiguous(), k[:, 0].contiguous())
    assert e.value.status == lkb.LK_ERR_CAPACITY
    empty = a.cache.append_rope(0, rope, k[:, :0], k[:, :0], q=_draw(4, B, 0, Hq, 128))
    assert empty.shape == (B, 0, Hq, 128)
    a.cache.check()
