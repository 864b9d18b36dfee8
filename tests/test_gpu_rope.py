"""Rotary positions on the GPU against fp64.

Bound: each result is rounded once to bf16 (at most 2^-8 of its magnitude) from
fp32 arithmetic.  The cosine and sine are off by at most 2^-21 together with the
angle's last bits (a fraction of a turn in 24 bits is off by 2^-25 of half a
turn: pi 2^-25 of angle), the two products and their sum by 3 * 2^-24 of |x_a| + |x_b|."""
import numpy as np
import pytest
import torch

from decode_attention_pruned_gb300 import binding as lkb
from oracle import chunk as OC

pytestmark = pytest.mark.gpu

LAYOUT = {"half": lkb.ROPE_HALF, "interleaved": lkb.ROPE_INTERLEAVED}
SCALING = {"none": lkb.ROPE_SCALE_NONE, "linear": lkb.ROPE_SCALE_LINEAR, "ntk": lkb.ROPE_SCALE_NTK,
           "yarn": lkb.ROPE_SCALE_YARN, "bands": lkb.ROPE_SCALE_BANDS}


def _draw(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()


def _check(x, got, pos, freq, layout, mag=1.0):
    x64 = x.double().cpu().numpy()
    ref = OC.rope(x64, pos, freq, layout, mag)
    big = np.abs(x64)
    half = len(freq)
    a, b = (slice(0, half), slice(half, 2 * half)) if layout == "half" else \
        (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    both = np.zeros_like(big)
    both[..., a] = both[..., b] = big[..., a] + big[..., b]
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= 2.0 ** -8 * np.abs(ref) + mag * 2.0 ** -20 * both), float((err - 2.0 ** -8 * np.abs(ref)).max())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens, hq, hk, dim", [(1, 1, 1, 128), (1, 32, 8, 128), (3, 28, 4, 64), (64, 32, 8, 128),
                                                 (67, 5, 1, 16), (130, 8, 8, 96), (1025, 7, 1, 128), (5, 1, 0, 112),
                                                 (700, 40, 40, 128)])
def test_rope_matches_the_oracle(cuda, tokens, hq, hk, dim, layout):
    rng = np.random.default_rng(tokens)
    pos = rng.integers(0, 100000, tokens).astype(np.int32)
    q, k = _draw(1, tokens, hq, 128), _draw(2, tokens, hk, 128) if hk else None
    rope = lkb.Rope(rotary_dim=dim, base=1e6, layout=LAYOUT[layout])
    qo, ko = rope.apply(q, k, torch.from_numpy(pos).cuda())
    freq = OC.rope_frequencies(dim, 1e6)
    _check(q, qo, pos, freq, layout)
    if hk:
        _check(k, ko, pos, freq, layout)
    else:
        assert ko is None
    # channels past rotary_dim pass through bit for bit
    assert torch.equal(qo[..., dim:], q[..., dim:])


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn", "bands"])
def test_rope_far_positions_and_scalings(cuda, scaling):
    # positions whose fp32 angle would be off by a quarter of a turn, the
    # smallest, the largest and negative ones
    pos = np.array([0, 1, 2, 4095, 65535, 1 << 20, (1 << 24) + 1, (1 << 30) + 7, (1 << 31) - 1, -1, -70000, -(1 << 31)],
                   np.int64).astype(np.int32)
    x = _draw(4, len(pos), 4, 128)
    trained = 8192
    rope = lkb.Rope(base=5e5, scaling=SCALING[scaling], factor=8.0, trained_positions=trained)
    out, _ = rope.apply(x, None, torch.from_numpy(pos).cuda())
    f = OC.rope_frequencies(128, 5e5, scaling, 8.0 if scaling != "none" else 1.0, trained)
    mag = 0.1 * np.log(8.0) + 1.0 if scaling == "yarn" else 1.0
    near = np.abs(pos.astype(np.int64)) <= 1 << 24
    # the fp64 oracle's own angle keeps 2^-53 of p w <= 2^31: 2^-22, over the bound's 2^-20 share only past 2^24
    sel = torch.from_numpy(near).cuda()
    _check(x[sel], out[sel], pos[near], f, "half", mag)
    # farther: turn the position's high part exactly, with integers, as the definition says
    turns = [[(int(p) * int(w / (2 * np.pi) * 2.0 ** 64)) % (1 << 64) / 2.0 ** 64 for w in f] for p in pos]
    ang = 2 * np.pi * np.array(turns)[:, None, :]
    x64 = x.double().cpu().numpy()
    a, b = x64[..., :64], x64[..., 64:]
    ref = mag * np.concatenate([a * np.cos(ang) - b * np.sin(ang), b * np.cos(ang) + a * np.sin(ang)], -1)
    err = np.abs(out.double().cpu().numpy() - ref)
    # w / 2 pi is held to 2^-53 of itself on both sides (2^-54 of a turn at most, times 2^31 positions)
    assert np.all(err <= 2.0 ** -8 * np.abs(ref) + mag * 2.0 ** -19 * (np.abs(np.concatenate([a, a], -1)) +
                                                                       np.abs(np.concatenate([b, b], -1))))


def test_rope_options(cuda):
    pos = np.arange(40, dtype=np.int32) * 37
    x = _draw(5, 40, 2, 128)
    for scaling, low, high in (("yarn", 2.0, 16.0), ("bands", 0.5, 8.0)):
        rope = lkb.Rope(base=1e4, scaling=SCALING[scaling], factor=3.0, trained_positions=2048, low_turns=low,
                        high_turns=high, magnitude=1.25)
        out, _ = rope.apply(x, None, torch.from_numpy(pos).cuda())
        _check(x, out, pos, OC.rope_frequencies(128, 1e4, scaling, 3.0, 2048, low, high), "half", 1.25)


@pytest.mark.parametrize("dim, layout", [(128, "half"), (64, "half"), (128, "interleaved"), (32, "interleaved")])
def test_rope_in_place_on_fused_rows(cuda, dim, layout):
    """q and k inside one projection's rows, turned where they are; v and what
    lies past the rows stays as it was; the result is the dense one's."""
    B, n, hq, hk = 3, 9, 8, 2
    rows = _draw(6, B, n, hq + 2 * hk + 1, 128)
    before = rows.clone()
    q, k, rest = rows[:, :, :hq], rows[:, :, hq:hq + hk], rows[:, :, hq + hk:]
    pos = torch.arange(B * n, dtype=torch.int32, device="cuda").view(B, n) * 11
    rope = lkb.Rope(rotary_dim=dim, layout=LAYOUT[layout])
    dq, dk = rope.apply(before[:, :, :hq].contiguous(), before[:, :, hq:hq + hk].contiguous(), pos)
    qo, ko = rope.apply(q, k, pos, q_out=q, k_out=k)
    assert qo.data_ptr() == q.data_ptr() and torch.equal(q, dq) and torch.equal(k, dk)
    assert torch.equal(rest, before[:, :, hq + hk:])
    # positions turned back give the input again, up to the two roundings
    back, _ = rope.apply(q, None, -pos)
    x = before[:, :, :hq].float()
    assert float((back.float() - x).abs().max()) <= 2.0 ** -6 * float(x.abs().max())


def test_rope_refuses_wrong_tensors(cuda):
    rope = lkb.Rope()
    x, pos = _draw(1, 4, 2, 128), torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        rope.apply(x.float(), None, pos)
    with pytest.raises(ValueError):
        rope.apply(x[..., :64], None, pos)
    with pytest.raises(ValueError):
        rope.apply(x, None, pos.long())
    with pytest.raises(ValueError):
        rope.apply(x, None, pos[:3])
    with pytest.raises(ValueError):
        rope.apply(x.transpose(0, 1).contiguous().transpose(0, 1), None, pos)      # heads not dense
    with pytest.raises(ValueError):
        rope.apply(None, None, pos)
    uneven = _draw(2, 3, 5, 2, 128)[:, :4]                                          # batches further apart than tokens
    with pytest.raises(ValueError):
        rope.apply(uneven, None, torch.zeros(3, 4, dtype=torch.int32, device="cuda"))
    empty, _ = rope.apply(x[:0], None, pos[:0])
    assert empty.shape == (0, 2, 128)


def test_rope_side_stream_and_graph(cuda):
    rope = lkb.Rope()
    x, pos = _draw(7, 33, 4, 128), torch.arange(33, dtype=torch.int32, device="cuda")
    ref, _ = rope.apply(x, None, pos)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.zeros_like(x)
    s.wait_stream(torch.cuda.current_stream())
    rope.apply(x, None, pos, q_out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
    g = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(g):
        rope.apply(x, None, pos, q_out=out)
    pos += 5
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, rope.apply(x, None, pos)[0])
