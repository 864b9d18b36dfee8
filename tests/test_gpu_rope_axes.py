"""Rotary positions on several axes on the GPU against fp64.

Bound: as for one axis.  Each result is rounded once to bf16 (2^-8 of its magnitude)
from fp32 arithmetic; cosine and sine are off by at most 2^-21 together with the
angle's last bits, the two products and their sum by 3 * 2^-24 of |x_a| + |x_b|."""
import numpy as np
import pytest
import torch

from decode_attention_pruned_gb300 import binding as lkb
from oracle import chunk as OC

pytestmark = pytest.mark.gpu

LAYOUT = {"half": lkb.ROPE_HALF, "interleaved": lkb.ROPE_INTERLEAVED}
ORDER = {"blocks": lkb.ROPE_AXES_BLOCKS, "cyclic": lkb.ROPE_AXES_CYCLIC}
SPECTRUM = {"shared": lkb.ROPE_SPECTRUM_SHARED, "own": lkb.ROPE_SPECTRUM_OWN}
SCALING = {"none": lkb.ROPE_SCALE_NONE, "linear": lkb.ROPE_SCALE_LINEAR, "ntk": lkb.ROPE_SCALE_NTK,
           "yarn": lkb.ROPE_SCALE_YARN, "bands": lkb.ROPE_SCALE_BANDS}


def _draw(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def _check(x, got, pos, freq, axis, layout, mag=1.0):
    x64 = x.double().cpu().numpy()
    ref = OC.rope_on_axes(x64, pos, freq, axis, layout, mag)
    half = len(freq)
    a, b = (slice(0, half), slice(half, 2 * half)) if layout == "half" else \
        (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    both = np.zeros_like(x64)
    both[..., a] = both[..., b] = np.abs(x64[..., a]) + np.abs(x64[..., b])
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= 2.0 ** -8 * np.abs(ref) + mag * 2.0 ** -20 * both)


CASES = [((16, 24, 24), "blocks", "shared"), ((24, 20, 20), "cyclic", "shared"), ((22, 21, 21), "blocks", "own"),
         ((24, 20, 20), "cyclic", "own"), ((32, 32), "blocks", "own"), ((16, 16, 16, 16), "cyclic", "shared"),
         ((64,), "blocks", "shared")]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("pairs, order, spectrum", CASES)
@pytest.mark.parametrize("tokens, hq, hk", [(1, 4, 1), (67, 7, 1), (2500, 3, 2)])
def test_matches_the_oracle(cuda, tokens, hq, hk, pairs, order, spectrum, layout):
    rng = np.random.default_rng(tokens)
    pos = rng.integers(-50, 100000, (len(pairs), tokens)).astype(np.int32)
    q, k = _draw(1, tokens, hq, 128), _draw(2, tokens, hk, 128)
    rope = lkb.Rope(base=1e6, layout=LAYOUT[layout], axes=pairs, axis_order=ORDER[order],
                    axis_spectrum=SPECTRUM[spectrum])
    qo, ko = rope.apply(q, k, torch.from_numpy(pos).cuda())
    freq, axis = OC.rope_axes(128, 1e6, pairs, order, spectrum)
    _check(q, qo, pos, freq, axis, layout)
    _check(k, ko, pos, freq, axis, layout)


@pytest.mark.parametrize("spectrum", ["shared", "own"])
@pytest.mark.parametrize("scaling", list(SCALING))
def test_scalings_on_part_of_the_head(cuda, scaling, spectrum):
    pairs, dim = (8, 12, 12), 64
    pos = np.random.default_rng(3).integers(0, 1 << 20, (3, 40)).astype(np.int32)
    x = _draw(4, 40, 2, 128)
    rope = lkb.Rope(rotary_dim=dim, base=5e5, scaling=SCALING[scaling], factor=8.0, trained_positions=8192, axes=pairs,
                    axis_spectrum=SPECTRUM[spectrum])
    out, _ = rope.apply(x, None, torch.from_numpy(pos).cuda())
    f = 8.0 if scaling != "none" else 1.0
    freq, axis = OC.rope_axes(dim, 5e5, pairs, "blocks", spectrum, scaling, f, 8192)
    _check(x, out, pos, freq, axis, "half", 0.1 * np.log(8.0) + 1.0 if scaling == "yarn" else 1.0)
    assert torch.equal(out[..., dim:], x[..., dim:])


def test_text_turns_as_without_axes(cuda):
    """Equal positions on every axis give, but for the last bits of the angle, what
    one axis gives; one axis gives exactly that."""
    pos = torch.arange(300, dtype=torch.int32, device="cuda") * 37
    x = _draw(5, 300, 4, 128)
    plain, _ = lkb.Rope(base=1e6).apply(x, None, pos)
    one, _ = lkb.Rope(base=1e6, axes=[64]).apply(x, None, pos[None])
    assert torch.equal(plain, one)
    many, _ = lkb.Rope(base=1e6, axes=[24, 20, 20], axis_order=lkb.ROPE_AXES_CYCLIC).apply(
        x, None, pos.expand(3, 300).contiguous())
    assert float((many != plain).float().mean()) < 1e-3
    assert float((many.float() - plain.float()).abs().max()) <= 2.0 ** -7 * float(plain.float().abs().max())


def test_fused_rows_in_place_and_batches(cuda):
    B, n, hq, hk = 3, 9, 8, 2
    rows = _draw(6, B, n, hq + 2 * hk, 128)
    before = rows.clone()
    q, k, v = rows[:, :, :hq], rows[:, :, hq:hq + hk], rows[:, :, hq + hk:]
    pos = torch.randint(0, 999, (3, B, n), dtype=torch.int32, device="cuda")
    rope = lkb.Rope(axes=[16, 24, 24])
    dq, dk = rope.apply(q.contiguous(), k.contiguous(), pos)
    rope.apply(q, k, pos, q_out=q, k_out=k)
    assert torch.equal(q, dq) and torch.equal(k, dk) and torch.equal(v, before[:, :, hq + hk:])


def test_refuses_wrong_positions(cuda):
    rope, x = lkb.Rope(axes=[16, 24, 24]), _draw(1, 4, 2, 128)
    for shape in ((4,), (2, 4), (3, 5), (4, 3)):
        with pytest.raises(ValueError):
            rope.apply(x, None, torch.zeros(shape, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        rope.apply(x, None, torch.zeros(4, 3, dtype=torch.int32, device="cuda").t())
    empty, _ = rope.apply(x[:0], None, torch.zeros(3, 0, dtype=torch.int32, device="cuda"))
    assert empty.shape == (0, 2, 128)


def test_side_stream_and_graph(cuda):
    rope = lkb.Rope(axes=[24, 20, 20], axis_order=lkb.ROPE_AXES_CYCLIC)
    x, pos = _draw(7, 33, 4, 128), torch.randint(0, 500, (3, 33), dtype=torch.int32, device="cuda")
    ref, _ = rope.apply(x, None, pos)
    s, out = torch.cuda.Stream(), torch.zeros_like(x)
    s.wait_stream(torch.cuda.current_stream())
    rope.apply(x, None, pos, q_out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rope.apply(x, None, pos, q_out=out)
    pos += 5
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, rope.apply(x, None, pos)[0])
