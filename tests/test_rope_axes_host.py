"""Rotary positions on several axes: refusals, the structure's layout, and pins of
the fp64 oracle.  No GPU."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from decode_attention_pruned_gb300 import binding as lkb
from oracle import chunk as OC

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("bad, status", [
    (dict(axes=[]), lkb.LK_ERR_UNSUPPORTED),
    (dict(axes=[16, 16, 16, 8, 8]), lkb.LK_ERR_UNSUPPORTED),
    (dict(axes=[16, 24, 23]), lkb.LK_ERR_ARG),                          # 63 of 64 pairs
    (dict(axes=[16, 24, 25]), lkb.LK_ERR_ARG),
    (dict(axes=[0, 32, 32]), lkb.LK_ERR_ARG),
    (dict(axes=[-8, 40, 32]), lkb.LK_ERR_ARG),
    (dict(axes=[2 ** 31 - 1, 2 ** 31 - 1, 66]), lkb.LK_ERR_ARG),
    (dict(axes=[24, 20, 20], axis_order=2), lkb.LK_ERR_ARG),
    (dict(axes=[24, 20, 20], axis_order=-1), lkb.LK_ERR_ARG),
    (dict(axes=[24, 20, 20], axis_spectrum=2), lkb.LK_ERR_ARG),
    (dict(axes=[16, 24, 24], axis_order=lkb.ROPE_AXES_CYCLIC), lkb.LK_ERR_ARG),    # 24 of every third of 64
    (dict(axes=[1, 63], axis_order=lkb.ROPE_AXES_CYCLIC), lkb.LK_ERR_ARG),
    (dict(axes=[24, 20, 20], rotary_dim=24), lkb.LK_ERR_UNSUPPORTED),
    (dict(axes=[24, 20, 20], base=1.0), lkb.LK_ERR_ARG),
    (dict(axes=[24, 20, 20], scaling=lkb.ROPE_SCALE_YARN, factor=2.0), lkb.LK_ERR_ARG),
])
def test_refusals(lib, bad, status):
    with pytest.raises(lkb.LeankError) as e:
        lkb.Rope(**bad)
    assert e.value.status == status


def test_reserved_and_null(lib):
    desc = lkb.RopeDesc(128, 0, 0, 0, 1e4, 1.0, 0.0, 0.0, 0.0)
    out = ctypes.c_void_p(7)
    axes = lkb.RopeAxes(3, (ctypes.c_int32 * 4)(24, 20, 20, 0), 0, 0, 1)
    assert lib.lk_build_rope_axes(ctypes.byref(desc), ctypes.byref(axes), ctypes.byref(out)) == lkb.LK_ERR_ARG
    assert not out.value
    assert lib.lk_build_rope_axes(ctypes.byref(desc), None, ctypes.byref(out)) == lkb.LK_ERR_ARG
    assert lib.lk_build_rope_axes(None, ctypes.byref(axes), ctypes.byref(out)) == lkb.LK_ERR_ARG
    axes.reserved = 0
    assert lib.lk_build_rope_axes(ctypes.byref(desc), ctypes.byref(axes), None) == lkb.LK_ERR_ARG


@pytest.mark.parametrize("kw", [
    dict(axes=[64]), dict(axes=[16, 24, 24]), dict(axes=[1, 1, 1, 61]), dict(axes=[16, 16, 16, 16]),
    dict(axes=[24, 20, 20], axis_order=lkb.ROPE_AXES_CYCLIC), dict(axes=[32, 32], axis_order=lkb.ROPE_AXES_CYCLIC),
    dict(axes=[16, 16, 16, 16], axis_order=lkb.ROPE_AXES_CYCLIC),
    dict(axes=[2, 3, 3], rotary_dim=16, axis_spectrum=lkb.ROPE_SPECTRUM_OWN),
    dict(axes=[1, 31, 32], axis_spectrum=lkb.ROPE_SPECTRUM_OWN, scaling=lkb.ROPE_SCALE_NTK, factor=4.0),
])
def test_accepted(lib, kw):
    assert lkb.Rope(**kw)._h.value


def test_structure_matches_the_header(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no host C compiler")
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    fields = [n for n, _ in lkb.RopeAxes._fields_]
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "leank.h"\nint main(void) {\n'
                   'printf("%zu", sizeof(lk_rope_axes));\n'
                   + "".join(f'printf(" %zu", offsetof(lk_rope_axes, {n}));\n' for n in fields)
                   + 'printf(" %d %d %d %d", LK_ROPE_AXES_BLOCKS, LK_ROPE_AXES_CYCLIC, LK_ROPE_SPECTRUM_SHARED, '
                     'LK_ROPE_SPECTRUM_OWN);\nreturn 0;\n}\n')
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", str(exe)], check=True)
    got = list(map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()))
    assert got == [ctypes.sizeof(lkb.RopeAxes), *(getattr(lkb.RopeAxes, n).offset for n in fields),
                   lkb.ROPE_AXES_BLOCKS, lkb.ROPE_AXES_CYCLIC, lkb.ROPE_SPECTRUM_SHARED, lkb.ROPE_SPECTRUM_OWN]


def test_oracle_axes():
    """The axes of the pairs, by hand; equal positions are one axis; own spectra
    start anew."""
    w, axis = OC.rope_axes(16, 1e4, (2, 3, 3))
    assert axis.tolist() == [0, 0, 1, 1, 1, 2, 2, 2]
    assert np.array_equal(w, OC.rope_frequencies(16, 1e4))
    w, axis = OC.rope_axes(16, 1e4, (4, 2, 2), "cyclic")
    assert axis.tolist() == [0, 1, 2, 0, 1, 2, 0, 0]
    w, axis = OC.rope_axes(16, 1e4, (2, 3, 3), "blocks", "own")
    assert np.allclose(w, [1, 1e-2, 1, 1e4 ** (-1 / 3), 1e4 ** (-2 / 3), 1, 1e4 ** (-1 / 3), 1e4 ** (-2 / 3)], rtol=1e-14)
    x = np.random.default_rng(0).standard_normal((5, 2, 16))
    pos = np.array([0, 3, -2, 70000, 11])
    w, axis = OC.rope_axes(16, 1e4, (4, 2, 2), "cyclic")
    for layout in ("half", "interleaved"):
        many, one = OC.rope_on_axes(x, np.stack([pos] * 3), w, axis, layout, 1.5), OC.rope(x, pos, w, layout, 1.5)
        assert np.allclose(many, one, atol=1e-12)
