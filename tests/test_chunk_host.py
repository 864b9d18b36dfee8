"""Chunk and rotary-position calls: host checks that need no GPU, and pins of
their fp64 oracle."""
import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest

from decode_attention_pruned_gb300 import binding as lkb
from decode_attention_pruned_gb300 import synth as S
from oracle import attention as OA
from oracle import chunk as OC

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ----------------------------------------------------------------- host checks

@pytest.mark.parametrize("bad, status", [
    (dict(rotary_dim=0), lkb.LK_ERR_UNSUPPORTED),
    (dict(rotary_dim=24), lkb.LK_ERR_UNSUPPORTED),
    (dict(rotary_dim=144), lkb.LK_ERR_UNSUPPORTED),
    (dict(layout=2), lkb.LK_ERR_ARG),
    (dict(scaling=5), lkb.LK_ERR_ARG),
    (dict(scaling=-1), lkb.LK_ERR_ARG),
    (dict(base=1.0), lkb.LK_ERR_ARG),
    (dict(base=math.nan), lkb.LK_ERR_ARG),
    (dict(base=math.inf), lkb.LK_ERR_ARG),
    (dict(scaling=lkb.ROPE_SCALE_LINEAR, factor=0.5), lkb.LK_ERR_ARG),
    (dict(scaling=lkb.ROPE_SCALE_YARN, factor=math.nan, trained_positions=4096), lkb.LK_ERR_ARG),
    (dict(scaling=lkb.ROPE_SCALE_YARN, factor=2.0), lkb.LK_ERR_ARG),                          # no trained length
    (dict(scaling=lkb.ROPE_SCALE_BANDS, factor=2.0, trained_positions=8, low_turns=4.0), lkb.LK_ERR_ARG),
    (dict(scaling=lkb.ROPE_SCALE_BANDS, factor=2.0, trained_positions=8, low_turns=-1.0), lkb.LK_ERR_ARG),
    (dict(magnitude=-1.0), lkb.LK_ERR_ARG),
])
def test_rope_refuses(lib, bad, status):
    with pytest.raises(lkb.LeankError) as e:
        lkb.Rope(**bad)
    assert e.value.status == status


def test_rope_apply_refuses_before_any_launch(lib):
    rope = lkb.Rope()
    a = 1 << 20                                     # 16-byte aligned, never dereferenced

    def call(q=a, qs=0, k=a, ks=0, pos=a, tokens=4, hq=8, hk=2, qo=a, qos=0, ko=a, kos=0, h=rope._h):
        return lib.lk_rope_apply(h, q, qs, k, ks, pos, tokens, hq, hk, qo, qos, ko, kos, None)

    assert call(h=None) == lkb.LK_ERR_ARG
    assert call(q=None) == lkb.LK_ERR_ARG
    assert call(ko=None) == lkb.LK_ERR_ARG
    assert call(pos=None) == lkb.LK_ERR_ARG
    assert call(tokens=-1) == lkb.LK_ERR_ARG
    assert call(tokens=1 << 31) == lkb.LK_ERR_ARG
    assert call(hq=-1) == lkb.LK_ERR_ARG
    assert call(hq=1 << 20) == lkb.LK_ERR_ARG
    assert call(qs=8 * 128 - 8) == lkb.LK_ERR_ARG    # tokens would overlap
    assert call(qs=8 * 128 + 4, qos=8 * 128 + 4) == lkb.LK_ERR_ARG
    assert call(qs=8 * 128 + 8) == lkb.LK_ERR_ARG    # in place with another stride
    assert call(q=a + 2, qo=a + 2) == lkb.LK_ERR_ALIGN
    assert call(pos=a + 1) == lkb.LK_ERR_ALIGN
    assert call(tokens=0) == lkb.LK_OK
    assert call(hq=0, hk=0) == lkb.LK_OK


def test_chunk_calls_refuse_null(lib):
    c = lkb.Chunk()
    n = ctypes.c_size_t()
    assert lib.lk_chunk_attn(None, 0, ctypes.byref(c), None, None, 0, None) == lkb.LK_ERR_ARG
    assert lib.lk_append_chunk(None, 0, ctypes.byref(c), None) == lkb.LK_ERR_ARG
    assert lib.lk_extend(None, 0, ctypes.byref(c), None, None, 0, None) == lkb.LK_ERR_ARG
    assert lib.lk_chunk_workspace_bytes(None, 1, 1, ctypes.byref(n)) == lkb.LK_ERR_ARG


def test_chunk_workspace_bytes(lib):
    w = S.WORKLOADS[1]
    plan = lkb.Plan.for_workload(w, S.masks_with_counts(w, [32] * 8), S.make_policies(w))
    n = ctypes.c_size_t()
    sizes = []
    for tokens in (0, 1, 4, 64, 4096):
        assert lib.lk_chunk_workspace_bytes(plan._h, 2, tokens, ctypes.byref(n)) == lkb.LK_OK
        sizes.append(n.value)
    assert sizes == sorted(sizes) and sizes[-1] < 1 << 28      # longer chunks never need less, none needs much
    assert lib.lk_chunk_workspace_bytes(plan._h, 0, 1, ctypes.byref(n)) == lkb.LK_ERR_ARG
    assert lib.lk_chunk_workspace_bytes(plan._h, 1, -1, ctypes.byref(n)) == lkb.LK_ERR_ARG


_PROBE = r"""
#include <stddef.h>
#include <stdio.h>
#include "leank.h"
#define SIZE(T) printf(#T " %zu\n", sizeof(T));
#define OFF(T, m) printf(#T "." #m " %zu\n", offsetof(T, m));
#define VAL(e) printf(#e " %d\n", (int)(e));
int main(void) {
  SIZE(lk_chunk) SIZE(lk_rope_desc)
  OFF(lk_chunk, q) OFF(lk_chunk, k) OFF(lk_chunk, v) OFF(lk_chunk, ids) OFF(lk_chunk, lens)
  OFF(lk_chunk, q_stride) OFF(lk_chunk, k_stride) OFF(lk_chunk, v_stride) OFF(lk_chunk, n_max)
  OFF(lk_chunk, reserved)
  OFF(lk_rope_desc, rotary_dim) OFF(lk_rope_desc, layout) OFF(lk_rope_desc, scaling)
  OFF(lk_rope_desc, trained_positions) OFF(lk_rope_desc, base) OFF(lk_rope_desc, factor)
  OFF(lk_rope_desc, low_turns) OFF(lk_rope_desc, high_turns) OFF(lk_rope_desc, magnitude)
  VAL(LK_ROPE_HALF) VAL(LK_ROPE_INTERLEAVED) VAL(LK_ROPE_SCALE_NONE) VAL(LK_ROPE_SCALE_LINEAR)
  VAL(LK_ROPE_SCALE_NTK) VAL(LK_ROPE_SCALE_YARN) VAL(LK_ROPE_SCALE_BANDS)
  return 0;
}
"""


def test_structs_match_the_header(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no host C compiler")
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text(_PROBE)
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()
    got = {k: int(v) for k, v in (line.rsplit(" ", 1) for line in out)}
    for cname, ct in {"lk_chunk": lkb.Chunk, "lk_rope_desc": lkb.RopeDesc}.items():
        assert ctypes.sizeof(ct) == got[cname]
        for field, _ in ct._fields_:
            assert getattr(ct, field).offset == got[f"{cname}.{field}"], (cname, field)
    for name in [k for k in got if k.startswith("LK_")]:
        assert getattr(lkb, name[3:]) == got[name], name


# ------------------------------------------------------------------ oracle pins

def test_chunk_oracle_is_one_masked_softmax():
    """Every query at once from explicit masks equals the step-by-step form."""
    r = np.random.default_rng(5)
    N, n, G, S_, W, Wl = 23, 19, 2, 3, 8, 5
    K, V, q = r.standard_normal((N + n, 128)), r.standard_normal((N + n, 128)), r.standard_normal((n, G, 128))
    flags = r.random(N + n) < 0.2
    kept = np.sort(r.choice(128, 32, replace=False))
    beta = np.zeros(128)
    beta[kept] = 1
    p, t = N + np.arange(n)[:, None], np.arange(N + n)[None]
    near = (t < S_) | (p - t < W)
    for pol, kp, see, whole in ((0, kept, t <= p, near), (0, kept[:0], (t <= p) & near, near | True),
                                (1, kept[:0], (t <= p) & (p - t < Wl), near | True),
                                (2, kept[:0], (t <= p) & flags[None], near | True)):
        for g in range(G):
            s = np.where(whole, q[:, g] @ K.T, (q[:, g] * beta) @ K.T) / math.sqrt(128)
            e = np.where(see, np.exp(s), 0)
            ref = e @ V / np.maximum(e.sum(1, keepdims=True), 1e-300)
            got = OC.chunk_head(q, K, V, pol, kp, N, S_, W, Wl, flags)[:, g]
            assert np.abs(got - ref).max() < 1e-12


def test_chunk_oracle_sees_nothing():
    q = np.ones((2, 1, 128))
    K = V = np.ones((2, 128))
    assert not OC.chunk_head(q, K, V, OA.SPECIAL, [], 0, 4, 8, 0, np.zeros(2, bool)).any()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_oracle(layout):
    r = np.random.default_rng(3)
    w = OC.rope_frequencies(64, 1e4)
    assert w[0] == 1.0 and w[-1] == pytest.approx(1e4 ** (-62 / 64))
    x, y = r.standard_normal((2, 1, 1, 128))
    at = lambda v, p: OC.rope(v, [p], w, layout)[0, 0]  # noqa: E731
    assert np.array_equal(at(x, 0), x[0, 0]) and np.array_equal(at(x, 9)[64:], x[0, 0, 64:])
    assert np.linalg.norm(at(x, 7)) == pytest.approx(np.linalg.norm(x))
    # scores depend on the distance alone
    assert at(x, 11) @ at(y, 4) == pytest.approx(at(x, 1007) @ at(y, 1000))
    # one pair by hand: position 1, angle w_1
    a, b = (1, 33) if layout == "half" else (2, 3)
    z = complex(x[0, 0, a], x[0, 0, b]) * complex(math.cos(w[1]), math.sin(w[1]))
    assert at(x, 1)[a] == pytest.approx(z.real) and at(x, 1)[b] == pytest.approx(z.imag)


def test_rope_frequencies_stretch_only_the_slow_pairs():
    w = OC.rope_frequencies(128, 5e5)
    for scaling in ("yarn", "bands"):
        v = OC.rope_frequencies(128, 5e5, scaling, 8.0, 8192)
        assert v[0] == w[0] and v[-1] == pytest.approx(w[-1] / 8)
        assert np.all(np.diff(v) < 0) and np.all(v <= w * (1 + 1e-12)) and np.all(v >= w / 8 * (1 - 1e-12))
    assert np.allclose(OC.rope_frequencies(128, 5e5, "linear", 4.0), w / 4)
    n = OC.rope_frequencies(128, 5e5, "ntk", 4.0)
    assert n[0] == 1.0 and n[-1] == pytest.approx(w[-1] / 4)       # the last pair is stretched by the factor
