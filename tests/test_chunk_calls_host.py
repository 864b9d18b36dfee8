"""The Python side of the chunk and rotary calls, without a GPU: stand-ins that
report a CUDA device carry the shapes and strides of CPU tensors, and a library
that must not be reached takes the place of the real one."""
import os
import re
import types

import pytest
import torch

from decode_attention_pruned_gb300 import binding as lkb

CUDA = torch.device("cuda", 0)


class OnGpu:
    """A CPU tensor that says it is on the GPU."""

    def __init__(self, t):
        self.t = t

    is_cuda, device = True, CUDA
    dtype = property(lambda self: self.t.dtype)
    shape = property(lambda self: self.t.shape)
    ndim = property(lambda self: self.t.ndim)

    def dim(self):
        return self.t.dim()

    def stride(self):
        return self.t.stride()

    def is_contiguous(self):
        return self.t.is_contiguous()

    def data_ptr(self):
        return self.t.data_ptr()


class NoCalls:
    """A library that no call may reach."""

    def __getattr__(self, name):
        raise AssertionError(f"{name} was reached")


def _rows(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _shared(B, n, H):
    """[B, n, H, 128] tensors whose tokens lie on one another: one row for all,
    for all of a sequence, for all sequences, or rows that overlap."""
    out = [_rows(1, 1, H, 128).expand(B, n, H, 128)]
    if n > 1:
        out += [_rows(B, 1, H, 128).expand(B, n, H, 128), _rows(B * n * H + H, 128).as_strided((B, n, H, 128),
                                                                                              (n * 128, 128, 128, 1))]
    if B > 1:
        out.append(_rows(1, n, H, 128).expand(B, n, H, 128))
    return [t for t in out if not t.is_contiguous()]


@pytest.mark.parametrize("B, n, H", [(1, 4, 8), (3, 1, 8), (4, 5, 2), (2, 2, 2)])
def test_tokens_that_share_rows_are_refused(B, n, H):
    cases = _shared(B, n, H)
    assert cases
    for t in cases:
        with pytest.raises(ValueError):
            lkb._token_stride(OnGpu(t), H, (B, n), "k")


def test_spaced_tokens_are_taken():
    stride = lkb._token_stride
    assert stride(OnGpu(_rows(3, 5, 2, 128)), 2, (3, 5), "k") == 256
    rows = _rows(3, 5, 7, 128)
    assert stride(OnGpu(rows[:, :, 1:3]), 2, (3, 5), "k") == 7 * 128
    assert stride(OnGpu(rows[:1, :, 1:3]), 2, (1, 5), "k") == 7 * 128
    assert stride(OnGpu(rows[:, :1, 1:3]), 2, (3, 1), "k") == 5 * 7 * 128
    assert stride(OnGpu(rows[:1, :1, 1:3]), 2, (1, 1), "k") == 2 * 128          # one token: nothing to step over
    # sizes of one may have any stride
    one = _rows(1, 2, 128).expand(1, 2, 128).unsqueeze(0)
    assert stride(OnGpu(one), 2, (1, 1), "k") == 2 * 128


def _cache(B, Hq, H):
    """A cache's Python side only."""
    c = object.__new__(lkb.Cache)
    c.plan = types.SimpleNamespace(num_q_heads=Hq, num_kv_heads=H)
    c.batch, c.buffer, c._h = B, OnGpu(torch.zeros(1)), None
    return c


@pytest.mark.parametrize("B, n", [(3, 1), (2, 4)])
def test_chunk_calls_refuse_shared_rows(monkeypatch, B, n):
    monkeypatch.setattr(lkb, "_lib", NoCalls())
    c = _cache(B, 4, 2)
    q, k = OnGpu(_rows(B, n, 4, 128)), OnGpu(_rows(B, n, 2, 128))
    for bad in map(OnGpu, _shared(B, n, 2)):
        for call in (lambda: c.append_chunk(0, bad, k), lambda: c.append_chunk(0, k, bad),
                     lambda: c.chunk_attn(0, q, bad, k), lambda: c.extend(0, q, k, bad)):
            with pytest.raises(ValueError):
                call()
    for bad in map(OnGpu, _shared(B, n, 4)):
        with pytest.raises(ValueError):
            c.chunk_attn(0, bad, k, k)


def test_rope_refuses_shared_rows(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    rope = object.__new__(lkb.Rope)
    rope._h = None
    monkeypatch.setattr(lkb, "_lib", NoCalls())
    x, pos = OnGpu(_rows(5, 8, 128)), OnGpu(torch.zeros(5, dtype=torch.int32))
    bad = OnGpu(_rows(1, 8, 128).expand(5, 8, 128))
    for call in (lambda: rope.apply(bad, None, pos, q_out=x), lambda: rope.apply(None, bad, pos, k_out=x),
                 lambda: rope.apply(x, None, pos, q_out=bad), lambda: rope.apply(None, x, pos, k_out=bad),
                 lambda: rope.apply(bad, None, pos, q_out=bad)):
        with pytest.raises(ValueError):
            call()


class Stream:
    cuda_stream = 0x5150


class Allocations:
    """Stands in for torch.empty and torch.cuda.stream: which stream was current
    when each tensor was made."""

    def __init__(self, monkeypatch):
        self.current, self.made = None, []
        real = torch.empty
        outer = self

        class On:
            def __init__(self, stream):
                self.stream = stream

            def __enter__(self):
                self.before, outer.current = outer.current, self.stream

            def __exit__(self, *_):
                outer.current = self.before

        def empty(*shape, dtype=None, device=None):
            self.made.append(self.current)
            return OnGpu(real(*shape, dtype=dtype))

        monkeypatch.setattr(torch, "empty", empty)
        monkeypatch.setattr(torch.cuda, "stream", On)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


class AllOk:
    def __getattr__(self, name):
        return lambda *a: lkb.LK_OK


@pytest.mark.parametrize("given", [False, True], ids=["current", "given"])
def test_new_tensors_belong_to_the_stream_of_the_call(monkeypatch, given):
    """What a call makes is used on the call's stream; made on another one, it
    could still be in use there."""
    made = Allocations(monkeypatch)
    monkeypatch.setattr(lkb, "_lib", AllOk())
    monkeypatch.setattr(lkb, "load", lambda *a, **k: lkb._lib)
    monkeypatch.setattr(lkb, "_stream", lambda stream=None: None)
    monkeypatch.setattr(OnGpu, "numel", lambda self: 1, raising=False)
    s = Stream() if given else None
    c = _cache(2, 4, 2)
    c.workspace, c.device, c.plan._h = OnGpu(torch.zeros(1)), CUDA, None
    c._chunk_tokens, c._chunk_workspaces = 0, []
    q, k = OnGpu(_rows(2, 3, 4, 128)), OnGpu(_rows(2, 3, 2, 128))
    q1, k1 = OnGpu(_rows(2, 4, 128)), OnGpu(_rows(2, 2, 128))
    ql, kl = OnGpu(_rows(1, 2, 4, 128)), OnGpu(_rows(1, 2, 2, 128))
    rope = object.__new__(lkb.Rope)
    rope._h = None
    plan = types.SimpleNamespace(_h=None, cache_bytes=lambda *a: 8, workspace_bytes=lambda *a: 8)
    alpha = OnGpu(torch.zeros(1, 2, 128))
    for n, call in ((2, lambda: c.chunk_attn(0, q, k, k, stream=s)), (1, lambda: c.extend(0, q, k, k, stream=s)),
                    (2, lambda: rope.apply(q1, k1, OnGpu(torch.zeros(2, dtype=torch.int32)), stream=s)),
                    (1, lambda: c.decode(0, q1, stream=s)), (1, lambda: c.step(0, q1, k1, k1, stream=s)),
                    (1, lambda: c.decode_layers(0, ql, stream=s)), (1, lambda: c.step_layers(0, ql, kl, kl, stream=s)),
                    (1, lambda: lkb.build_masks(alpha, 50.0, stream=s)),
                    (2, lambda: lkb.Cache(plan, 1, 8, stream=s))):
        made.made.clear()
        call()
        assert made.made == [s] * n


@pytest.mark.parametrize("has_raw", [True, False])
def test_current_stream_with_and_without_the_short_way(monkeypatch, has_raw):
    """The short way to the current stream's handle is torch's own affair: without
    it the public one gives the same."""
    if has_raw:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x5150 + device, raising=False)
    else:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream())
    assert lkb._stream().value == 0x5150
    assert lkb._stream(Stream()).value == 0x5150


def test_every_tensor_core_helper_is_used():
    csrc = os.path.join(os.path.dirname(lkb.__file__), "csrc")
    text = {f: open(os.path.join(csrc, f)).read() for f in os.listdir(csrc)}
    names = re.findall(r"__forceinline__ \w+ (\w+)\(", text["lk_tensor.cuh"])
    assert len(names) > 10
    for name in names:
        assert sum(len(re.findall(rf"\b{name}\b", t)) for t in text.values()) > 1, name


def test_shared_arrays_have_the_alignment_of_their_reads():
    """A __shared__ array of a smaller type is not read through a pointer to float4
    or uint4: its place is aligned for its own type only."""
    csrc = os.path.join(os.path.dirname(lkb.__file__), "csrc")
    for f in ("lk_rope.cu", "lk_chunk.cu", "lk_chunk_append.cu"):
        text = open(os.path.join(csrc, f)).read()
        for kind, name in re.findall(r"__shared__ (\w+) (\w+)\[", text):
            wide = re.findall(rf"reinterpret_cast<(?:const )?(\w+4)\*>\(&?{name}\b", text)
            assert kind.endswith("4") or not wide, (f, name, wide)
