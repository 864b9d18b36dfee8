"""Rotary positions on several axes, the append that turns keys on their way
into the cache, and attention over a cache whose middle is held in 8 bits with a
scale for each block of tokens and head: the cases they are measured on, in
plain form and through the package.

The three follow one another in a serving program.  A token of an image or a
video has a position on each of several axes, and its q and k turn by all of
them (``Rope(axes=...)``); a decode step or a prompt enters the cache with its
keys turned on the way (``Cache.append_rope``), which seals complete blocks of
the middle; and decode steps and chunks attend over the sealed blocks
(``Cache.decode``, ``Cache.chunk_attn`` of a cache with ``KV_FP8_BLOCK``).

Rotary positions: pair i of a head turns by magnitude * e^(i p_a w_i), a the
pair's axis, p_a the token's position on it.  The pairs go to the axes in runs
("blocks") or in turn ("cyclic": axis a >= 1 takes its pairs from i mod A = a, the
rest are axis 0's); w_i counts the pairs of the whole head ("shared") or of
their axis alone ("own").

Sealed blocks: 128 tokens of the middle of one kv head; the keys' scale is
max(largest magnitude / 448, 2^-64) over the 128 tokens and the kept channels,
the values' the same over their 128 channels; codes are x / scale in e4m3.

A query at position p sees of the token at position t <= p, per kv head with k
kept channels: q.k / sqrt(128) over all channels where t < S or p - t < W, else
over the kept channels, else (k = 0) nothing; one softmax over it.

A case is a dict of plain values:
  op "axes"    tokens, Hq, Hkv, dim, layout, sections (pairs of each axis),
               order, spectrum, scaling, factor, trained, base, span (positions
               drawn below it), frame (h x w patches of one frame; "": text)
  op "append"  B sequences of n tokens that enter empty slots, `step` at a
               time; heads (kept channels), S, W, ragged, paged, kv: bf16 |
               fp8_block; dim, layout, sections ("": one axis, the tokens' own
               positions); fused (q | k | v are one row per token); then a chunk
               of `verify` tokens attends over what the slots hold
  op "decode"  B sequences of up to N tokens, one query each
  op "chunk"   the same with n new tokens each
"""
import math

import torch

own = False

D = 128


def listed():
    return [
        # one decode step of 64 sequences whose tokens have time, height and width
        dict(name="axes_step", op="axes", tokens=64, Hq=32, Hkv=8, dim=128, layout="half", sections="16,24,24",
             order="blocks", spectrum="shared", scaling="none", factor=1.0, trained=8192, base=1.0e6, span=32768,
             frame=""),
        # an image's patches in a prompt, the axes in turn, an odd number of tokens
        dict(name="axes_image", op="axes", tokens=2585, Hq=28, Hkv=4, dim=128, layout="half", sections="24,20,20",
             order="cyclic", spectrum="shared", scaling="yarn", factor=2.0, trained=32768, base=5.0e6, span=8192,
             frame="47x55"),
        # a video's latent frames, each axis with its own frequencies, neighbouring pairs
        dict(name="axes_video", op="axes", tokens=14040, Hq=16, Hkv=16, dim=128, layout="interleaved",
             sections="22,21,21", order="blocks", spectrum="own", scaling="none", factor=1.0, trained=4096, base=1.0e4,
             span=64, frame="30x52"),
        # 64 decode steps of 8 sequences, one token of each at a time, into pages
        dict(name="append_steps", op="append", B=8, n=64, step=1, Hq=32, heads="0,32,32,32,64,32,0,32", S=4, W=32,
             ragged=False, paged=True, kv="bf16", dim=128, layout="half", sections="", fused=True, verify=1),
        # a prompt of 8K tokens into an empty slot, straight from the projection's rows
        dict(name="append_prompt", op="append", B=1, n=8192, step=8192, Hq=32, heads="0,32,32,32,64,32,0,32", S=16,
             W=1024, ragged=False, paged=False, kv="bf16", dim=128, layout="half", sections="", fused=True, verify=0),
        # two prompts with positions on three axes, 30 blocks of each head sealed on the way
        dict(name="append_sealed", op="append", B=2, n=4500, step=4500, Hq=32, heads="64,32,32,32,64,32,0,96", S=16,
             W=512, ragged=True, paged=True, kv="fp8_block", dim=128, layout="half", sections="16,24,24", fused=False,
             verify=2),
        # short sequences of odd lengths: a few sealed blocks each
        dict(name="decode_short", op="decode", B=8, N=777, Hq=8, heads="32,128", S=4, W=64, ragged=True, paged=False),
        # one 32K-token sequence
        dict(name="decode_one", op="decode", B=1, N=32768, Hq=32, heads="32,32,32,32,32,32,32,32", S=16, W=1024,
             ragged=False, paged=False),
        # 64 sequences of 2K to 4K tokens in pages
        dict(name="decode_batch", op="decode", B=64, N=4096, Hq=32, heads="0,32,32,32,64,32,0,32", S=16, W=512,
             ragged=True, paged=True),
        # four 128K-token sequences, seven query heads to a kv head
        dict(name="decode_long", op="decode", B=4, N=131072, Hq=28, heads="32,0,64,96", S=16, W=2048, ragged=False,
             paged=False),
        # four drafted tokens for each of 16 sequences of 8K tokens
        dict(name="verify_batch", op="chunk", B=16, N=8192, n=4, Hq=32, heads="64,32,32,32,64,32,0,96", S=16, W=512,
             ragged=False, paged=False),
        # one 512-token chunk of a long prompt, 32K tokens in
        dict(name="chunk_32k", op="chunk", B=1, N=32768, n=512, Hq=32, heads="0,32,32,32,64,32,0,32", S=16, W=1024,
             ragged=False, paged=True),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["axes", "axes", "append", "append", "decode", "decode", "chunk"])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 7, 8])
    layout = rng.choice(["half", "interleaved"])
    heads = ",".join(rng.choice(["0", "32", "32", "64", "96", "128"]) for _ in range(Hkv))
    S, W = rng.choice([0, 4, 16]), log(16, 2048)
    if op == "axes":
        dim = rng.choice([48, 64, 96, 128, 128, 128])
        a = rng.choice([2, 3, 3])
        rest = dim // 2 // a
        sections = [dim // 2 - (a - 1) * rest] + [rest] * (a - 1)
        frame = "" if rng.random() < 0.3 else "%dx%d" % (log(2, 64), log(2, 64))
        return dict(op=op, tokens=log(1, 14000), Hq=min(Hq, 28), Hkv=min(Hkv, 4), dim=dim, layout=layout,
                    sections=",".join(map(str, sections)), order=rng.choice(["blocks", "cyclic"]),
                    spectrum=rng.choice(["shared", "own"]), scaling=rng.choice(["none", "linear", "yarn"]),
                    factor=rng.uniform(1.5, 8.0), trained=rng.choice([4096, 8192, 32768]),
                    base=rng.choice([1.0e4, 5.0e5, 1.0e6]), span=log(64, 1 << 17), frame=frame)
    if op == "append":
        B, n = log(1, 8), log(1, 8192)
        while B * n > 8192:
            n //= 2
        step = 1 if n <= 64 else n
        paged, kv = rng.random() < 0.5, rng.choice(["bf16", "fp8_block"])
        dim = rng.choice([64, 128, 128])
        return dict(op=op, B=B, n=n, step=step, Hq=Hq, heads=heads, S=S, W=min(W, 1024),
                    ragged=step > 1 and rng.random() < 0.5, paged=paged, kv=kv, dim=dim, layout=layout,
                    sections="" if rng.random() < 0.5 else ",".join(map(str, [dim // 2 - 2 * (dim // 6), dim // 6, dim // 6])),
                    fused=rng.random() < 0.5, verify=rng.randint(1, 4) if paged or kv != "bf16" else rng.randint(0, 4))
    B, N = log(1, 64), log(1, 131072)
    n = log(1, 512) if op == "chunk" else 1
    while B * N * Hkv > 1 << 20 or B * (N + n) * n * Hq > 1 << 29:
        if B > 1 and rng.random() < 0.7:
            B //= 2
        elif n > 16:
            n //= 2
        else:
            N //= 2
    case = dict(op=op, B=B, N=N, Hq=Hq, heads=heads, S=S, W=W, ragged=rng.random() < 0.5, paged=rng.random() < 0.5)
    return dict(case, n=n) if op == "chunk" else case


# --------------------------------------------------------------------------
# what a case says
# --------------------------------------------------------------------------

def _kept(case):
    return [int(x) for x in case["heads"].split(",")]


def _spread(count, top, step):
    """`count` lengths between half of top and top."""
    return [top - i * step % (top // 2 + 1) for i in range(count)]


def _held(case):
    """Tokens that the sequences of a decode or chunk case hold."""
    return _spread(case["B"], case["N"], 37 * max(1, case["N"] // 500)) if case["ragged"] else [case["N"]] * case["B"]


def _taken(case):
    """Tokens that the slots of an append case take."""
    return _spread(case["B"], case["n"], 131) if case["ragged"] else [case["n"]] * case["B"]


def _resident(case, N, k, sealed):
    """Bytes that N tokens of a head with k kept channels hold."""
    S, W = case["S"], case["W"]
    middle = max(N - S - W, 0) if k else 0
    blocks = middle // 128 if sealed else 0
    return min(N, S + W) * 4 * D + blocks * (128 * (k + D) + 8) + (middle - 128 * blocks) * 2 * (k + D)


def _seen(case, N, n, k):
    """Multiply-adds, twice, of n queries that follow N tokens."""
    S, W, G = case["S"], case["W"], case["Hq"] // len(_kept(case))
    total = 0.0
    for p in range(N, N + n):
        near = min(p + 1, S) + min(max(p + 1 - S, 0), W)
        far = max(p + 1 - S - W, 0)
        total += 4.0 * D * near + ((2.0 * k + 2 * D) * far if k else 0.0)
    return G * total


def work(case):
    """Each input once, each output once, the cache's rows once; two operations
    per channel and (query, token) pair that the query sees, three per turned
    channel."""
    if case["op"] == "axes":
        heads = case["tokens"] * (case["Hq"] + case["Hkv"])
        axes = len(case["sections"].split(","))
        return {"bytes": 2.0 * 2 * D * heads + 4.0 * axes * case["tokens"], "flops": 3.0 * case["dim"] * heads}
    kept, Hq = _kept(case), case["Hq"]
    H = len(kept)
    if case["op"] == "append":
        move, ops = 0.0, 0.0
        for n in _taken(case):
            move += n * 2 * D * (2 * Hq + 2 * H)
            ops += 3.0 * case["dim"] * n * (Hq + H)
            for k in kept:
                move += _resident(case, n, k, case["kv"] != "bf16")
                if case["verify"]:
                    ops += _seen(case, n, case["verify"], k)
        return {"bytes": float(move), "flops": float(ops)}
    move, ops = 0.0, 0.0
    for N in _held(case):
        for k in kept:
            move += _resident(case, N, k, True)
            ops += _seen(case, N, case["n"], k) if case["op"] == "chunk" else _seen(case, N - 1, 1, k)
        move += case["n"] * 2 * D * (2 * Hq + 2 * H) if case["op"] == "chunk" else Hq * D * 6
    return {"bytes": float(move), "flops": float(ops)}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _keys(g, *shape):
    """Keys with a few large channels, as trained ones have."""
    x = _randn(g, *shape)
    x[..., 5] *= 4
    x[..., 69] *= 4
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"axes": _prepare_axes, "append": _prepare_append}.get(case["op"], _prepare_attend)(case, g)


def _grid(case, g, tokens, axes):
    """Positions [axes, tokens]: of text (the same on every axis), or of frames of
    h x w patches, one after another, from a drawn start on."""
    at = torch.arange(tokens, device="cuda")
    start = torch.randint(0, case["span"], (), generator=g, device="cuda")
    if not case["frame"]:
        far = torch.randint(0, case["span"], (tokens,), generator=g, device="cuda")
        return far.to(torch.int32).expand(axes, tokens).contiguous()
    h, w = map(int, case["frame"].split("x"))
    pos = [at // (h * w) + start, at % (h * w) // w + start, at % w + start]
    return torch.stack(pos[-axes:]).to(torch.int32).contiguous()


def _frequencies(case):
    """Angle per position and the axis of every pair, in 64 bits."""
    sections = [int(x) for x in case["sections"].split(",")] if case["sections"] else [case["dim"] // 2]
    pairs, A = case["dim"] // 2, len(sections)
    i = torch.arange(pairs)
    if case.get("order", "blocks") == "blocks":
        axis = torch.repeat_interleave(torch.arange(A), torch.tensor(sections))
    else:
        axis = torch.where(i < A * torch.tensor(sections)[i % A], i % A, 0)
    if case.get("spectrum", "shared") == "own":
        rank = (torch.nn.functional.one_hot(axis, A).cumsum(0) - 1)[i, axis].double()
        dim = 2.0 * torch.tensor(sections, dtype=torch.float64)[axis]
    else:
        rank, dim = i.double(), torch.full((pairs,), float(case["dim"]), dtype=torch.float64)
    base = case.get("base", 1.0e6)
    w = base ** (-2 * rank / dim)
    scaling, f = case.get("scaling", "none"), case.get("factor", 1.0)
    if scaling == "linear":
        w = w / f
    if scaling == "yarn":
        at = lambda turns: dim * math.log(case["trained"] / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = at(32.0).floor().clamp(min=0), torch.minimum(at(1.0).ceil(), dim - 1)
        ramp = ((rank - lo) / (hi - lo).clamp(min=1e-3)).clamp(0, 1)
        w = w / f * ramp + w * (1 - ramp)
    return w.cuda(), axis.cuda(), 0.1 * math.log(f) + 1.0 if scaling == "yarn" else 1.0


def _rope(case):
    from decode_attention_pruned_gb300 import binding as lk
    layout = {"half": lk.ROPE_HALF, "interleaved": lk.ROPE_INTERLEAVED}[case["layout"]]
    scaling = {"none": lk.ROPE_SCALE_NONE, "linear": lk.ROPE_SCALE_LINEAR, "yarn": lk.ROPE_SCALE_YARN}
    more = {}
    if case["sections"]:
        more = dict(axes=[int(x) for x in case["sections"].split(",")],
                    axis_order={"blocks": lk.ROPE_AXES_BLOCKS, "cyclic": lk.ROPE_AXES_CYCLIC}[case.get("order", "blocks")],
                    axis_spectrum={"shared": lk.ROPE_SPECTRUM_SHARED,
                                   "own": lk.ROPE_SPECTRUM_OWN}[case.get("spectrum", "shared")])
    return lk.Rope(rotary_dim=case["dim"], base=case.get("base", 1.0e6), layout=layout,
                   scaling=scaling[case.get("scaling", "none")], factor=case.get("factor", 1.0),
                   trained_positions=case.get("trained", 0), **more)


def _prepare_axes(case, g):
    T, Hq, H = case["tokens"], case["Hq"], case["Hkv"]
    freq, axis, mag = _frequencies(case)
    s = dict(case=case, q=_randn(g, T, Hq, D), k=_randn(g, T, H, D), freq=freq, axis=axis, mag=mag,
             pos=_grid(case, g, T, len(case["sections"].split(","))))
    s["qo"], s["ko"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    if own:
        s["rope"] = _rope(case)
    return s


def _masks(case, g):
    """Which channels each head keeps, [H, 128]."""
    kept = torch.tensor(_kept(case), device="cuda")
    order = torch.rand(len(kept), D, generator=g, device="cuda").argsort(1)
    keep = torch.zeros(len(kept), D, device="cuda", dtype=torch.bool)
    return keep.scatter_(1, order, torch.arange(D, device="cuda")[None] < kept[:, None]), kept


def _plan(case, keep):
    from decode_attention_pruned_gb300 import binding as lk
    return lk.Plan(1, case["Hq"], keep.shape[0], case["S"], case["W"], keep.to(torch.uint8).cpu().numpy()[None])


def _prepare_append(case, g):
    B, n, Hq, step, m = case["B"], case["n"], case["Hq"], case["step"], case["verify"]
    keep, kept = _masks(case, g)
    H = len(kept)
    if case["fused"]:
        row = _randn(g, B, n, Hq + 2 * H, D)
        q, k, v = row[:, :, :Hq], row[:, :, Hq:Hq + H], row[:, :, Hq + H:]
    else:
        q, k, v = _randn(g, B, n, Hq, D), _keys(g, B, n, H, D), _randn(g, B, n, H, D)
    freq, axis, mag = _frequencies(case)
    A = len(case["sections"].split(","))
    taken = _taken(case)
    s = dict(case=case, q=q, k=k, v=v, keep=keep, kept=kept, freq=freq, axis=axis, mag=mag, taken=taken,
             taken_d=torch.tensor(taken, device="cuda"), qo=torch.zeros(B, n, Hq, D, device="cuda", dtype=torch.bfloat16))
    if case["sections"]:
        # a frame of 32 x 40 patches after some text, and text again
        at = torch.arange(n, device="cuda")
        inside = (at >= 7) & (at < 7 + 1280)
        text = torch.where(at < 7, at, at - 1280 + 40)
        grid = torch.stack([torch.full_like(at, 7), 7 + (at - 7) // 40, 7 + (at - 7) % 40])
        pos = torch.where(inside, grid, torch.where(at < 7, at, text))[:, None].expand(A, B, n)
        off = torch.randint(0, 4096, (B, 1), generator=g, device="cuda")
        s["pos"] = (pos + off).to(torch.int32).contiguous()
        s["pos_of"] = [s["pos"][:, :, i:i + step].contiguous() for i in range(0, n, step)]
    if m:
        s["q2"], s["k2"], s["v2"] = _randn(g, B, m, Hq, D), _randn(g, B, m, H, D), _randn(g, B, m, H, D)
        s["o"] = torch.zeros_like(s["q2"])
    if own:
        from decode_attention_pruned_gb300 import binding as lk
        middle = sum(max(x - case["S"] - case["W"], 0) for x in taken)
        c = lk.Cache(_plan(case, keep), B, n, middle_tokens=middle if case["paged"] else None,
                     kv_format=lk.KV_FP8_BLOCK if case["kv"] == "fp8_block" else lk.KV_BF16)
        s["cache"], s["rope"] = c, _rope(case)
        # the resident rows: full-width ones [H, B, rows, 128], and where they are bf16 and in
        # one piece the middle of each head [B, rows, kept]
        r = [c.region(0, 0, h) for h in range(H)]
        s["rows"] = [c.rows(at, H * B * r[0].rows_a, D).view(H, B, r[0].rows_a, D)
                     for at in (r[0].k_a_offset, r[0].v_a_offset)]
        s["middle"] = [(c.rows(x.k_b_offset, B * x.rows_b, x.n_kept).view(B, x.rows_b, x.n_kept),
                        c.rows(x.v_b_offset, B * x.rows_b, D).view(B, x.rows_b, D))
                       for x in r if x.rows_b and not case["paged"] and case["kv"] == "bf16"]
    return s


def _seal(x, dims):
    """e4m3 codes of blocks and their scales, shared along `dims`; x is 0 where a
    channel is not held."""
    scale = x.abs().amax(dims, keepdim=True) / torch.tensor(448.0, device=x.device)
    scale = scale.clamp(min=2.0 ** -64)
    return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn), scale


def _blocks(case, hk, hv, keep):
    """Codes and scales of every 128 tokens of the middle that the longest sequence has complete."""
    B, N, H, _ = hk.shape
    nb = max(N - case["S"] - case["W"], 0) // 128
    at = slice(case["S"], case["S"] + 128 * nb)
    kc, ks = _seal((hk[:, at].float() * keep).view(B, nb, 128, H, D), (2, 4))
    vc, vs = _seal(hv[:, at].float().view(B, nb, 128, H, D), (2, 4))
    return dict(kc=kc, ks=ks, vc=vc, vs=vs)


def _prepare_attend(case, g):
    B, N, Hq = case["B"], case["N"], case["Hq"]
    n = case["n"] if case["op"] == "chunk" else 0
    keep, kept = _masks(case, g)
    H = len(kept)
    held = _held(case)
    s = dict(case=case, keep=keep, kept=kept, hk=_keys(g, B, N, H, D), hv=_randn(g, B, N, H, D), held=held,
             held_d=torch.tensor(held, device="cuda"), q=_randn(g, *((B, n, Hq, D) if n else (B, Hq, D))),
             k=_keys(g, B, n, H, D), v=_randn(g, B, n, H, D))
    s |= _blocks(case, s["hk"], s["hv"], keep)
    s["o"] = torch.zeros_like(s["q"], dtype=torch.bfloat16 if n else torch.float32)
    if own:
        from decode_attention_pruned_gb300 import binding as lk
        middle = sum(max(x - case["S"] - case["W"], 0) for x in held)
        s["cache"] = lk.Cache(_plan(case, keep), B, N + n, middle_tokens=middle if case["paged"] else None,
                              kv_format=lk.KV_FP8_BLOCK)
        s["cache"].prefill_ragged(0, s["hk"], s["hv"], held)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if op == "axes":
        return s["rope"].apply(s["q"], s["k"], s["pos"], q_out=s["qo"], k_out=s["ko"]) if own else _axes_plain(s)
    if op == "append":
        return _append_own(s) if own else _append_plain(s)
    if op == "decode":
        return s["cache"].decode(0, s["q"], s["o"]) if own else _decode_plain(s)
    if own:
        return s["cache"].chunk_attn(0, s["q"], s["k"], s["v"], o=s["o"])
    hk, hv = _history(s, s["hk"], s["hv"], s["held_d"], s)
    return _attend(s, s["q"], hk, hv, s["held_d"], s["k"], s["v"]).to(torch.bfloat16)


def _append_own(s):
    c, case = s["cache"], s["case"]
    step, lens = case["step"], s["taken"] if case["ragged"] else None
    none = s["k"][0, :0].contiguous()
    for b in range(case["B"]):              # the slots' last requests are done
        c.release(b)
        c.prefill_sequence(0, b, none, none)
    for i in range(0, case["n"], step):
        c.append_rope(0, s["rope"], s["k"][:, i:i + step], s["v"][:, i:i + step], q=s["q"][:, i:i + step],
                      q_out=s["qo"][:, i:i + step], lens=lens, positions=s["pos_of"][i // step] if "pos" in s else None)
    out = dict(q=s["qo"], rows=s["rows"], middle=s["middle"])
    if case["verify"]:
        out["o"] = c.chunk_attn(0, s["q2"], s["k2"], s["v2"], o=s["o"])
    return out


def _turn(x, turn, dim, layout):
    """x [..., tokens, heads, 128] turned by (cosine, sine) [..., tokens, 1, dim / 2]."""
    cos, sin = turn
    x = x.float()
    y = x[..., :dim]
    a, b = (y[..., :dim // 2], y[..., dim // 2:]) if layout == "half" else (y[..., 0::2], y[..., 1::2])
    c, e = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([c, e], -1) if layout == "half" else torch.stack([c, e], -1).flatten(-2)
    return torch.cat([y, x[..., dim:]], -1).to(torch.bfloat16)


def _turns(pos, s):
    """(cosine, sine) of every pair for positions [axes, ...]."""
    angle = (pos.double().movedim(0, -1)[..., s["axis"]] * s["freq"])[..., None, :]
    return (torch.cos(angle) * s["mag"]).float(), (torch.sin(angle) * s["mag"]).float()


def _axes_plain(s):
    turn = _turns(s["pos"], s)
    dim, layout = s["case"]["dim"], s["case"]["layout"]
    return _turn(s["q"], turn, dim, layout), _turn(s["k"], turn, dim, layout)


def _append_plain(s):
    case, kept = s["case"], s["kept"]
    S, W, n, B = case["S"], case["W"], case["n"], case["B"]
    H = len(kept)
    pos = s["pos"] if "pos" in s else torch.arange(n, device="cuda").expand(1, B, n)
    turn = _turns(pos, s)
    q, k = (_turn(x, turn, case["dim"], case["layout"]) for x in (s["q"], s["k"]))
    end = s["taken_d"][:, None]
    i = torch.arange(n, device="cuda")[None]
    q = torch.where((i < end)[..., None, None], q, 0)
    # the token in each full-width row: sinks, then a ring of the last W
    r = torch.arange(min(n, S + W), device="cuda")[None]
    last = end - 1 - (end - 1 - r) % W
    token = torch.where((end <= S + W) | (r < S), r, last)
    there = (r < torch.minimum(end, torch.tensor(S + W, device="cuda")))[..., None, None]
    b = torch.arange(B, device="cuda")[:, None]
    rows = [torch.where(there, x[b, token.clamp(0, n - 1)], 0).permute(2, 0, 1, 3) for x in (k, s["v"])]
    middle = []
    if not case["paged"] and case["kv"] == "bf16" and n > S + W:
        held = (i[:, S:n - W] < end - W)[..., None]
        middle = [(torch.where(held, k[:, S:n - W, h][..., keep], 0), torch.where(held, s["v"][:, S:n - W, h], 0))
                  for h, keep in enumerate(s["keep"]) if keep.any()]
    out = dict(q=q, rows=rows, middle=middle)
    if case["verify"]:
        blocks = _blocks(case, k, s["v"], s["keep"]) if case["kv"] != "bf16" else None
        hk, hv = _history(s, k, s["v"], s["taken_d"], blocks)
        out["o"] = _attend(s, s["q2"], hk, hv, s["taken_d"], s["k2"], s["v2"]).to(torch.bfloat16)
    return out


def _history(s, hk, hv, held, blocks):
    """Keys and values of the held tokens as the cache gives them: sealed blocks as
    codes times scale."""
    hk, hv = hk.float(), hv.float()
    if blocks is None or not blocks["kc"].shape[1]:
        return hk, hv
    case = s["case"]
    B, nb, _, H, _ = blocks["kc"].shape
    at = slice(case["S"], case["S"] + 128 * nb)
    sealed = torch.arange(nb, device="cuda").repeat_interleave(128)[None] < (held[:, None] - case["S"] - case["W"]).clamp(min=0) // 128
    sealed = sealed[..., None, None] & (s["kept"] > 0)[:, None]
    k, v = hk.clone(), hv.clone()
    k[:, at] = torch.where(sealed & s["keep"], (blocks["kc"].float() * blocks["ks"]).view(B, nb * 128, H, D), hk[:, at])
    v[:, at] = torch.where(sealed, (blocks["vc"].float() * blocks["vs"]).view(B, nb * 128, H, D), hv[:, at])
    return k, v


def _softmax(x, see):
    """Weights over what is seen, 0 for a query that sees nothing."""
    x = torch.where(see, x / math.sqrt(D), -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(m > -math.inf, m, 0))
    total = x.sum(-1, keepdim=True)
    return x / torch.where(total > 0, total, 1)


def _decode_plain(s):
    """One query at the last held token's position, over the held tokens."""
    hk, hv = _history(s, s["hk"], s["hv"], s["held_d"], s)
    B, Hq, _ = s["q"].shape
    return _attend(s, s["q"].view(B, 1, Hq, D), hk, hv, s["held_d"], None, None).view(B, Hq, D)


def _attend(s, q, hk, hv, held, k_new, v_new):
    """Queries q [B, n, Hq, 128] of new tokens (or of the last held one) over the
    held and the new tokens, in fp32."""
    case, kept, keep = s["case"], s["kept"], s["keep"]
    B, n, Hq, _ = q.shape
    H, N = len(kept), hk.shape[1]
    G = Hq // H
    S, W = case["S"], case["W"]
    K = (hk if k_new is None else torch.cat([hk, k_new.float()], 1)).permute(0, 2, 3, 1)       # [B, H, D, T]
    V = (hv if v_new is None else torch.cat([hv, v_new.float()], 1)).permute(0, 2, 1, 3)       # [B, H, T, D]
    # the position of every token, -1 where there is none
    i, j = torch.arange(N, device="cuda")[None], torch.arange(n, device="cuda")[None]
    held = held[:, None]
    t, p = torch.where(i < held, i, -1), held + j
    if k_new is not None:
        t = torch.cat([t, p], 1)
    else:
        p = p - 1
    t, p = t[:, None, None], p[:, None, :, None]                                               # [B, 1, n, T]
    near = (t < S) | (p - t < W)
    see = (t >= 0) & (t <= p) & (near | (kept > 0)[:, None, None])                             # [B, H, n, T]
    q = q.float().view(B, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, D)
    shape = (B, H, G, n, -1)
    x = torch.where(near[:, :, None], (q @ K).view(shape), ((q * keep[:, None]) @ K).view(shape))
    o = _softmax(x, see[:, :, None]).view(B, H, G * n, -1) @ V
    return o.view(B, H, G, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "axes":
        z = _spin(case, s["pos"])
        return _rotate(case, s["q"], z), _rotate(case, s["k"], z)
    if case["op"] == "append":
        return _exact_append(case, s)
    n = case["n"] if case["op"] == "chunk" else 1
    if 6.0 * D * case["Hq"] * n * sum(N + n for N in s["held"]) > 4.0e12:
        return None
    new = (s["k"], s["v"]) if case["op"] == "chunk" else None
    q = s["q"] if new else s["q"][:, None]
    return _exact_attend(case, s, q, s["hk"], s["hv"], s["held"], new, True).view(s["q"].shape)


def _spin(case, pos):
    """magnitude e^(i p w) of every token and pair, a complex [..., tokens, pairs]."""
    sections = [int(x) for x in case["sections"].split(",")] if case["sections"] else [case["dim"] // 2]
    A, half = len(sections), case["dim"] // 2
    if case.get("order", "blocks") == "blocks":
        owner = [a for a, c in enumerate(sections) for _ in range(c)]
    else:
        owner = [i % A if i < A * sections[i % A] else 0 for i in range(half)]
    seen, mag, base = [0] * A, 1.0, case.get("base", 1.0e6)
    w = torch.empty(half, dtype=torch.float64)
    for i, a in enumerate(owner):
        d, j = (2 * sections[a], seen[a]) if case.get("spectrum", "shared") == "own" else (2 * half, i)
        seen[a] += 1
        w[i] = math.exp(-math.log(base) * 2 * j / d)
        f = case.get("factor", 1.0)
        if case.get("scaling", "none") == "linear":
            w[i] /= f
        elif case.get("scaling", "none") == "yarn":
            # keep the pairs that turn over 32 times in the trained length, stretch those below one turn
            lo, hi = (d / 2.0 * math.log(case["trained"] / (r * 2 * math.pi), base) for r in (32.0, 1.0))
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), d - 1)
            stretch = min(max((j - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            w[i] *= stretch / f + 1 - stretch
            mag = 0.1 * math.log(f) + 1.0
    p = pos.double()[torch.tensor(owner, device="cuda")].movedim(0, -1)
    return mag * torch.exp(1j * p * w.cuda())


def _rotate(case, x, z):
    """Every pair (a, b) of x [..., tokens, heads, 128] as the number a + ib, times z."""
    d = case["dim"]
    i = torch.arange(d // 2, device="cuda")
    first, second = (i, i + d // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
    x = x.double().clone()
    y = torch.complex(x[..., first], x[..., second]) * z[..., None, :]
    x[..., first], x[..., second] = y.real, y.imag
    return x


def _exact_append(case, s):
    B, n, S, W = case["B"], case["n"], case["S"], case["W"]
    pos = s["pos"] if case["sections"] else torch.arange(n, device="cuda")[None, None].expand(1, B, n)
    z = _spin(case, pos)
    q, k, v = _rotate(case, s["q"], z), _rotate(case, s["k"], z), s["v"].double()
    H, width = k.shape[2], min(n, S + W)
    rows = [torch.zeros(H, B, width, D, dtype=torch.float64, device="cuda") for _ in range(2)]
    flat = not case["paged"] and case["kv"] == "bf16" and n > S + W
    middle = [(torch.zeros(B, n - S - W, c, dtype=torch.float64, device="cuda"),
               torch.zeros(B, n - S - W, D, dtype=torch.float64, device="cuda")) for c in _kept(case) if c and flat]
    for b, end in enumerate(s["taken"]):
        q[b, end:] = 0
        first = list(range(min(end, S)))
        tail = list(range(max(S, end - W), end)) if end > S else []
        at = torch.tensor([*first, *(S + (t - S) % W for t in tail)], dtype=torch.long, device="cuda")
        src = torch.tensor([*first, *tail], dtype=torch.long, device="cuda")
        for to, x in zip(rows, (k, v)):
            to[:, b, at] = x[b, src].transpose(0, 1)
        for (mk, mv), h in zip(middle, [h for h, c in enumerate(_kept(case)) if c]):
            count = max(end - S - W, 0)
            mk[b, :count] = k[b, S:S + count, h][:, s["keep"][h]]
            mv[b, :count] = v[b, S:S + count, h]
    out = dict(q=q, rows=rows, middle=middle)
    if case["verify"]:
        # what the cache holds of the keys are their bf16 roundings
        out["o"] = _exact_attend(case, s, s["q2"], k.to(torch.bfloat16), s["v"], s["taken"], (s["k2"], s["v2"]),
                                 case["kv"] != "bf16")
    return out


def _e4m3(x):
    """The e4m3 value nearest to x, ties to the even code, at most 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_attend(case, s, q, hk, hv, held, new, sealed):
    S, W = case["S"], case["W"]
    B, n, Hq, _ = q.shape
    kept = _kept(case)
    G = Hq // len(kept)
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for b, N in enumerate(held):
        for h, c in enumerate(kept):
            k, v = hk[b, :N, h].double(), hv[b, :N, h].double()
            keep = s["keep"][h]
            m = max(N - S - W, 0) // 128 * 128 if sealed and c else 0
            if m:
                for x, cols in ((k, keep), (v, torch.ones_like(keep))):
                    y = x[S:S + m][:, cols].view(m // 128, 128, -1)
                    scale = (y.abs().amax((1, 2), keepdim=True).float() / torch.tensor(448.0, device="cuda")).clamp(min=2.0 ** -64)
                    code = _e4m3((y.float() / scale).double())        # (the division is the format's, in 32 bits)
                    held_rows = x[S:S + m].clone()
                    held_rows[:, cols] = (code * scale.double()).reshape(m, -1)
                    x[S:S + m] = held_rows
            if new is not None:
                k, v = torch.cat([k, new[0][b, :, h].double()]), torch.cat([v, new[1][b, :, h].double()])
            at = torch.arange(N, N + n, device="cuda") - (0 if new is not None else 1)
            age = at[:, None] - torch.arange(k.shape[0], device="cuda")
            far = age >= W
            far[:, :S] = False
            hide = (age < 0) | far if c == 0 else age < 0
            for x in range(G):
                qx = q[b, :, h * G + x].double()
                y = torch.where(far, torch.einsum("nd,td->nt", qx * keep, k), torch.einsum("nd,td->nt", qx, k))
                y = (y / 128.0 ** 0.5).masked_fill_(hide, -math.inf)
                y -= torch.logsumexp(y, 1, keepdim=True)
                o[b, :, h * G + x] = torch.einsum("nt,td->nd", y.exp_().nan_to_num_(0.0), v)
    return o
