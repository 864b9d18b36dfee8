"""Rotary positions, attention of a chunk of new tokens over the pruned cache,
and the chunk's entry into it: the cases they are measured on, in plain form
and through the package.

The three belong together.  A serving program that feeds a prompt in chunks,
or verifies drafted tokens, turns each chunk's q and k by their positions
(``Rope.apply``), attends with the chunk's queries over the cache and the
chunk itself (``Cache.chunk_attn``), and then lets the chunk's tokens into the
cache (``Cache.append_chunk``; ``Cache.extend`` is the two in one call).

What a query at position p sees of the token at position t <= p, per kv head:
  FULL     t < S or p - t < W: the score q.k / sqrt(128) over all channels;
           else, with k > 0 kept channels, the score over those channels
           alone; else (k = 0) nothing
  LOCAL    the tokens with p - t < W_loc
  SPECIAL  the tokens whose id is special
One softmax runs over what it sees; a query that sees nothing gives 0.

A case is a dict of plain values:
  op "rope"    tokens, Hq, Hkv, dim (channels turned), layout, scaling, base,
               factor, trained (positions), span (positions drawn below it),
               fused (q and k are views of one row per token: q | k | v)
  op "chunk"   B sequences holding up to N tokens, n new ones each; heads: the
               kv heads' kept counts (FULL), "L" (LOCAL) or "S" (SPECIAL);
               ragged: sequences of several lengths; paged; kv: bf16 | int8 | fp8
  op "extend"  one sequence of T tokens that enters an empty slot n at a time
"""
import math

import numpy as np
import torch

own = False

D = 128
VOCAB = 32000


def listed():
    return [
        # one decode step of a 64-sequence batch: what a step waits for
        dict(name="rope_step", op="rope", tokens=64, Hq=32, Hkv=8, dim=128, layout="half", scaling="none",
             base=5.0e5, factor=1.0, trained=8192, span=4096, fused=False),
        # a long chunk far into a context stretched past the trained length
        dict(name="rope_far", op="rope", tokens=8192, Hq=28, Hkv=4, dim=128, layout="half", scaling="yarn",
             base=1.0e6, factor=4.0, trained=32768, span=131072, fused=False),
        # half of each head turned, neighbouring pairs, q and k inside the projection's rows
        dict(name="rope_part", op="rope", tokens=2053, Hq=32, Hkv=8, dim=64, layout="interleaved",
             scaling="linear", base=1.0e4, factor=2.0, trained=4096, span=8192, fused=True),
        # five drafted tokens verified against one 32K-token sequence
        dict(name="verify_one", op="chunk", B=1, N=32768, n=5, Hq=32, heads="0,32,32,32,64,32,0,32", S=16, W=1024,
             Wl=0, ragged=False, paged=True, kv="bf16"),
        # four drafted tokens for each of 64 sequences of 2K to 4K tokens
        dict(name="verify_batch", op="chunk", B=64, N=4096, n=4, Hq=32, heads="0,32,32,32,64,32,0,32", S=16, W=512,
             Wl=0, ragged=True, paged=True, kv="bf16"),
        # the same kind of step over a cache with an FP8 middle
        dict(name="verify_fp8", op="chunk", B=16, N=8192, n=4, Hq=32, heads="64,32,32,32,64,32,0,96", S=16, W=512,
             Wl=0, ragged=False, paged=False, kv="fp8"),
        # one 512-token chunk of a long prompt, 32K tokens in
        dict(name="chunk_32k", op="chunk", B=1, N=32768, n=512, Hq=32, heads="0,32,32,32,64,32,0,32", S=16, W=1024,
             Wl=0, ragged=False, paged=True, kv="bf16"),
        # an odd chunk 128K tokens in, seven query heads to a kv head
        dict(name="chunk_128k", op="chunk", B=1, N=131072, n=1000, Hq=28, heads="32,0,32,32", S=16, W=2048,
             Wl=0, ragged=False, paged=False, kv="bf16"),
        # short chunks of 16 sequences, heads of every policy
        dict(name="chunk_mix", op="chunk", B=16, N=16384, n=64, Hq=32, heads="32,L,64,S,L,32,L,S", S=16, W=512,
             Wl=256, ragged=True, paged=False, kv="bf16"),
        # the first chunk of two prompts: nothing in the cache yet
        dict(name="chunk_first", op="chunk", B=2, N=0, n=4096, Hq=32, heads="0,32,32,32,64,32,0,32", S=16, W=512,
             Wl=0, ragged=False, paged=False, kv="bf16"),
        # a 4K-token prompt that enters a slot 512 tokens at a time
        dict(name="extend_4k", op="extend", T=4096, n=512, Hq=32, heads="0,32,32,32,64,32,0,32", S=16, W=512, Wl=0),
        # a short prompt in odd pieces, heads of two policies
        dict(name="extend_odd", op="extend", T=777, n=100, Hq=8, heads="96,L,128,0", S=4, W=64, Wl=48),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["rope", "chunk", "chunk", "chunk", "extend"])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 7, 8])
    if op == "rope":
        scaling = rng.choice(["none", "linear", "ntk", "yarn", "bands"])
        return dict(op=op, tokens=log(1, 8192), Hq=min(Hq, 28), Hkv=min(Hkv, 4), dim=rng.choice([32, 64, 96, 128, 128]),
                    layout=rng.choice(["half", "interleaved"]), scaling=scaling,
                    base=rng.choice([1.0e4, 5.0e5, 1.0e6]), factor=1.0 if scaling == "none" else rng.uniform(1.5, 8.0),
                    trained=rng.choice([4096, 8192, 32768]), span=log(64, 1 << 20), fused=rng.random() < 0.5)
    S, W, Wl = rng.choice([0, 4, 16]), log(16, 2048), log(16, 512)
    kept = ["0", "32", "64", "96", "128"]
    if op == "extend":
        T = log(1, 4096)
        return dict(op=op, T=T, n=max(log(1, 1024), T // 16 + 1), Hq=Hq, S=S, W=W, Wl=Wl,
                    heads=",".join(rng.choice(kept + ["L"]) for _ in range(Hkv)))
    kv = rng.choice(["bf16", "bf16", "int8", "fp8"])
    heads = ",".join(rng.choice(kept if kv != "bf16" else kept + ["L", "S"]) for _ in range(Hkv))
    B, n = log(1, 64), log(1, 1000)
    N = 0 if rng.random() < 0.1 else log(1, 65536)
    while B * N * Hkv > 1 << 20 or B * (N + n) * n * Hq > 450 * 131072 * 28:
        if n > 64 and (rng.random() < 0.5 or N < 64):
            n //= 2
        elif B > 1:
            B //= 2
        else:
            N //= 2
    return dict(op=op, B=B, N=N, n=n, Hq=Hq, heads=heads, S=S, W=W, Wl=Wl, ragged=kv == "bf16" and rng.random() < 0.5,
                paged=rng.random() < 0.5, kv=kv)


# --------------------------------------------------------------------------
# what a case says
# --------------------------------------------------------------------------

def _heads(case):
    """Per kv head: policy (0 FULL, 1 LOCAL, 2 SPECIAL) and kept channels."""
    names = case["heads"].split(",")
    return [{"L": 1, "S": 2}.get(x, 0) for x in names], [int(x) if x.isdigit() else 0 for x in names]


def _lengths(case):
    """Tokens held and new tokens of every sequence."""
    b = range(case["B"])
    if not case["ragged"]:
        return [case["N"] for _ in b], [case["n"] for _ in b]
    return ([case["N"] - i * 37 * max(1, case["N"] // 500) % (case["N"] // 2 + 1) for i in b],
            [case["n"] - i * 5 % (case["n"] // 2 + 1) for i in b])


def _specials(w):
    """Whether each id of the vocabulary is special: one in twenty."""
    return torch.arange(VOCAB, device=w) % 20 == 7


def work(case):
    """Each tensor once, the cache rows that the heads hold once; two
    multiply-adds per channel and (query, token) pair that the query sees."""
    if case["op"] == "rope":
        n = case["tokens"] * (case["Hq"] + case["Hkv"])
        return {"bytes": 2 * 2 * D * n + 4 * case["tokens"], "flops": 3 * case["dim"] * n}
    policy, kept = _heads(case)
    H = len(policy)
    G = case["Hq"] // H
    S, W, Wl = case["S"], case["W"], case["Wl"]
    held, new = ([0], [case["T"]]) if case["op"] == "extend" else _lengths(case)
    move, pairs = 0.0, 0.0
    for N, n in zip(held, new):
        p = N + np.arange(n, dtype=np.int64)
        near = np.minimum(p + 1, S) + np.minimum(np.maximum(p + 1 - S, 0), W)
        far = np.maximum(p + 1 - S - W, 0)
        move += n * (2 * case["Hq"] + 2 * H) * 2 * D
        for pol, k in zip(policy, kept):
            if pol == 0:
                pairs += G * (4.0 * D * near.sum() + (2.0 * k + 2 * D) * (far.sum() if k else 0))
                middle = max(N - S - W, 0) if k else 0
                sealed = 0 if case.get("kv", "bf16") == "bf16" else middle // 128
                move += min(N, S + W) * 4 * D + sealed * 132 * (k + 128) + (middle - 128 * sealed) * 2 * (k + D)
                if case["op"] == "extend":
                    move += min(n, S + W) * 4 * D + (max(n - S - W, 0) * 2 * (k + D) if k else 0)
            elif pol == 1:
                pairs += G * 4.0 * D * np.minimum(p + 1, Wl).sum()
                move += min(N, Wl) * 4 * D + (min(n, Wl) * 4 * D if case["op"] == "extend" else 0)
            else:
                pairs += G * 4.0 * D * (p / 20.0 + 0.05).sum()
                move += N / 20.0 * 4 * D
    return {"bytes": float(move), "flops": float(pairs)}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _history(g, *shape):
    """Keys with a few large channels, as trained ones have."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    x[..., 5] *= 4
    x[..., 69] *= 4
    return x


def _seal(x, dims, kv):
    """Codes of 128-row blocks and their scales: largest magnitude / 127 or
    / 448, shared along `dims`."""
    top = torch.tensor(127.0 if kv == "int8" else 448.0, device="cuda")
    scale = x.abs().amax(dims, keepdim=True) / top
    y = torch.where(scale > 0, x / torch.where(scale > 0, scale, torch.ones_like(scale)), torch.zeros_like(x))
    if kv == "int8":
        return y.round().clamp(-127, 127).to(torch.int8), scale
    return y.clamp(-448, 448).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "rope":
        return _prepare_rope(case, g)
    policy, kept = _heads(case)
    H, G, Hq = len(policy), case["Hq"] // len(policy), case["Hq"]
    beta = torch.zeros(H, D, device="cuda")
    order = torch.rand(H, D, generator=g, device="cuda").argsort(1)
    beta.scatter_(1, order, (torch.arange(D, device="cuda")[None] < torch.tensor(kept, device="cuda")[:, None]).float())
    s = dict(case=case, H=H, G=G, beta=beta, policy=torch.tensor(policy, device="cuda"),
             kept=torch.tensor(kept, device="cuda"))
    special = "S" in case["heads"]
    if case["op"] == "extend":
        T = case["T"]
        s |= dict(q=_randn(g, 1, T, Hq, D).bfloat16(), k=_history(g, 1, T, H, D), v=_randn(g, 1, T, H, D).bfloat16(),
                  hk=torch.empty(1, 0, H, D, device="cuda", dtype=torch.bfloat16),
                  hv=torch.empty(1, 0, H, D, device="cuda", dtype=torch.bfloat16), held=[0], new=[T])
    else:
        B, N, n = case["B"], case["N"], case["n"]
        held, new = _lengths(case)
        s |= dict(q=_randn(g, B, n, Hq, D).bfloat16(), k=_history(g, B, n, H, D), v=_randn(g, B, n, H, D).bfloat16(),
                  hk=_history(g, B, N, H, D), hv=torch.randn(B, N, H, D, generator=g, device="cuda", dtype=torch.bfloat16),
                  held=held, new=new)
        if special:
            s["ids"] = torch.randint(0, VOCAB, (B, N + n), generator=g, device="cuda", dtype=torch.int32)
        if case["kv"] != "bf16":
            # what the cache holds of the middle: complete 128-row blocks as codes and scales
            nb = max(N - case["S"] - case["W"], 0) // 128
            at = slice(case["S"], case["S"] + 128 * nb)
            s["kc"], s["ks"] = _seal(s["hk"][:, at].float().view(B, nb, 128, H, D), 2, case["kv"])
            s["vc"], s["vs"] = _seal(s["hv"][:, at].float().view(B, nb, 128, H, D), 4, case["kv"])
    s["held_d"] = torch.tensor(s["held"], device="cuda")
    s["new_d"] = torch.tensor(s["new"], device="cuda")
    s["o"] = torch.zeros_like(s["q"])
    if own:
        _prepare_cache(s, special)
    return s


def _prepare_rope(case, g):
    T, Hq, H = case["tokens"], case["Hq"], case["Hkv"]
    pos = torch.randint(0, case["span"], (T,), generator=g, device="cuda", dtype=torch.int32)
    if case["fused"]:
        row = _randn(g, T, Hq + 2 * H, D).bfloat16()
        q, k = row[:, :Hq], row[:, Hq:Hq + H]
    else:
        q, k = _randn(g, T, Hq, D).bfloat16(), _randn(g, T, H, D).bfloat16()
    s = dict(case=case, q=q, k=k, pos=pos, freq=_frequencies(case).cuda(), mag=_magnitude(case))
    s["qo"], s["ko"] = torch.empty(T, Hq, D, device="cuda", dtype=torch.bfloat16), \
        torch.empty(T, H, D, device="cuda", dtype=torch.bfloat16)
    if own:
        from decode_attention_pruned_gb300 import binding as lk
        layout = {"half": lk.ROPE_HALF, "interleaved": lk.ROPE_INTERLEAVED}[case["layout"]]
        scaling = {"none": lk.ROPE_SCALE_NONE, "linear": lk.ROPE_SCALE_LINEAR, "ntk": lk.ROPE_SCALE_NTK,
                   "yarn": lk.ROPE_SCALE_YARN, "bands": lk.ROPE_SCALE_BANDS}[case["scaling"]]
        s["rope"] = lk.Rope(rotary_dim=case["dim"], base=case["base"], layout=layout, scaling=scaling,
                            factor=case["factor"], trained_positions=case["trained"])
    return s


def _frequencies(case):
    """Angle per position of every pair, in 64 bits."""
    d, b, f, L = case["dim"], case["base"], case["factor"], case["trained"]
    i = torch.arange(d // 2, dtype=torch.float64)
    if case["scaling"] == "ntk":
        b = b * f ** (d / (d - 2))
    w = b ** (-2 * i / d)
    if case["scaling"] == "linear":
        return w / f
    if case["scaling"] == "yarn":
        at = lambda turns: d * math.log(L / (turns * 2 * math.pi)) / (2 * math.log(b))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), d - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return w / f * ramp + w * (1 - ramp)
    if case["scaling"] == "bands":
        turns = L * w / (2 * math.pi)
        mix = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return (1 - mix) * w / f + mix * w
    return w


def _magnitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "yarn" else 1.0


def _prepare_cache(s, special):
    """The cache a serving program holds before the call, filled as it fills it."""
    from decode_attention_pruned_gb300 import binding as lk
    case, H = s["case"], s["H"]
    masks = s["beta"].to(torch.uint8).cpu().numpy()[None]
    masks[0, s["policy"].cpu().numpy() != 0] = 1
    plan = lk.Plan(1, case["Hq"], H, case["S"], case["W"], masks, s["policy"].cpu().numpy()[None].astype(np.int32),
                   local_only_window=case["Wl"],
                   is_special=_specials("cuda").cpu().numpy().astype(np.uint8) if special else None)
    if case["op"] == "extend":
        c = lk.Cache(plan, 1, case["T"])
        regions = [c.region(0, 0, h) for h in range(H)]
        s["rows"] = [(c.rows(r.k_a_offset, r.rows_a, D), c.rows(r.v_a_offset, r.rows_a, D)) for r in regions]
        s["middle"] = [(c.rows(r.k_b_offset, r.rows_b, r.n_kept), c.rows(r.v_b_offset, r.rows_b, D))
                       for r in regions if r.n_kept]
    else:
        fmt = {"bf16": lk.KV_BF16, "int8": lk.KV_INT8, "fp8": lk.KV_FP8}[case["kv"]]
        mid = sum(max(N - case["S"] - case["W"], 0) for N in s["held"])
        c = lk.Cache(plan, case["B"], case["N"] + case["n"], middle_tokens=mid if case["paged"] else None, kv_format=fmt)
        ids = s["ids"][:, :case["N"]].contiguous() if special else None
        c.prefill_ragged(0, s["hk"], s["hv"], s["held"], ids)
        s["new_ids"] = s["ids"][:, case["N"]:].contiguous() if special else None
    s["cache"] = c


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    if s["case"]["op"] == "rope":
        return _rope_own(s) if own else _rope_plain(s)
    if s["case"]["op"] == "chunk":
        return _chunk_own(s) if own else _attend(s)
    return _extend_own(s) if own else _extend_plain(s)


def _rope_own(s):
    return s["rope"].apply(s["q"], s["k"], s["pos"], q_out=s["qo"], k_out=s["ko"])


def _chunk_own(s):
    return s["cache"].chunk_attn(0, s["q"], s["k"], s["v"], lens=s["new"] if s["case"]["ragged"] else None,
                                 ids=s["new_ids"], o=s["o"])


def _extend_own(s):
    c, n = s["cache"], s["case"]["n"]
    none = s["k"][0, :0]
    c.release(0)                        # the slot's last request is done
    c.prefill_sequence(0, 0, none, none)
    for i in range(0, s["case"]["T"], n):
        c.extend(0, s["q"][:, i:i + n], s["k"][:, i:i + n], s["v"][:, i:i + n], o=s["o"][:, i:i + n])
    return s["o"], s["rows"], s["middle"]


def _turn(x, cos, sin, dim, layout):
    x = x.float()
    y = x[..., :dim]
    a, b = (y[..., :dim // 2], y[..., dim // 2:]) if layout == "half" else (y[..., 0::2], y[..., 1::2])
    c, e = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([c, e], -1) if layout == "half" else torch.stack([c, e], -1).flatten(-2)
    return torch.cat([y, x[..., dim:]], -1).to(torch.bfloat16)


def _rope_plain(s):
    angle = s["pos"].double()[:, None, None] * s["freq"]
    cos, sin = (torch.cos(angle) * s["mag"]).float(), (torch.sin(angle) * s["mag"]).float()
    dim, layout = s["case"]["dim"], s["case"]["layout"]
    return _turn(s["q"], cos, sin, dim, layout), _turn(s["k"], cos, sin, dim, layout)


def _history_seen(s):
    """Keys and values of the held tokens as the cache gives them."""
    k, v = s["hk"].float(), s["hv"].float()
    if "kc" in s:
        B, nb, _, H, _ = s["kc"].shape
        S = s["case"]["S"]
        at = lambda c, e: (c.float() * e).reshape(B, nb * 128, H, D)  # noqa: E731
        k = torch.cat([k[:, :S], at(s["kc"], s["ks"]), k[:, S + 128 * nb:]], 1) if nb else k
        v = torch.cat([v[:, :S], at(s["vc"], s["vs"]), v[:, S + 128 * nb:]], 1) if nb else v
    return k, v


def _attend(s):
    case, H, G = s["case"], s["H"], s["G"]
    B, n = s["q"].shape[:2]
    hk, hv = _history_seen(s)
    K = torch.cat([hk, s["k"].float()], 1).permute(0, 2, 3, 1)               # [B, H, D, T]
    V = torch.cat([hv, s["v"].float()], 1).permute(0, 2, 1, 3)               # [B, H, T, D]
    N = hk.shape[1]
    # the position of every token, -1 where there is none
    i, j = torch.arange(N, device="cuda")[None], torch.arange(n, device="cuda")[None]
    held, new = s["held_d"][:, None], s["new_d"][:, None]
    t = torch.cat([torch.where(i < held, i, -1), torch.where(j < new, held + j, -1)], 1)[:, None]    # [B, 1, T]
    V = torch.where(t[..., None] >= 0, V, 0)
    p = (held + j)[..., None]                                                # [B, n, 1]
    near = (t < case["S"]) | (p - t < case["W"])
    seen = ((t >= 0) & (t <= p))[:, None]                                    # [B, 1, n, T]
    pol, kept = s["policy"][None, :, None, None], s["kept"][None, :, None, None]
    see = seen & torch.where(pol == 0, near[:, None] | (kept > 0), True)
    whole = (pol != 0) | near[:, None]
    see = torch.where(pol == 1, seen & (p - t < case["Wl"])[:, None], see)
    if "ids" in s:
        flag = _specials("cuda")[s["ids"].long()][:, None, None]
        see = torch.where(pol == 2, seen & flag, see)
    q = s["q"].float().view(B, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, D)
    shape = (B, H, G, n, -1)
    x = torch.where(whole[:, :, None], (q @ K).view(shape), ((q * s["beta"][:, None]) @ K).view(shape))
    x = torch.where(see[:, :, None], x / math.sqrt(D), -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(m > -math.inf, m, 0))
    l = x.sum(-1, keepdim=True)
    o = (x.view(B, H, G * n, -1) @ V).view(B, H, G, n, D)
    o = torch.where((l > 0) & (j < new)[:, None, None, :, None], o / torch.where(l > 0, l, 1), 0)
    return o.permute(0, 3, 1, 2, 4).reshape(B, n, H * G, D).to(torch.bfloat16)


def _ring(first, window, end):
    """The tokens that `window` rows hold once `end` tokens are in, row r of
    them taking the tokens first + r, first + r + window, ..."""
    r = torch.arange(window, device="cuda")
    return end - 1 - (end - 1 - first - r) % window


def _extend_plain(s):
    case, T = s["case"], s["case"]["T"]
    S, W, Wl = case["S"], case["W"], case["Wl"]
    full = torch.arange(T, device="cuda") if T <= S + W else \
        torch.cat([torch.arange(S, device="cuda"), _ring(S, W, T)])
    local = torch.arange(T, device="cuda") if T <= Wl else _ring(0, Wl, T)
    policy, kept = _heads(case)
    rows = [(s["k"][0, full if p == 0 else local, h], s["v"][0, full if p == 0 else local, h])
            for h, p in enumerate(policy)]
    at = torch.arange(S, max(T - W, S), device="cuda")
    middle = [(s["k"][0, at, h][:, s["beta"][h].nonzero()[:, 0]], s["v"][0, at, h]) for h, c in enumerate(kept) if c]
    return _attend(s), rows, middle


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    if 6.0 * D * case["Hq"] * sum(n * (N + n) for N, n in zip(s["held"], s["new"])) > 1.0e13:
        return None
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    policy, kept = _heads(case)
    S, W, G = case["S"], case["W"], s["G"]
    for b, (N, n) in enumerate(zip(s["held"], s["new"])):
        for h, (pol, c) in enumerate(zip(policy, kept)):
            k = torch.cat([s["hk"][b, :N, h], s["k"][b, :n, h]]).double()
            v = torch.cat([s["hv"][b, :N, h], s["v"][b, :n, h]]).double()
            if "kc" in s and c:
                m = max(N - S - W, 0) // 128 * 128
                k[S:S + m] = (s["kc"][b, :, :, h].double() * s["ks"][b, :, :, h].double()).reshape(m, D)
                v[S:S + m] = (s["vc"][b, :, :, h].double() * s["vs"][b, :, :, h].double()).reshape(m, D)
            age = torch.arange(N, N + n, device="cuda")[:, None] - torch.arange(N + n, device="cuda")
            hide = age < 0
            far = torch.zeros_like(hide)
            if pol == 0:
                far = age >= W
                far[:, :S] = False
                hide = hide | (far if c == 0 else torch.zeros_like(far))
            elif pol == 1:
                hide = hide | (age >= case["Wl"])
            else:
                ids = torch.cat([s["ids"][b, :N], s["ids"][b, case["N"]:case["N"] + n]])
                hide = hide | (ids % 20 != 7)
            rest = k * (1 - s["beta"][h].double())
            for g in range(G):
                q = s["q"][b, :n, h * G + g].double()
                x = torch.einsum("nd,td->nt", q, k)
                if bool(far.any()) and c:
                    x -= far * torch.einsum("nd,td->nt", q, rest)
                x = (x / 128.0 ** 0.5).masked_fill_(hide, -math.inf)
                x -= torch.logsumexp(x, 1, keepdim=True)
                o[b, :n, h * G + g] = torch.einsum("nt,td->nd", x.exp_().nan_to_num_(0.0), v)
    return o if case["op"] == "chunk" else (o, None, None)


def _exact_rope(case, s):
    """Every pair (x, y) as the complex number x + iy, times magnitude e^(i p w)."""
    d = case["dim"]
    i = np.arange(d // 2)
    b, f, L = case["base"], case["factor"], case["trained"]
    if case["scaling"] == "ntk":
        b = b * f ** (d / (d - 2.0))
    w = np.power(b, -2.0 * i / d)
    mag = 1.0
    if case["scaling"] == "linear":
        w = w / f
    elif case["scaling"] == "yarn":
        # keep the pairs that turn over 32 times in the trained length, stretch those below one turn
        edge = [d / 2.0 * math.log(L / (r * 2 * math.pi), b) for r in (32.0, 1.0)]
        lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), d - 1)
        keep = 1.0 - np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        w, mag = w * (keep + (1 - keep) / f), 0.1 * math.log(f) + 1.0
    elif case["scaling"] == "bands":
        wave = 2 * math.pi / w
        keep = np.clip((L / wave - 1.0) / 3.0, 0, 1)
        w = w * (keep + (1 - keep) / f)
    turn = torch.polar(torch.full((1,), mag, dtype=torch.float64), torch.zeros(1, dtype=torch.float64)).cuda() * \
        torch.exp(1j * s["pos"].double()[:, None] * torch.from_numpy(w).cuda())
    out = []
    for x in (s["q"], s["k"]):
        x = x.double().clone()
        a = torch.arange(d // 2, device="cuda")
        first, second = (a, a + d // 2) if case["layout"] == "half" else (2 * a, 2 * a + 1)
        z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
        x[..., first], x[..., second] = z.real, z.imag
        out.append(x)
    return tuple(out)
