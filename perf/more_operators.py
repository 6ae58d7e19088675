"""Measured cases of a step's operators around the paged cache: norm and rotation of queries and
keys on their way into the cache, attention with a sliding window and a few first tokens that
stay visible (one token per request, or a chunk), and verification of drafted tokens.

Every case names its operator (``op``) and the ranges its lengths are drawn from; ``lens`` seeds
those lengths, so a case always has the same amount of work, while the values, the block
permutation and the random numbers come from the seed given to ``prepare``. Blocks that have
left the window have gone back to the free list: their table entries are -1.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "fp8": torch.bfloat16}
_EPS = 1e-6


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # the decode step of eight requests, one kv-head per query head: latency
        dict(name="rope_step_bf16", op="rope", kv="bf16", T=8, pad=0, H=32, H_kv=32, D=128, R=128,
             half=True, norm=False, fused=True, bs=16, far=4096, stretch=1.0, lens=1),
        # the decode step of 256 requests over long contexts into an 8-bit cache, with norms and
        # frequencies stretched by parts; a few rows are padding
        dict(name="rope_decode_fp8", op="rope", kv="fp8", T=256, pad=5, H=32, H_kv=8, D=128,
             R=128, half=True, norm=True, fused=True, bs=16, far=131072, stretch=8.0, lens=2),
        # the tokens of a large prefill batch
        dict(name="rope_prefill_bf16", op="rope", kv="bf16", T=16384, pad=0, H=32, H_kv=8, D=128,
             R=128, half=True, norm=True, fused=True, bs=16, far=32768, stretch=1.0, lens=3),
        # half of each head rotated, pairs side by side, an odd number of tokens, 32 bits
        dict(name="rope_pairs_f32", op="rope", kv="f32", T=1021, pad=0, H=16, H_kv=2, D=64, R=32,
             half=False, norm=False, fused=False, bs=64, far=8192, stretch=1.0, lens=4),
        # one short-window step of a small batch: latency
        dict(name="window_small_f16", op="wdec", kv="f16", B=4, H=16, H_kv=2, D=64, bs=16, W=250,
             S=4, past_lo=1, past_hi=1500, lens=5),
        # the decode step of the 256-request batch, over 4096 keys and 4 first ones
        dict(name="window_decode_bf16", op="wdec", kv="bf16", B=256, H=32, H_kv=8, D=128, bs=16,
             W=4096, S=4, past_lo=16, past_hi=32767, lens=6),
        # a short odd window over an 8-bit cache in larger blocks
        dict(name="window_decode_fp8", op="wdec", kv="fp8", B=128, H=32, H_kv=8, D=128, bs=64,
             W=1023, S=16, past_lo=100, past_hi=32767, lens=7),
        # drafted tokens of a decode batch
        dict(name="window_verify_bf16", op="wchunk", kv="bf16", B=32, H=32, H_kv=8, D=128, bs=16,
             W=2048, S=4, n_lo=1, n_hi=8, past_lo=512, past_hi=8192, lens=8),
        # a chunk of a long prompt
        dict(name="window_chunk_bf16", op="wchunk", kv="bf16", B=1, H=32, H_kv=8, D=128, bs=16,
             W=4096, S=64, n_lo=4096, n_hi=4096, past_lo=12288, past_hi=12288, lens=9),
        # ragged prompts longer than a short window, one kv-head per query head
        dict(name="window_prompts_f16", op="wchunk", kv="f16", B=6, H=40, H_kv=40, D=128, bs=16,
             W=513, S=0, n_lo=300, n_hi=1900, past_lo=0, past_hi=0, lens=10),
        # four drafted tokens of one request
        dict(name="verify_one_bf16", op="verify", kv="bf16", B=1, n_lo=5, n_hi=5, V=32000,
             drafted=True, cut=False, lens=11),
        # a batch of drafts over a large vocabulary
        dict(name="verify_batch_f32", op="verify", kv="f32", B=64, n_lo=2, n_hi=9, V=131072,
             drafted=True, cut=True, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "wdec", "wdec", "wchunk", "wchunk", "verify"])
    lens = rng.randrange(1 << 20)
    bs = rng.choice([16, 16, 32, 64, 128, 256])
    if op == "verify":
        V, B, n = _log(rng, 100, 150000), _log(rng, 1, 96), rng.randint(1, 9)
        return dict(op=op, kv=rng.choice(["f32", "f32", "bf16", "f16"]), B=B,
                    n_lo=rng.randint(1, n), n_hi=n, V=V, drafted=rng.choice([True, True, False]),
                    cut=rng.choice([True, False]), lens=lens)
    kv = rng.choice(["bf16", "bf16", "f16", "fp8", "f32"])
    H, H_kv = rng.choice([(32, 32), (32, 8), (40, 40), (16, 2), (8, 1), (12, 6)])
    if op == "rope":
        D = rng.choice([64, 128, 128, 256])
        T = _log(rng, 1, min(16384, 16384 * 48 * 128 // ((H + 2 * H_kv) * D)))
        return dict(op=op, kv=kv, T=T, pad=rng.choice([0, T // 5]), H=H, H_kv=H_kv, D=D,
                    R=rng.choice([D, D, D // 2, D // 4]), half=rng.choice([True, True, False]),
                    norm=rng.choice([True, False]), fused=rng.choice([True, False]), bs=bs,
                    far=_log(rng, 16, 1 << 20), stretch=rng.choice([1.0, 1.0, 4.0, 16.0]),
                    lens=lens)
    D = rng.choice([64, 128, 128])
    S = rng.choice([0, 1, 4, rng.randint(2, 300)])
    if op == "wdec":
        while True:
            B, W, past = _log(rng, 1, 256), _log(rng, 1, 8192), _log(rng, 1, 40000)
            if B * H_kv * D * (W + S) <= 256 * 8 * 128 * 4100:
                break
        return dict(op=op, kv=kv, B=B, H=H, H_kv=H_kv, D=D, bs=bs, W=W, S=S,
                    past_lo=rng.choice([0, past // 2, past]), past_hi=past, lens=lens)
    top = 256 if kv == "f32" else 4096
    while True:
        B, n, past = _log(rng, 1, 48), _log(rng, 1, top), _log(rng, 1, 4 * top)
        # the plain form's padded scores and gathered caches stay within the listed largest
        if (B * H * n * (n + past) <= 32 * 4096 * 16384
                and B * H_kv * D * (n + past) <= 48 * 8 * 128 * 8192):
            break
    return dict(op=op, kv=kv, B=B, H=H, H_kv=H_kv, D=D, bs=bs, W=_log(rng, 1, 8192), S=S,
                n_lo=max(1, n // rng.choice([1, 4, 20])), n_hi=n,
                past_lo=rng.choice([0, past // 2, past]), past_hi=past, lens=lens)


def _lengths(case):
    """(new tokens, tokens before them) of each request."""
    r = np.random.RandomState(case["lens"])
    B = case["B"]
    lo, hi = case.get("n_lo", 1), case.get("n_hi", 1)
    n = r.randint(lo, hi + 1, B).astype(np.int64)
    if case["op"] == "verify":
        return n, np.zeros_like(n)
    return n, r.randint(case["past_lo"], case["past_hi"] + 1, B).astype(np.int64)


def _blocks(lengths, bs):
    return (lengths + bs - 1) // bs


def _inverse_frequencies(case):
    """Radians per position of each rotated pair, in 64 bits; with ``stretch`` s, pairs that turn
    less than once within 4096 positions are slowed by s, those that turn 32 times or more are
    kept, and those between are mixed linearly in their turns."""
    f = 10000.0 ** (-np.arange(0, case["R"], 2) / case["R"])
    if case["stretch"] == 1.0:
        return f
    keep = np.clip((4096 * f / (2 * math.pi) - 1) / 31, 0, 1)
    return f * keep + f / case["stretch"] * (1 - keep)


def _attention_factor(case):
    return 1.0 if case["stretch"] == 1.0 else 0.1 * math.log(case["stretch"]) + 1.0


# ------------------------------------------------------------------------------ inputs
def _randn(shape, gen, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _prepare_rope(case, s, rng, gen):
    T, H, H_kv, D, bs, kv = (case[k] for k in ("T", "H", "H_kv", "D", "bs", "kv"))
    dt = _DT[kv]
    if case["fused"]:  # slices of one projection's output
        x = _randn((T, H + 2 * H_kv, D), gen, dt)
        s["q"], s["k"], s["v"] = x[:, :H], x[:, H:H + H_kv], x[:, H + H_kv:]
    else:
        s["q"], s["k"], s["v"] = (_randn((T, h, D), gen, dt) for h in (H, H_kv, H_kv))
    s["q_weight"] = s["k_weight"] = None
    if case["norm"]:
        s["q_weight"] = (1 + 0.2 * _randn((D,), gen, torch.float32)).to(dt)
        s["k_weight"] = (1 + 0.2 * _randn((D,), gen, torch.float32)).to(dt)
    NB = _blocks(T, bs) * 2 + 8
    s["k_scale"], s["v_scale"] = (0.03125, 0.046875) if kv == "fp8" else (1.0, 1.0)
    for name in ("k_cache", "v_cache"):
        c = _randn((NB, bs, H_kv, D), gen, dt)
        s[name] = c.to(torch.float8_e4m3fn) if kv == "fp8" else c
    live = T - case["pad"]
    slots = np.full(T, -1)
    slots[:live] = rng.permutation(NB * bs)[:live]
    s.update(slots=_i32(slots), live=live, positions=_i32(rng.randint(0, case["far"], T)),
             inv_freq=torch.from_numpy(_inverse_frequencies(case)).cuda(),
             factor=_attention_factor(case))
    if own:
        import paged_decode_attention_02_gb300 as pda
        s["freqs"] = pda.rope_frequencies(
            case["R"], 10000.0, stretch=case["stretch"], original_length=4096, device="cuda")


def _prepare_verify(case, s, gen):
    n, V, dt = s["n"], case["V"], _DT[case["kv"]]
    T = int(n.sum())
    x = torch.randn((T, V), generator=gen, device="cuda") * 2.5
    y = x + 0.7 * torch.randn((T, V), generator=gen, device="cuda")
    p, q = torch.softmax(x, 1), torch.softmax(y, 1)
    if case["cut"]:  # only the likeliest tokens are left
        for z in (p, q):
            z.masked_fill_(z < z.amax(1, keepdim=True) * 1e-3, 0).div_(z.sum(1, keepdim=True))
    drawn = torch.multinomial(q, 1, generator=gen)[:, 0]
    s["tokens"] = torch.cat([drawn[:1], drawn[:-1]]).int()  # row r judges token r + 1
    s["p"], s["q"] = p.to(dt), q.to(dt) if case["drafted"] else None
    s["accept_u"] = torch.rand(T, generator=gen, device="cuda")
    s["sample_u"] = torch.rand(case["B"], generator=gen, device="cuda")
    s["query_start"] = _i32(np.concatenate([[0], np.cumsum(n)]))


def _prepare_window(case, s, rng, gen):
    n, L, bs, B = s["n"], s["L"], case["bs"], case["B"]
    H, H_kv, D, kv = case["H"], case["H_kv"], case["D"], case["kv"]
    # the blocks that some of the new tokens see; the others have been freed
    nblk = _blocks(L, bs)
    mb = int(nblk.max())
    j = np.arange(mb)[None, :]
    first = np.maximum(L - n - case["W"] + 1, 0)[:, None]
    held = (j < nblk[:, None]) & ((j * bs < case["S"]) | (j * bs + bs > first))
    NB = int(held.sum()) + 8
    table = np.full((B, mb), -1)
    table[held] = rng.permutation(NB)[:int(held.sum())]
    s.update(tables=_i32(table), lens=_i32(L), NB=NB)
    T = int(n.sum())
    s["q"] = _randn((T, H, D), gen, _DT[kv])
    s["k_scale"], s["v_scale"] = (0.03125, 0.046875) if kv == "fp8" else (1.0, 1.0)
    for name in ("k", "v"):
        if kv == "fp8":
            x = _randn((NB, bs, H_kv, D), gen, torch.float32) / s[name + "_scale"]
            s[name] = x.to(torch.float8_e4m3fn)
        else:
            s[name] = _randn((NB, bs, H_kv, D), gen, _DT[kv])
    s["query_start"] = _i32(np.concatenate([[0], np.cumsum(n)]))
    s["n_max"], s["L_max"], s["scale"] = int(n.max()), int(L.max()), D ** -0.5
    if own:
        import paged_decode_attention_02_gb300 as pda
        s["workspace"] = (
            pda.alloc_workspace(B, H, H_kv, D, bs, s["k"].dtype) if case["op"] == "wdec" else
            pda.alloc_chunk_workspace(B, T, H, H_kv, D, bs, s["k"].dtype))


def prepare(case, seed):
    rng = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "rope":
        _prepare_rope(case, s, rng, gen)
        return s
    s["n"], past = _lengths(case)
    s["L"] = s["n"] + past
    if case["op"] == "verify":
        _prepare_verify(case, s, gen)
    else:
        _prepare_window(case, s, rng, gen)
    return s


# ------------------------------------------------------------------------------ plain forms
def _rope_plain(s):
    c = s["case"]
    R, live = c["R"], s["live"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos = (angle.cos() * s["factor"]).float()[:, None]
    sin = (angle.sin() * s["factor"]).float()[:, None]

    def turned(x, weight):
        c_x, s_x = cos[:x.shape[0]], sin[:x.shape[0]]
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * weight.float()
        x, rest = x[..., :R], x[..., R:]
        if c["half"]:
            a, b = x[..., :R // 2], x[..., R // 2:]
            x = torch.cat([a * c_x - b * s_x, b * c_x + a * s_x], -1)
        else:
            a, b = x[..., 0::2], x[..., 1::2]
            x = torch.stack([a * c_x - b * s_x, b * c_x + a * s_x], -1).flatten(-2)
        return torch.cat([x, rest], -1)

    slots = s["slots"][:live].long()
    new = (turned(s["k"][:live], s["k_weight"]), s["v"][:live].float())
    for cache, x, scale in zip((s["k_cache"], s["v_cache"]), new, (s["k_scale"], s["v_scale"])):
        if c["kv"] == "fp8":
            x = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            cache = cache.view(torch.uint8)
        cache.view(-1, c["H_kv"], c["D"])[slots] = x.to(cache.dtype)
    return turned(s["q"], s["q_weight"]).to(s["q"].dtype), s["k_cache"], s["v_cache"]


def _wdec_plain(s):
    c = s["case"]
    B, H_kv, D, bs, W, S = (c[k] for k in ("B", "H_kv", "D", "bs", "W", "S"))
    G = c["H"] // H_kv
    L = s["lens"].long()[:, None]
    # the first S tokens, then the window's that are not among them
    dev = L.device
    first = torch.arange(S, device=dev).expand(B, S)
    last = L - W + torch.arange(W, device=dev)
    t = torch.cat([first, last], 1)
    seen = torch.cat([first < L, last >= S], 1)
    t = torch.where(seen, t, 0)
    block = s["tables"].long().gather(1, t // bs).clamp(min=0)
    k, v = s["k"][block, t % bs].float(), s["v"][block, t % bs].float()
    q = s["q"].float().view(B, H_kv, G, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * (s["scale"] * s["k_scale"])
    x = x.masked_fill(~seen[:, None, None], float("-inf"))
    x = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(x, v.transpose(1, 2)) * (s["v_scale"] / x.sum(-1, keepdim=True))
    return o.view(B, c["H"], D).to(s["q"].dtype)


def _wchunk_plain(s):
    c = s["case"]
    H_kv, D, bs, B = c["H_kv"], c["D"], c["bs"], c["B"]
    G, n_max, L_max = c["H"] // H_kv, s["n_max"], s["L_max"]
    dev = s["q"].device
    start, L = s["query_start"].long(), s["lens"].long()
    n = start[1:] - start[:-1]
    i = torch.arange(n_max, device=dev)
    row = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(B, n_max, H_kv, G, D).permute(0, 2, 3, 1, 4)
    nb = (L_max + bs - 1) // bs
    at = s["tables"][:, :nb].long().clamp(min=0)
    k = s["k"][at].float().view(B, nb * bs, H_kv, D)[:, :L_max].permute(0, 2, 3, 1)
    v = s["v"][at].float().view(B, nb * bs, H_kv, D)[:, :L_max].permute(0, 2, 1, 3)
    x = torch.matmul(q.reshape(B, H_kv, G * n_max, D), k) * (s["scale"] * s["k_scale"])
    x = x.view(B, H_kv, G, n_max, L_max)
    t = torch.arange(L_max, device=dev)
    last = ((L - n)[:, None] + i)[:, :, None]
    hidden = (t > last) | ((t <= last - c["W"]) & (t >= c["S"]))
    x = x.masked_fill(hidden[:, None, None], float("-inf"))
    # rows behind a request's last token are dropped below, whatever they see
    x = torch.exp(x - x.amax(-1, keepdim=True))
    total = x.sum(-1)
    o = torch.matmul(x.view(B, H_kv, G * n_max, L_max), v).view(B, H_kv, G, n_max, D)
    o = o * (s["v_scale"] / total[..., None])
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n_max, H_kv * G, D)
    # each token's place among the padded rows
    T = s["q"].shape[0]
    r = torch.arange(T, device=dev)
    b = (r[:, None] >= start[None, 1:]).sum(1)
    return o[b, r - start[b]].to(s["q"].dtype)


def _verify_plain(s):
    p, q, tokens = s["p"], s["q"], s["tokens"].long()
    start = s["query_start"].long()
    n = start[1:] - start[:-1]
    T, V = p.shape
    i = torch.arange(int(s["n"].max()), device=p.device)
    row = (start[:-1, None] + i).clamp(max=T - 1)
    judged = i < (n - 1)[:, None]
    token = tokens[(row + 1).clamp(max=T - 1)]
    pt = p[row, token].float()
    qt = q[row, token].float() if q is not None else torch.ones_like(pt)
    ok = (s["accept_u"][row] * qt < pt) & judged
    accepted = ok.int().cumprod(1).sum(1)
    at = start[:-1] + accepted
    rejected = accepted < n - 1
    weight = p[at].float()
    if q is not None:
        left = (weight - q[at].float()).clamp(min=0)
    else:
        left = torch.where(torch.arange(V, device=p.device) ==
                           tokens[(at + 1).clamp(max=T - 1)][:, None], 0.0, weight)
    some = rejected & (left.sum(1) > 0)
    end = torch.where(some[:, None], left, weight).double().cumsum(1)
    drawn = (end <= s["sample_u"].double()[:, None] * end[:, -1:]).sum(1)
    return accepted.int(), drawn.int()


# ------------------------------------------------------------------------------ own calls
def _rope_own(s):
    import paged_decode_attention_02_gb300 as pda
    q_out = torch.empty(s["q"].shape, dtype=s["q"].dtype, device=s["q"].device)
    pda.qk_norm_rope_append(q_out, s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"],
                            s["positions"], s["freqs"], q_weight=s["q_weight"],
                            k_weight=s["k_weight"], eps=_EPS,
                            interleaved=not s["case"]["half"], attention_factor=s["factor"],
                            k_scale=s["k_scale"], v_scale=s["v_scale"])
    return q_out, s["k_cache"], s["v_cache"]


def _window_own(s):
    import paged_decode_attention_02_gb300 as pda
    c = s["case"]
    out = torch.empty_like(s["q"])
    args = [out, s["q"], s["k"], s["v"], s["tables"], s["lens"]]
    if c["op"] == "wchunk":
        args.append(s["query_start"])
    args += [s["L_max"], s["scale"]]
    calls = {"wdec": (pda.paged_decode_attention, pda.paged_decode_attention_fp8),
             "wchunk": (pda.paged_chunk_attention, pda.paged_chunk_attention_fp8)}[c["op"]]
    if c["kv"] == "fp8":
        args += [s["k_scale"], s["v_scale"]]
    return calls[c["kv"] == "fp8"](*args, workspace=s["workspace"], window=c["W"],
                                   sinks=c["S"])


def _verify_own(s):
    import paged_decode_attention_02_gb300 as pda
    accepted = torch.empty(s["case"]["B"], dtype=torch.int32, device=s["p"].device)
    drawn = torch.empty_like(accepted)
    pda.verify_drafts(accepted, drawn, s["p"], s["q"], s["tokens"], s["query_start"],
                      s["accept_u"], s["sample_u"])
    return accepted, drawn


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _rope_own, "wdec": _window_own, "wchunk": _window_own,
                "verify": _verify_own}[op](state)
    return {"rope": _rope_plain, "wdec": _wdec_plain, "wchunk": _wchunk_plain,
            "verify": _verify_plain}[op](state)


# ------------------------------------------------------------------------------ 64 bits
def _rope_exact(s):
    """The rotation as a product of complex numbers."""
    c = s["case"]
    R, live = c["R"], s["live"]
    turn = torch.polar(torch.full_like(s["inv_freq"], s["factor"]).expand(c["T"], -1),
                       s["positions"].double()[:, None] * s["inv_freq"])

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = x / (x.square().mean(-1, keepdim=True) + _EPS).sqrt() * weight.double()
        pairs = x[..., :R].unflatten(-1, (2, -1) if c["half"] else (-1, 2))
        axis = -2 if c["half"] else -1
        z = torch.complex(pairs.select(axis, 0), pairs.select(axis, 1)) * turn[:x.shape[0], None]
        return torch.cat([torch.stack([z.real, z.imag], axis).flatten(-2), x[..., R:]], -1)

    out = [turned(s["q"], s["q_weight"])]
    for name, x in (("k", turned(s["k"][:live], s["k_weight"])), ("v", s["v"][:live].double())):
        cache = s[name + "_cache"].double()
        if c["kv"] == "fp8":
            x = (x / s[name + "_scale"]).clamp(-448, 448)
        cache.view(-1, c["H_kv"], c["D"])[s["slots"][:live].long()] = x
        out.append(cache)
    return tuple(out)


def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers: the plain form's are compared as they are
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _rope_exact(s)
    G, D, bs, W, S = case["H"] // case["H_kv"], case["D"], case["bs"], case["W"], case["S"]
    ends = np.cumsum(s["n"]).tolist()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, end in enumerate(ends):
        first = ends[b - 1] if b else 0
        L, n = int(s["L"][b]), end - first
        lowest = max(0, L - n - W + 1)
        head = torch.arange(min(S, lowest), device="cuda")
        t = torch.cat([head, torch.arange(lowest, L, device="cuda")])
        blocks = s["tables"][b].long()[t // bs]
        k = s["k"][blocks, t % bs].double() * s["k_scale"]
        v = s["v"][blocks, t % bs].double() * s["v_scale"]
        for lo in range(0, n, 2048):
            hi = min(n, lo + 2048)
            p = torch.arange(L - n + lo, L - n + hi, device="cuda")[:, None]
            hidden = (t > p) | ((t <= p - W) & (t >= S))
            mask = torch.zeros(hidden.shape, dtype=torch.float64,
                               device="cuda").masked_fill_(hidden, -math.inf)
            for h in range(case["H_kv"]):
                q = s["q"][first + lo:first + hi, h * G:h * G + G].double()
                x = torch.einsum("ngd,td->gnt", q, k[:, h]) * s["scale"] + mask
                o = torch.softmax(x, -1) @ v[:, h]
                out[first + lo:first + hi, h * G:h * G + G] = o.transpose(0, 1)
    return out


def work(case):
    """Bytes read once and written once, and operations, of one pass."""
    e_q = 4 if case["kv"] == "f32" else 2
    e_kv = {"f32": 4, "fp8": 1}.get(case["kv"], 2)
    if case["op"] == "rope":
        T, H, H_kv, D = case["T"], case["H"], case["H_kv"], case["D"]
        live = T - case["pad"]
        return {"bytes": (2 * T * H + 2 * live * H_kv) * D * e_q + 2 * live * H_kv * D * e_kv
                + 8 * T + 4 * case["R"] + (2 * D * e_q if case["norm"] else 0),
                "flops": (T * H + live * H_kv) * (3 * case["R"] + (4 * D if case["norm"] else 0))}
    n, past = _lengths(case)
    B = case["B"]
    if case["op"] == "verify":
        # of the probabilities, a request needs its drafted tokens' and the row (two where a
        # draft is turned down) that its next token is drawn from
        rows = 2 if case["drafted"] else 1
        return {"bytes": B * case["V"] * rows * e_q + 16 * int(n.sum()) + 16 * B + 4,
                "flops": B * case["V"] * (rows + 1)}
    L, bs, W, S = n + past, case["bs"], case["W"], case["S"]
    lowest = np.maximum(past - W + 1, 0)
    keys = L - lowest + np.minimum(S, lowest)
    blocks = _blocks(L, bs) - lowest // bs + np.minimum(_blocks(np.minimum(S, L), bs),
                                                       lowest // bs)
    pairs = 0
    for x, y in zip(n.tolist(), past.tolist()):
        p = np.arange(y, x + y)
        low = np.maximum(p - W + 1, 0)
        pairs += int((p + 1 - low + np.minimum(S, low)).sum())
    return {"bytes": int(2 * n.sum() * case["H"] * case["D"] * e_q
                         + 2 * keys.sum() * case["H_kv"] * case["D"] * e_kv
                         + 4 * blocks.sum() + 8 * B + 4),
            "flops": 4 * case["H"] * case["D"] * pairs}
