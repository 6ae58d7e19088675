"""Measured cases of the paged-cache step operators: attention of a chunk of new tokens over
the paged cache, block tables assigned from request lengths, and slot maps.

Every case names its operator (``op``) and the ranges its request lengths are drawn from;
``lens`` seeds those lengths, so a case always has the same amount of work, while the values,
the block permutation and the free list come from the seed given to ``prepare``.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "fp8": torch.bfloat16}


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest attention call: the repository's tiny fp32 shape, four short chunks
        dict(name="attn_tiny_f32", op="attn", kv="f32", B=4, H=2, H_kv=2, D=64, bs=16,
             n_lo=1, n_hi=33, past_lo=0, past_hi=80, lens=1),
        # one request's short follow-up turn over a short history: latency
        dict(name="attn_turn_bf16", op="attn", kv="bf16", B=1, H=32, H_kv=8, D=128, bs=16,
             n_lo=17, n_hi=17, past_lo=586, past_hi=586, lens=2),
        # verification of drafted tokens in a decode batch: few rows, long histories
        dict(name="attn_verify_bf16", op="attn", kv="bf16", B=32, H=32, H_kv=8, D=128, bs=16,
             n_lo=1, n_hi=8, past_lo=512, past_hi=8192, lens=3),
        # a chunk of a long prompt over what earlier chunks left in the cache
        dict(name="attn_chunk_bf16", op="attn", kv="bf16", B=1, H=32, H_kv=8, D=128, bs=16,
             n_lo=4096, n_hi=4096, past_lo=12288, past_hi=12288, lens=4),
        # fresh prompts of ragged length, one kv-head per query head (the 13B shape)
        dict(name="attn_prompts_f16", op="attn", kv="f16", B=6, H=40, H_kv=40, D=128, bs=16,
             n_lo=300, n_hi=1900, past_lo=0, past_hi=0, lens=5),
        # chunks over a prefix that other requests share, small heads, large blocks
        dict(name="attn_prefix_d64_bf16", op="attn", kv="bf16", B=4, H=16, H_kv=2, D=64, bs=64,
             n_lo=129, n_hi=1000, past_lo=1500, past_hi=6000, lens=6),
        # chunks over an 8-bit cache
        dict(name="attn_chunk_fp8", op="attn", kv="fp8", B=3, H=32, H_kv=8, D=128, bs=16,
             n_lo=500, n_hi=2048, past_lo=1000, past_hi=8000, lens=7),
        # one decode step of the 256-request batch: one row in sixteen needs a block
        dict(name="assign_decode", op="assign", B=256, bs=16, lo=16, hi=32768, finish=0, admit=0,
             spare=125, lens=8),
        # a scheduling step: a quarter of the rows end, a quarter are admitted
        dict(name="assign_admit", op="assign", B=512, bs=16, lo=16, hi=32768, finish=25,
             admit=25, spare=125, lens=9),
        # one decode step's slots
        dict(name="slots_decode", op="slots", B=256, bs=16, n_lo=1, n_hi=1, past_lo=15,
             past_hi=32767, pad=0, lens=10),
        # the slots of a large prefill batch, with padding rows behind the last token
        dict(name="slots_prefill", op="slots", B=96, bs=16, n_lo=16, n_hi=4096, past_lo=0,
             past_hi=8192, pad=1000, lens=11),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "assign", "slots"])
    lens = rng.randrange(1 << 20)
    bs = rng.choice([16, 16, 32, 64, 128, 256])
    if op == "assign":
        lo = _log(rng, 1, 512)
        return dict(op=op, B=_log(rng, 1, 512), bs=bs, lo=lo, hi=lo + _log(rng, 16, 32768),
                    finish=rng.choice([0, 10, 50]), admit=rng.choice([0, 20, 50]),
                    spare=rng.choice([60, 100, 125]), lens=lens)
    if op == "slots":
        n = _log(rng, 1, 4096)
        past = _log(rng, 1, 16384)
        return dict(op=op, B=_log(rng, 1, 96), bs=bs, n_lo=max(1, n // rng.choice([1, 3, 10])),
                    n_hi=n, past_lo=rng.choice([0, past // 2]), past_hi=past,
                    pad=rng.choice([0, 77]), lens=lens)
    kv = rng.choice(["bf16", "bf16", "f16", "fp8", "f32"])
    H, H_kv = rng.choice([(32, 32), (32, 8), (40, 40), (16, 2), (8, 1), (12, 6)])
    D = rng.choice([64, 128, 128])
    top = 256 if kv == "f32" else 4096
    while True:
        B, n, past = _log(rng, 1, 48), _log(rng, 1, top), _log(rng, 1, 4 * top)
        # the plain form's padded scores and gathered caches stay within the listed largest
        if (B * H * n * (n + past) <= 32 * 4096 * 16384
                and B * H_kv * D * (n + past) <= 48 * 8 * 128 * 8192):
            break
    return dict(op="attn", kv=kv, B=B, H=H, H_kv=H_kv, D=D, bs=bs,
                n_lo=max(1, n // rng.choice([1, 4, 20])), n_hi=n,
                past_lo=rng.choice([0, past // 2, past]), past_hi=past, lens=lens)


def _lengths(case):
    """(new tokens, tokens before them) of each request, or (old, new) lengths for assign."""
    r = np.random.RandomState(case["lens"])
    B = case["B"]
    if case["op"] == "assign":
        def some():
            x = np.exp(r.uniform(math.log(case["lo"]), math.log(case["hi"]), B))
            return np.clip(x.astype(np.int64), case["lo"], case["hi"])
        old, fresh = some(), some()
        u = r.uniform(0, 100, B)
        ends, admits = u < case["finish"], u >= 100 - case["admit"]
        new = np.where(ends, 0, np.where(admits, fresh, old + 1))
        return np.where(admits, 0, old), new
    n = r.randint(case["n_lo"], case["n_hi"] + 1, B).astype(np.int64)
    past = r.randint(case["past_lo"], case["past_hi"] + 1, B).astype(np.int64)
    return n, past


def _blocks(lengths, bs):
    return (lengths + bs - 1) // bs


# ------------------------------------------------------------------------------ inputs
def _randn(shape, gen, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def prepare(case, seed):
    rng = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    bs, B = case["bs"], case["B"]
    a, b = _lengths(case)
    s = dict(case=case)
    if case["op"] == "assign":
        held, need = _blocks(a, bs), _blocks(b, bs)
        mb = int(max(held.max(), need.max()))
        grow = int(np.maximum(need - held, 0).sum())
        back = int(np.maximum(held - need, 0).sum())
        free = max(1, (grow * case["spare"]) // 100 - back)
        NB = int(held.sum()) + free
        perm = rng.permutation(NB)
        table = np.full((B, mb), -1)
        table[np.arange(mb)[None, :] < held[:, None]] = perm[free:]
        room = np.full(NB, -1)
        room[:free] = perm[:free]
        s.update(tables=_i32(table), held=_i32(held), free_list=_i32(room),
                 free_count=_i32([free]), lens=_i32(b), NB=NB)
        return s
    n, L = a, a + b
    nblk = _blocks(L, bs)
    NB = int(nblk.sum()) + 8
    mb = int(nblk.max())
    table = np.full((B, mb), -1)
    table[np.arange(mb)[None, :] < nblk[:, None]] = rng.permutation(NB)[:int(nblk.sum())]
    s.update(tables=_i32(table), lens=_i32(L), NB=NB)
    if case["op"] == "slots":
        s.update(query_lens=_i32(n), N=int(n.sum()) + case["pad"])
        return s
    H, H_kv, D, kv = case["H"], case["H_kv"], case["D"], case["kv"]
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
        s["workspace"] = pda.alloc_chunk_workspace(B, T, H, H_kv, D, bs, s["k"].dtype)
    return s


# ------------------------------------------------------------------------------ plain forms
def _attn_plain(s):
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
    last = (L - n)[:, None] + i
    x = x.masked_fill((t > last[:, :, None])[:, None, None], float("-inf"))
    x = torch.exp(x - x.amax(-1, keepdim=True))
    total = x.sum(-1)
    o = torch.matmul(x.view(B, H_kv, G * n_max, L_max), v).view(B, H_kv, G, n_max, D)
    o = o * (s["v_scale"] / total[..., None])
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n_max, H_kv * G, D)
    return o[i < n[:, None]].to(s["q"].dtype)


def _assign_plain(s):
    bs, NB = s["case"]["bs"], s["NB"]
    table, held, free = s["tables"], s["held"].long(), s["free_count"].long()
    need = (s["lens"].long() + bs - 1) // bs
    j = torch.arange(table.shape[1], device=table.device)
    back, grow = (held - need).clamp(min=0), (need - held).clamp(min=0)
    back_end, grow_end = back.cumsum(0), grow.cumsum(0)
    room = free + back_end[-1]
    fits = grow_end <= room
    # the blocks given back go onto the stack in row order
    gives = (j >= need[:, None]) & (j < held[:, None])
    to = torch.where(gives, free + (back_end - back - need)[:, None] + j, NB)
    stack = torch.cat([s["free_list"], s["free_list"].new_zeros(1)])
    stack[to.view(-1)] = torch.where(gives, table, 0).view(-1)
    stack = stack[:NB]
    # and the growing rows take theirs from its top
    takes = (j >= held[:, None]) & (j < need[:, None]) & fits[:, None]
    order = (grow_end - grow - held)[:, None] + j
    out = torch.where(takes, stack[(room - 1 - order).clamp(0, NB - 1)], table)
    taken = torch.where(fits, grow_end, 0).amax()
    held_out = torch.where((grow > 0) & ~fits, held, need)
    return out, held_out.int(), (room - taken).int(), stack


def _slots_plain(s):
    bs, N = s["case"]["bs"], s["N"]
    n, L = s["query_lens"].long(), s["lens"].long()
    end = n.cumsum(0)
    start = torch.cat([end.new_zeros(1), end])
    t = torch.arange(N, device=n.device)
    b = (t[:, None] >= end[None, :]).sum(1).clamp(max=len(n) - 1)
    p = (L - n)[b] + t - start[b]
    inside = t < end[-1]
    p = torch.where(inside, p, 0)
    slot = s["tables"][b, p // bs].long() * bs + p % bs
    return torch.where(inside, slot, -1).int(), start.int()


# ------------------------------------------------------------------------------ own calls
def _attn_own(s):
    import paged_decode_attention_02_gb300 as pda
    out = torch.empty_like(s["q"])
    common = (s["tables"], s["lens"], s["query_start"], s["L_max"], s["scale"])
    if s["case"]["kv"] == "fp8":
        return pda.paged_chunk_attention_fp8(out, s["q"], s["k"], s["v"], *common, s["k_scale"],
                                             s["v_scale"], workspace=s["workspace"])
    return pda.paged_chunk_attention(out, s["q"], s["k"], s["v"], *common,
                                     workspace=s["workspace"])


def _assign_own(s):
    import paged_decode_attention_02_gb300 as pda
    held, count = torch.empty_like(s["held"]), torch.empty_like(s["free_count"])
    pda.kv_assign_blocks(s["tables"], s["held"], s["free_list"], s["free_count"], s["lens"],
                         s["case"]["bs"], blocks_held_out=held, free_count_out=count)
    return s["tables"], held, count, s["free_list"]


def _slots_own(s):
    import paged_decode_attention_02_gb300 as pda
    dev = s["lens"].device
    slots = torch.empty(s["N"], dtype=torch.int32, device=dev)
    start = torch.empty(s["case"]["B"] + 1, dtype=torch.int32, device=dev)
    pda.kv_build_slots(slots, start, s["query_lens"], s["lens"], s["tables"], s["case"]["bs"],
                       s["NB"])
    return slots, start


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attn": _attn_own, "assign": _assign_own, "slots": _slots_own}[op](state)
    return {"attn": _attn_plain, "assign": _assign_plain, "slots": _slots_plain}[op](state)


# ------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    if case["op"] != "attn":
        return None  # whole numbers: the plain form's are compared as they are
    s = prepare(case, seed)
    G, D = case["H"] // case["H_kv"], case["D"]
    ends = np.cumsum(_lengths(case)[0]).tolist()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, end in enumerate(ends):
        first = ends[b - 1] if b else 0
        L, n = int(s["lens"][b]), end - first
        blocks = s["tables"][b, :-(-L // case["bs"])].long()
        k = s["k"][blocks].double().reshape(-1, case["H_kv"], D)[:L] * s["k_scale"]
        v = s["v"][blocks].double().reshape(-1, case["H_kv"], D)[:L] * s["v_scale"]
        for h in range(case["H"]):
            for lo in range(0, n, 2048):
                hi = min(n, lo + 2048)
                seen = L - n + hi
                q = s["q"][first + lo:first + hi, h].double()
                x = (q @ k[:seen, h // G].T) * s["scale"]
                x += torch.full_like(x, -math.inf).triu_(L - n + lo + 1)
                out[first + lo:first + hi, h] = torch.softmax(x, 1) @ v[:seen, h // G]
    return out


def work(case):
    """Bytes read once and written once, and operations, of one pass."""
    bs, B = case["bs"], case["B"]
    a, b = _lengths(case)
    if case["op"] == "assign":
        moved = int(np.abs(_blocks(b, bs) - _blocks(a, bs)).sum())
        return {"bytes": 12 * B + 8 + 8 * moved, "flops": 0}
    n, L = a, a + b
    if case["op"] == "slots":
        entries = int((_blocks(L, bs) - (L - n) // bs).sum())
        return {"bytes": 12 * B + 4 + 4 * entries + 4 * int(n.sum() + case["pad"]), "flops": 0}
    e_q = 4 if case["kv"] == "f32" else 2
    e_kv = {"f32": 4, "fp8": 1}.get(case["kv"], 2)
    pairs = int((n * (L - n) + n * (n + 1) // 2).sum())
    return {"bytes": int(2 * n.sum() * case["H"] * case["D"] * e_q
                         + 2 * L.sum() * case["H_kv"] * case["D"] * e_kv
                         + 4 * _blocks(L, bs).sum() + 8 * B + 4),
            "flops": 4 * case["H"] * case["D"] * pairs}
