"""Cases of the serving and position operators: rotary positions, the paged KV cache's append, attention over
the paged cache, and attention of a batch that shares a prefix.

``run`` computes them in plain torch (``own`` false) or through the package's entry points (``own`` true).
"""
import math

import torch

own = False

_GOLD = 0.6180339887498949  # spreads the sequences' lengths evenly, whatever their number


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _rope(name, **kw):
    c = dict(op="rope", B=1, H=12, Hk=12, N=256, d=64, rot=64, interleaved=False, backward=False, base=10000.0,
             scaling="none", factor=1.0, offset=0, packed_positions=False)
    c.update(kw)
    c["name"] = name
    return c


def _append(name, **kw):
    c = dict(op="append", B=16, H=32, Hk=8, T=1, d=128, rot=128, interleaved=False, base=500000.0, scaling="none",
             factor=1.0, offset=0, page=16, token_major=False, context=1024, ragged_new=False)
    c.update(kw)
    c["name"] = name
    return c


def _paged(name, **kw):
    c = dict(op="paged", B=8, H=12, Hk=12, T=1, d=64, page=16, token_major=False, context=1024, left=-1, right=0,
             ragged_new=False)
    c.update(kw)
    c["name"] = name
    return c


def _prefix(name, **kw):
    c = dict(op="prefix", B=4, H=12, Hk=12, T=1, d=64, page=16, token_major=False, prefix=1000, context=100,
             ragged_new=False)
    c.update(kw)
    c["name"] = name
    return c


def listed():
    return [
        # one short prompt of the GPT-2-small-shaped heads: a call whose cost is its launch
        _rope("rope_prompt_256"),
        # a training step's queries and keys, from the packed token-major projection, grouped heads
        _rope("rope_train_8192", B=4, H=32, Hk=8, N=8192, d=128, rot=128, base=500000.0),
        # its backward in the interleaved layout, half of the head rotated, documents packed in a row, odd length
        _rope("rope_bwd_packed_4099", B=3, H=16, Hk=16, N=4099, d=128, rot=64, interleaved=True, backward=True,
              scaling="by_parts", factor=8.0, packed_positions=True),
        # one decoded token for each of 16 sequences
        _append("append_decode_16"),
        # a chunk of the prompts of 4 sequences, of different lengths, far into long contexts
        _append("append_chunk_4x2048", B=4, T=2048, page=64, context=4000, ragged_new=True, offset=100000,
                scaling="linear", factor=4.0),
        # decoding 8 short sequences, one KV head per query head: a call of a few microseconds
        _paged("decode_8x1024_d64"),
        # decoding 32 sequences of 1 to 8192 tokens, grouped heads: the bulk of serving
        _paged("decode_32x8192", B=32, H=32, Hk=8, d=128, context=8192),
        # a prompt's next 256 tokens over what is in the cache already
        _paged("chunk_2x256_over_8192", B=2, H=32, Hk=8, T=256, d=128, page=64, context=8192, ragged_new=True),
        # checking 4 drafted tokens under a sliding window in long contexts; token-major pages, odd length
        _paged("draft_window_16x32000", B=16, H=32, Hk=4, T=4, d=128, page=128, token_major=True, context=31999,
               left=4095),
        # four short continuations of one prompt
        _prefix("prefix_4x1000_d64"),
        # 64 continuations of an 8192-token prompt: 256 query rows for each KV head
        _prefix("prefix_64x8192", B=64, H=32, Hk=8, d=128, prefix=8192, context=512),
        # drafted tokens behind a very long document, a KV head per query head
        _prefix("prefix_24x32000_draft", B=24, H=16, Hk=16, T=3, d=128, page=32, prefix=32000, context=301),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 0.25 / hi)))))


def _cost(c):
    """What a pass of the case moves and computes at most, in units that listed cases bound."""
    if c["op"] == "rope":
        return c["B"] * c["N"] * (c["H"] + c["Hk"]) * c["d"] / (4 * 8192 * 40 * 128)
    cache = c["B"] * c["context"] * c["Hk"] * c["d"] / (32 * 8192 * 8 * 128)
    if c["op"] == "append":
        return max(c["B"] * c["T"] * (c["H"] + 2 * c["Hk"]) * c["d"] / (4 * 2048 * 48 * 128), 2 * cache)
    rows = c["B"] * c["H"] * c["T"]
    if c["op"] == "paged":
        return max(cache, rows * c["context"] / (2 * 32 * 256 * 8192))
    shared = c["prefix"] * c["Hk"] * c["d"] / (32000 * 16 * 128)
    return max(cache * 8, shared, rows * (c["prefix"] + c["context"]) / (24 * 16 * 3 * 32301))


def draw(rng):
    while True:
        op = rng.choice(["rope", "append", "paged", "prefix"])
        d = rng.choice([64, 128])
        Hk = rng.choice([1, 2, 3, 4, 8, 12, 16])
        H = Hk * rng.choice([1, 1, 2, 4, 5, 8])
        if H > 64:
            continue
        rot = rng.choice([d, d, d // 2, d // 4])
        page = rng.choice([16, 32, 64, 128, 256])
        rotary = dict(d=d, H=H, Hk=Hk, rot=rot, interleaved=rng.random() < 0.5,
                      base=rng.choice([10000.0, 500000.0, 1000000.0]),
                      scaling=rng.choice(["none", "linear", "by_parts"]), factor=rng.choice([2.0, 4.0, 8.0, 32.0]),
                      offset=rng.choice([0, 0, rng.randrange(1, 1000000)]))
        cache = dict(page=page, token_major=rng.random() < 0.4, ragged_new=rng.random() < 0.4)
        if op == "rope":
            c = _rope("", B=rng.randint(1, 8), N=_log(rng, 1, 8192), backward=rng.random() < 0.5,
                      packed_positions=rng.random() < 0.3, **rotary)
        elif op == "append":
            T = rng.choice([1, 1, _log(rng, 2, 2048)])
            c = _append("", B=_log(rng, 1, 128), T=T, context=max(T, _log(rng, 1, 8192)), **rotary, **cache)
        elif op == "paged":
            T = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 2, 256)])
            c = _paged("", B=_log(rng, 1, 128), H=H, Hk=Hk, T=T, d=d, context=max(T, _log(rng, 1, 32000)), **cache)
            if rng.random() < 0.3:
                c["left"] = _log(rng, 1, 8192)
            if rng.random() < 0.15:
                c["right"] = -1  # every cached key, as for an encoder's states
        else:
            T = rng.choice([1, 1, rng.randint(2, 8)])
            c = _prefix("", B=_log(rng, 2, 128), H=H, Hk=Hk, T=T, d=d, prefix=_log(rng, 64, 32000),
                        context=max(T, _log(rng, 1, 1024)), **cache)
        del c["name"]
        if _cost(c) <= 1.0:
            return c


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _lengths(case):
    """Tokens of each sequence once the new ones are in: the first has `context`, the others spread below it."""
    lo, hi = case["T"], case["context"]
    return [lo + int((hi - lo) * ((1.0 + b * _GOLD) % 1.0 if b else 1.0)) for b in range(case["B"])]


def _new(case):
    """New tokens of each sequence: T, or where they differ something from 1 to T."""
    if not case["ragged_new"]:
        return [case["T"]] * case["B"]
    return [1 + int((case["T"] - 1) * ((1.0 + b * _GOLD * _GOLD) % 1.0 if b else 1.0)) for b in range(case["B"])]


def _frequencies(case):
    """Radians per position of each pair, in 64 bits, and the factor on the rotated part."""
    r = case["rot"]
    w = case["base"] ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    if case["scaling"] == "linear":
        return (w / case["factor"]).cuda(), 1.0
    if case["scaling"] == "by_parts":  # far-reaching pairs are stretched, fast ones kept, a ramp between
        turns = 4096.0 * w / (2.0 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        return (w * keep + (w / case["factor"]) * (1.0 - keep)).cuda(), 0.1 * math.log(case["factor"]) + 1.0
    return w.cuda(), 1.0


def _normal(gen, *shape):
    return torch.randn(*shape, device="cuda", dtype=torch.bfloat16, generator=gen)


def _cache(case, gen, lens, extra):
    """A pool of pages in which the sequences' pages lie in any order; `extra` pages more for a prefix."""
    P, Hk, d = case["page"], case["Hk"], case["d"]
    used = [-(-n // P) for n in lens]
    total = sum(used) + extra
    pool = total + 3
    shape = (pool, P, Hk, d) if case["token_major"] else (pool, Hk, P, d)
    k, v = _normal(gen, *shape), _normal(gen, *shape)
    if case["token_major"]:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    order = torch.randperm(pool, device="cuda", generator=gen).to(torch.int32)
    table = torch.full((case["B"], max(used)), -1, dtype=torch.int32)
    at = torch.cat([torch.zeros(1, dtype=torch.int64), torch.tensor(used).cumsum(0)])
    slot = torch.arange(max(used))[None, :].expand(case["B"], -1)
    there = slot < torch.tensor(used)[:, None]
    table[there] = (slot + at[:-1, None])[there].to(torch.int32)
    table = table.cuda()
    table = torch.where(table >= 0, order[table.clamp(min=0).long()], table)
    return k, v, table.contiguous(), order[sum(used):total].contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 + seed)
    s = {"case": case}
    if case["op"] in ("rope", "append"):
        s["w"], s["mag"] = _frequencies(case)
    if case["op"] == "rope":
        B, N, H, Hk, d = (case[x] for x in ("B", "N", "H", "Hk", "d"))
        if case["backward"]:  # gradients as the attention backward leaves them
            s["q"], s["k"] = _normal(gen, B, H, N, d), _normal(gen, B, Hk, N, d)
        else:  # slices of the packed projection
            x = _normal(gen, B, N, (H + 2 * Hk) * d)
            s["q"] = x[..., :H * d].unflatten(-1, (H, d)).transpose(1, 2)
            s["k"] = x[..., H * d:(H + Hk) * d].unflatten(-1, (Hk, d)).transpose(1, 2)
        s["positions"] = None
        if case["packed_positions"]:  # documents of up to 1500 tokens after one another, cut elsewhere for each seed
            cut = torch.randint(0, 1500, (B, 1), device="cuda", generator=gen)
            p = (torch.arange(N, device="cuda")[None, :] + cut) % 1500 + case["offset"]
            s["positions"] = p.to(torch.int32).contiguous()
        return s
    lens = _lengths(case)
    new = _new(case)
    s["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
    s["new"] = torch.tensor(new, dtype=torch.int32).cuda() if case["ragged_new"] else None
    B, T, H, Hk, d = (case[x] for x in ("B", "T", "H", "Hk", "d"))
    extra = -(-case["prefix"] // case["page"]) if case["op"] == "prefix" else 0
    s["k_cache"], s["v_cache"], s["table"], s["prefix_pages"] = _cache(case, gen, lens, extra)
    if case["op"] == "append":
        x = _normal(gen, B, T, (H + 2 * Hk) * d)
        s["q"] = x[..., :H * d].unflatten(-1, (H, d)).transpose(1, 2)
        s["k"] = x[..., H * d:(H + Hk) * d].unflatten(-1, (Hk, d)).transpose(1, 2)
        s["v"] = x[..., (H + Hk) * d:].unflatten(-1, (Hk, d)).transpose(1, 2)
        s["q_out"] = torch.zeros(B, H, T, d, device="cuda", dtype=torch.bfloat16)
    else:
        s["q"] = _normal(gen, B, H, T, d)
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def _rotated(x, positions, w, mag, interleaved, inverse):
    """x [B, H, N, d] turned by positions [B or 1, N] * w, in 32 bits with the angles in 64."""
    a = positions.double()[:, None, :, None] * w
    cos, sin = (mag * a.cos()).float(), (mag * a.sin()).float()
    sin = -sin if inverse else sin
    r = 2 * w.numel()
    x = x.float()
    y = x.clone(memory_format=torch.contiguous_format)
    first, second = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    y[..., first] = x[..., first] * cos - x[..., second] * sin
    y[..., second] = x[..., second] * cos + x[..., first] * sin
    return y.to(torch.bfloat16)


def _plain_rope(s):
    c = s["case"]
    p = s["positions"]
    if p is None:
        p = torch.arange(c["N"], device="cuda")[None, :] + c["offset"]
    return tuple(_rotated(x, p, s["w"], s["mag"], c["interleaved"], c["backward"]) for x in (s["q"], s["k"]))


def _plain_append(s):
    c = s["case"]
    new = s["new"] if s["new"] is not None else torch.full_like(s["lens"], c["T"])
    t = torch.arange(c["T"], device="cuda")[None, :]
    own_pos = (s["lens"] - new)[:, None] + t
    live = t < new[:, None]
    p = own_pos + c["offset"]
    q = _rotated(s["q"], p, s["w"], s["mag"], c["interleaved"], False)
    k = _rotated(s["k"], p, s["w"], s["mag"], c["interleaved"], False)
    s["q_out"].copy_(torch.where(live[:, None, :, None], q, s["q_out"]))
    b, j = live.nonzero(as_tuple=True)
    at = own_pos[b, j]
    page = s["table"][b, at // c["page"]].long()
    s["k_cache"][page, :, at % c["page"]] = k[b, :, j]
    s["v_cache"][page, :, at % c["page"]] = s["v"][b, :, j]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _gathered(cache, table):
    """[B, Hk, L, d] in 32 bits: the pages of each row of the table, one after another."""
    x = cache[table.clamp(min=0).long()]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3).float()


def _softmax(scores):
    """exp(scores - max) and its sum, a row without a visible key giving zeros."""
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = (scores - top).exp()
    return e, e.sum(-1), top.squeeze(-1)


def _visible(c, s, keys, first, left, right):
    """[B, 1, T, keys]: which of `keys` keys of each sequence its new tokens see; `first` positions lie before them."""
    new = s["new"] if s["new"] is not None else torch.full_like(s["lens"], c["T"])
    t = torch.arange(c["T"], device="cuda")
    pos = (s["lens"] - new)[:, None, None] + t[None, :, None] + first
    j = torch.arange(keys, device="cuda")[None, None, :]
    ok = (j < s["lens"][:, None, None] + first) & (t[None, :, None] < new[:, None, None])
    if left >= 0:
        ok = ok & (j >= pos - left)
    if right >= 0:
        ok = ok & (j <= pos + right)
    return ok[:, None]


def _plain_paged(s):
    c = s["case"]
    B, T, H, Hk, d = (c[x] for x in ("B", "T", "H", "Hk", "d"))
    k, v = _gathered(s["k_cache"], s["table"]), _gathered(s["v_cache"], s["table"])
    q = s["q"].float().view(B, Hk, H // Hk * T, d)
    x = (q @ k.transpose(-1, -2)) / math.sqrt(d)
    ok = _visible(c, s, k.shape[2], 0, c["left"], c["right"])
    x = x.reshape(B, H, T, -1).masked_fill(~ok, -math.inf)
    e, total, top = _softmax(x)
    o = (e.reshape(B, Hk, H // Hk * T, -1) @ v).reshape(B, H, T, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))[..., None]
    return o.to(torch.bfloat16), total.log() + top


def _plain_prefix(s):
    c = s["case"]
    B, T, H, Hk, d, n = (c[x] for x in ("B", "T", "H", "Hk", "d", "prefix"))
    G = H // Hk
    kp, vp = (_gathered(x, s["prefix_pages"][None, :])[0, :, :n] for x in (s["k_cache"], s["v_cache"]))
    k, v = _gathered(s["k_cache"], s["table"]), _gathered(s["v_cache"], s["table"])
    q = s["q"].float().view(B, Hk, G * T, d)
    rows = q.transpose(0, 1).reshape(Hk, B * G * T, d)  # the batch's rows against the one prefix
    xp = (rows @ kp.transpose(-1, -2)).view(Hk, B, G * T, n).transpose(0, 1)
    x = torch.cat([xp, q @ k.transpose(-1, -2)], -1) / math.sqrt(d)
    ok = _visible(c, s, n + k.shape[2], n, -1, 0)
    x = x.reshape(B, H, T, -1).masked_fill(~ok, -math.inf)
    e, total, top = _softmax(x)
    e = e.reshape(B, Hk, G * T, -1)
    op = (e[..., :n].transpose(0, 1).reshape(Hk, B * G * T, n) @ vp).view(Hk, B, G * T, d).transpose(0, 1)
    o = (op + e[..., n:] @ v).reshape(B, H, T, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))[..., None]
    return o.to(torch.bfloat16), total.log() + top


def run(state):
    s, c = state, state["case"]
    if own:
        import exact_attention_19_gb300 as fa

        if c["op"] == "rope":
            turn = fa.rope_bwd if c["backward"] else fa.rope
            return turn(s["q"], s["k"], s["w"], positions=s["positions"],
                        offset=0 if s["positions"] is not None else c["offset"], interleaved=c["interleaved"],
                        mag=s["mag"])
        if c["op"] == "append":
            fa.kv_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["w"],
                         new_lens=s["new"], offset=c["offset"], interleaved=c["interleaved"], mag=s["mag"],
                         q_out=s["q_out"])
            return s["q_out"], s["k_cache"], s["v_cache"]
        if c["op"] == "paged":
            return fa.fwd_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], new_lens=s["new"],
                                window=(c["left"], c["right"]))
        return fa.fwd_prefix(s["q"], s["k_cache"], s["v_cache"], s["prefix_pages"], c["prefix"], s["table"],
                             s["lens"], new_lens=s["new"])
    return {"rope": _plain_rope, "append": _plain_append, "paged": _plain_paged, "prefix": _plain_prefix}[c["op"]](s)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    H, Hk, d = case["H"], case["Hk"], case["d"]
    if case["op"] == "rope":
        n = case["B"] * case["N"] * (H + Hk)
        index = 4 * case["B"] * case["N"] if case["packed_positions"] else 0
        return {"bytes": 4 * n * d + index + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    lens, new, P = _lengths(case), _new(case), case["page"]
    table = 4 * sum(-(-n // P) for n in lens) + 4 * case["B"]
    if case["op"] == "append":
        n = sum(new)
        return {"bytes": 4 * n * (H + 2 * Hk) * d + table + 4 * case["rot"], "flops": 3 * n * (H + Hk) * case["rot"]}
    first = case.get("prefix", 0)
    left, right = case.get("left", -1), case.get("right", 0)
    keys = pairs = 0  # keys that some row sees, and (token, key) pairs
    for n, m in zip(lens, new):
        lowest = n
        for t in range(m):
            pos = n - m + t
            lo = max(0, pos - left) if left >= 0 else 0
            hi = min(n, pos + right + 1) if right >= 0 else n
            lowest = min(lowest, lo)
            pairs += max(0, hi - lo) + first
        keys += n - lowest
    rows = case["B"] * H * case["T"]
    live = sum(new) * H
    moved = 4 * d * Hk * (keys + first) + 2 * d * (live + rows) + 4 * rows + table
    if case["op"] == "prefix":
        moved += 4 * -(-first // P)
    return {"bytes": moved, "flops": 4 * d * H * pairs}


# ----------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence
# ----------------------------------------------------------------------------
def _turn64(x, p, w, mag, interleaved, sign):
    """One sequence's x [H, N, d]: complex multiplication of its pairs by mag * e^(i sign p w)."""
    x = x.double()
    half = w.numel()
    part = x[..., :2 * half]
    z = torch.view_as_complex(part.unflatten(-1, (half, 2)).contiguous()) if interleaved else \
        torch.complex(part[..., :half].contiguous(), part[..., half:].contiguous())
    z = z * torch.polar(torch.full_like(w, mag)[None, :].expand(p.numel(), -1).contiguous(),
                        sign * torch.outer(p.double(), w))
    turned = torch.view_as_real(z).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _attend64(q, k, v, lo, hi):
    """One head's rows q [n, d] over keys lo[i] <= j < hi[i]."""
    n = q.shape[0]
    x = q @ k.T / math.sqrt(q.shape[1])
    j = torch.arange(k.shape[0], device=q.device)
    x = torch.where((j >= lo[:, None]) & (j < hi[:, None]), x, torch.full_like(x, -math.inf))
    lse = torch.logsumexp(x, -1) if k.shape[0] else torch.full((n,), -math.inf, dtype=q.dtype, device=q.device)
    weight = torch.where(lse[:, None] == -math.inf, torch.zeros_like(x), (x - lse[:, None]).exp())
    return weight @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        sign = -1.0 if case["backward"] else 1.0
        outs = []
        for x in (s["q"], s["k"]):
            y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
            for b in range(case["B"]):
                p = s["positions"][b] if s["positions"] is not None else \
                    torch.arange(case["N"], device="cuda") + case["offset"]
                y[b] = _turn64(x[b], p, s["w"], s["mag"], case["interleaved"], sign)
            outs.append(y)
        return tuple(outs)
    lens, new, P = _lengths(case), _new(case), case["page"]
    if case["op"] == "append":
        q_out, kc, vc = s["q_out"].double(), s["k_cache"].double(), s["v_cache"].double()
        for b in range(case["B"]):
            at = torch.arange(lens[b] - new[b], lens[b], device="cuda")
            page = s["table"][b][at // P].long()
            p = at + case["offset"]
            q_out[b, :, :new[b]] = _turn64(s["q"][b, :, :new[b]], p, s["w"], s["mag"], case["interleaved"], 1.0)
            turned = _turn64(s["k"][b, :, :new[b]], p, s["w"], s["mag"], case["interleaved"], 1.0)
            kc[page, :, at % P] = turned.transpose(0, 1)
            vc[page, :, at % P] = s["v"][b, :, :new[b]].double().transpose(0, 1)
        return q_out, kc, vc
    B, T, H, Hk, d = (case[x] for x in ("B", "T", "H", "Hk", "d"))
    if B * H > 2100:
        return None
    n = case.get("prefix", 0)
    left, right = case.get("left", -1), case.get("right", 0)
    o = torch.zeros(B, H, T, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        m, length = new[b], n + lens[b]
        pages = s["table"][b, :-(-lens[b] // P)].long()
        i = length - m + torch.arange(m, device="cuda")
        lo = (i - left).clamp(min=0) if left >= 0 else torch.zeros_like(i)
        hi = (i + right + 1).clamp(max=length) if right >= 0 else torch.full_like(i, length)
        for h in range(Hk):
            k = s["k_cache"][pages, h].reshape(-1, d)[:lens[b]].double()
            v = s["v_cache"][pages, h].reshape(-1, d)[:lens[b]].double()
            if n:
                shared = s["prefix_pages"].long()
                k = torch.cat([s["k_cache"][shared, h].reshape(-1, d)[:n].double(), k])
                v = torch.cat([s["v_cache"][shared, h].reshape(-1, d)[:n].double(), v])
            group = slice(h * (H // Hk), (h + 1) * (H // Hk))
            g = H // Hk
            oo, ll = _attend64(s["q"][b, group, :m].double().reshape(g * m, d), k, v, lo.repeat(g), hi.repeat(g))
            o[b, group, :m] = oo.view(g, m, d)
            lse[b, group, :m] = ll.view(g, m)
    return o, lse
