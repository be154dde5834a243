"""Cases of the operators that norm queries and keys on their way into attention and that keep a cache small: the
norm of each head with the rotation, forward and backward; the same in the paged cache's append; the attention weight
that cached keys gather; and the eviction of the keys that gathered least.

``run`` computes them in plain torch (``own`` false) or through the package's entry points (``own`` true).
"""
import math

import torch

own = False

_STEP = 0.6180339887498949  # fractional parts of its multiples cover (0, 1) evenly
_EPS = 1e-6


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
_ROTARY = dict(d=128, rot=128, interleaved=False, base=500000.0, offset=0, weight="bf16")


def _norm(name, **kw):
    return {**dict(op="norm", B=1, H=12, Hk=12, N=256, packed=False), **_ROTARY, **kw, "name": name}


def _norm_bwd(name, **kw):
    return {**dict(op="norm_bwd", B=1, H=12, Hk=12, N=256, packed=False), **_ROTARY, **kw, "name": name}


def _append(name, **kw):
    return {**dict(op="append", B=16, H=32, Hk=8, T=1, page=16, token_major=False, context=1024, ragged=False,
                   shifted=False), **_ROTARY, **kw, "name": name}


def _weights(name, **kw):
    return {**dict(op="weights", B=8, H=12, Hk=12, T=1, d=64, page=16, token_major=False, context=1024, ragged=False,
                   left=-1, right=0, decay=1.0), **kw, "name": name}


def _evict(name, **kw):
    return {**dict(op="evict", B=8, Hk=12, d=64, page=16, token_major=False, context=1024, budget=768, recent=64,
                   sinks=4, slack=0, fork=False), **kw, "name": name}


def listed():
    return [
        # one short prompt: a call whose cost is its launch
        _norm("norm_prompt_256", d=64, rot=64, base=10000.0),
        # a training step's queries and keys, out of the packed token-major projection, grouped heads
        _norm("norm_train_4x8192", B=4, H=32, Hk=8, N=8192),
        # the gradients of a small model's layer, with those of the norms' weights
        _norm_bwd("norm_bwd_8x1024_d64", B=8, N=1024, d=64, rot=64, base=10000.0),
        # the same with documents packed in a row, interleaved pairs, half of the head turned, weights in 32 bits, odd length
        _norm_bwd("norm_bwd_packed_3x4099", B=3, H=16, Hk=16, N=4099, rot=64, interleaved=True, packed=True,
                  weight="fp32"),
        # one decoded token for each of 16 sequences
        _append("append_decode_16"),
        # a chunk of the prompts of 4 sequences, of different lengths, behind caches that lost other numbers of tokens
        _append("append_chunk_4x2048", B=4, T=2048, page=64, context=4000, ragged=True, shifted=True),
        # one decoded token's weights over 8 short caches: a call of a few microseconds
        _weights("weights_decode_8x1024_d64"),
        # decoding 32 sequences of 1 to 8192 tokens, grouped heads, older weight fading
        _weights("weights_decode_32x8192", B=32, H=32, Hk=8, d=128, context=8192, decay=0.98),
        # a prompt's next 2048 tokens over what is in the cache already, lengths of their own
        _weights("weights_chunk_2x2048_over_8192", B=2, H=32, Hk=8, T=2048, d=128, page=64, context=8192, ragged=True),
        # trimming short caches, where latency counts; some are within their budget
        _evict("evict_8x1024_d64"),
        # halving the long caches of a batch in place
        _evict("evict_16x8192_half", B=16, Hk=8, d=128, context=8192, budget=4096, recent=512),
        # long documents cut to a quarter into pages of their own, the originals kept; token-major pages, odd length
        _evict("evict_fork_4x31999", B=4, Hk=4, d=128, page=128, token_major=True, context=31999, budget=8000,
               recent=1000, sinks=16, fork=True),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _cost(c):
    """What a case moves and computes at most, against the largest listed ones."""
    if c["op"] in ("norm", "norm_bwd"):
        each = c["B"] * c["N"] * (c["H"] + c["Hk"]) * c["d"]
        return each / (4 * 8192 * 40 * 128 if c["op"] == "norm" else 3 * 4099 * 32 * 128)
    cache = c["B"] * c["context"] * c["Hk"] * c["d"]
    if c["op"] == "append":
        return max(c["B"] * c["T"] * (c["H"] + 2 * c["Hk"]) * c["d"] / (4 * 2048 * 48 * 128), cache / (16 << 20))
    if c["op"] == "weights":
        return max(cache / (32 * 8192 * 8 * 128), c["B"] * c["H"] * c["T"] * c["context"] / (2 * 32 * 2048 * 8192))
    return cache / (16 * 8192 * 8 * 128)


def draw(rng):
    while True:
        op = rng.choice(["norm", "norm_bwd", "append", "weights", "weights", "evict", "evict"])
        d = rng.choice([64, 128])
        Hk = rng.choice([1, 2, 3, 4, 8, 12, 16])
        H = Hk * rng.choice([1, 1, 2, 4, 5, 8])
        if H > 64:
            continue
        rotary = dict(d=d, H=H, Hk=Hk, rot=rng.choice([d, d, d // 2, d // 4, 0]), interleaved=rng.random() < 0.5,
                      base=rng.choice([10000.0, 500000.0, 1000000.0]),
                      offset=rng.choice([0, 0, rng.randrange(1, 1000000)]), weight=rng.choice(["bf16", "fp32", "none"]))
        pages = dict(page=rng.choice([16, 32, 64, 128, 256]), token_major=rng.random() < 0.4)
        if op in ("norm", "norm_bwd"):
            c = (_norm if op == "norm" else _norm_bwd)("", B=rng.randint(1, 8), N=_spread(rng, 1, 8192),
                                                       packed=rng.random() < 0.3, **rotary)
        elif op == "append":
            T = rng.choice([1, 1, _spread(rng, 2, 2048)])
            c = _append("", B=_spread(rng, 1, 128), T=T, context=max(T, _spread(rng, 1, 8192)),
                        ragged=rng.random() < 0.4, shifted=rng.random() < 0.5, **rotary, **pages)
        elif op == "weights":
            T = rng.choice([1, 1, rng.randint(2, 8), _spread(rng, 2, 2048)])
            c = _weights("", B=_spread(rng, 1, 128), H=H, Hk=Hk, T=T, d=d, context=max(T, _spread(rng, 1, 32000)),
                         ragged=rng.random() < 0.4, decay=rng.choice([1.0, 1.0, 0.95, 0.5, 0.0]), **pages)
            if rng.random() < 0.3:
                c["left"] = _spread(rng, 1, 8192)
            if rng.random() < 0.15:
                c["right"] = -1  # every cached key, as for an encoder's states
        else:
            context = _spread(rng, 24, 32000)
            budget = rng.randint(max(1, context // 10), context)
            sinks = rng.choice([0, 0, min(budget, 4), rng.randint(0, budget // 4)])
            c = _evict("", B=_spread(rng, 1, 128), Hk=Hk, d=d, context=context, budget=budget, sinks=sinks,
                       recent=rng.choice([0, rng.randint(0, budget - sinks), (budget - sinks) // 8]),
                       slack=rng.choice([0, 0, rng.randint(1, 64)]), fork=rng.random() < 0.4, **pages)
        del c["name"]
        if _cost(c) <= 1.0:
            return c


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _lengths(c):
    """Tokens of each sequence's cache, the new ones among them: the first has `context`, the others fewer."""
    lo, hi = c.get("T", 1), c["context"]
    return [hi] + [lo + int((hi - lo) * (1.0 + b * _STEP) % (hi - lo + 1)) if hi > lo else hi for b in range(1, c["B"])]


def _fresh(c):
    """New tokens of each sequence: T, or where they differ something from 1 to T."""
    T = c["T"]
    return [T] * c["B"] if not c["ragged"] else [T] + [1 + int(T * ((b * _STEP * _STEP) % 1.0)) for b in range(1, c["B"])]


def _normal(gen, *shape):
    return torch.randn(*shape, device="cuda", dtype=torch.bfloat16, generator=gen)


def _heads(x, sizes, d):
    """[B, heads, N, d] views of the packed projection x [B, N, sum(sizes) * d]."""
    return [part.unflatten(-1, (n, d)).transpose(1, 2)
            for part, n in zip(x.split([n * d for n in sizes], -1), sizes)]


def _norm_inputs(c, gen, s):
    """Frequencies (64 bits) and the norms' weights, near one."""
    rot = c["rot"]
    s["w"] = (c["base"] ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).cuda() if rot else None
    kind = {"bf16": torch.bfloat16, "fp32": torch.float32, "none": None}[c["weight"]]
    for name in ("wq", "wk"):
        near = 1.0 + 0.25 * torch.randn(c["d"], device="cuda", generator=gen)
        s[name] = near.to(kind) if kind is not None else None


def _pool(c, gen, lens, more=()):
    """K, V and weights of a pool in which the sequences' pages lie in any order, the block table, and where `more`
    names lengths, a second table of other pages for them."""
    P, Hk, d = c["page"], c["Hk"], c["d"]
    need = [[-(-n // P) for n in ns] for ns in (lens, more)]
    pages = sum(need[0]) + sum(need[1]) + 2
    shape = (pages, P, Hk, d) if c["token_major"] else (pages, Hk, P, d)
    k, v = _normal(gen, *shape), _normal(gen, *shape)
    if c["token_major"]:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    tables, at = [], 0
    for counts in need:
        t = torch.full((len(counts), max(counts, default=1)), -1, dtype=torch.int64)
        for b, n in enumerate(counts):
            t[b, :n] = torch.arange(at, at + n)
            at += n
        t = t.cuda()
        tables.append(torch.where(t >= 0, order[t.clamp(min=0)], t.to(torch.int32)).contiguous())
    # what keys gather is spread widely, and some have gathered nothing
    w = torch.randn(pages, Hk, P, device="cuda", generator=gen).mul_(1.5).exp_()
    w = torch.where(torch.rand(pages, Hk, P, device="cuda", generator=gen) < 0.1, torch.zeros_like(w), w)
    return k, v, w, tables[0], tables[1]


def _int32(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7919 + 2 * seed)
    s = {"case": c}
    d = c["d"]
    if c["op"] in ("norm", "norm_bwd"):
        B, N, H, Hk = c["B"], c["N"], c["H"], c["Hk"]
        _norm_inputs(c, gen, s)
        s["q"], s["k"], _ = _heads(_normal(gen, B, N, (H + 2 * Hk) * d), (H, Hk, Hk), d)
        if c["op"] == "norm_bwd":  # gradients as the attention's backward leaves them
            s["dq"], s["dk"] = _normal(gen, B, H, N, d), _normal(gen, B, Hk, N, d)
        s["positions"] = None
        if c["packed"]:  # documents of 1200 tokens after one another, cut elsewhere for each seed
            cut = torch.randint(0, 1200, (B, 1), device="cuda", generator=gen)
            s["positions"] = ((torch.arange(N, device="cuda") + cut) % 1200 + c["offset"]).to(torch.int32).contiguous()
        return s
    lens = _lengths(c)
    s["lens"] = _int32(lens)
    if c["op"] == "evict":
        most = c["budget"] + c["slack"]
        out = [c["budget"] if n > most else n for n in lens] if c["fork"] else ()
        s["k_cache"], s["v_cache"], s["weights"], s["table"], t = _pool(c, gen, lens, out)
        s["table_out"] = None
        if c["fork"]:
            room = -(-most // c["page"])
            s["table_out"] = torch.nn.functional.pad(t[:, :room], (0, max(0, room - t.shape[1])), value=-1).contiguous()
        s["shift"] = torch.randint(0, 100000, (c["B"],), device="cuda", generator=gen).to(torch.int32)
        return s
    fresh = _fresh(c)
    s["new"] = _int32(fresh) if c["ragged"] else None
    s["k_cache"], s["v_cache"], s["weights"], s["table"], _ = _pool(c, gen, lens)
    B, T, H, Hk = c["B"], c["T"], c["H"], c["Hk"]
    if c["op"] == "append":
        _norm_inputs(c, gen, s)
        s["q"], s["k"], s["v"] = _heads(_normal(gen, B, T, (H + 2 * Hk) * d), (H, Hk, Hk), d)
        s["q_out"] = torch.zeros(B, H, T, d, device="cuda", dtype=torch.bfloat16)
        s["shift"] = torch.randint(0, 100000, (B,), device="cuda", generator=gen).to(torch.int32) if c["shifted"] else None
        return s
    s["q"] = _normal(gen, B, H, T, d)
    s["lse"] = torch.full((B, H, T), -math.inf, device="cuda")  # what the attention over this cache returns beside O
    for b in range(B):
        n, m = lens[b], min(fresh[b], lens[b])
        k = s["k_cache"][s["table"][b, :-(-n // c["page"])].long()].transpose(0, 1).reshape(Hk, -1, d)[:, :n].float()
        x = (s["q"][b, :, :fresh[b]].reshape(Hk, -1, d).float() @ k.transpose(1, 2)).view(H, fresh[b], n) / math.sqrt(d)
        pos = n - fresh[b] + torch.arange(fresh[b], device="cuda")[:, None]
        j = torch.arange(n, device="cuda")
        hidden = torch.zeros(fresh[b], n, dtype=torch.bool, device="cuda")
        if c["left"] >= 0:
            hidden = hidden | (j < pos - c["left"])
        if c["right"] >= 0:
            hidden = hidden | (j > pos + c["right"])
        s["lse"][b, :, :fresh[b]] = x.masked_fill_(hidden, -math.inf).logsumexp(-1)
    return s


# ----------------------------------------------------------------------------
# one pass, plain
# ----------------------------------------------------------------------------
def _angles(positions, w):
    """cos and sin [B or 1, 1, N, rot / 2] in 32 bits, of angles in 64."""
    a = positions.double()[:, None, :, None] * w
    return a.cos().float(), a.sin().float()


def _halves(rot, interleaved):
    return (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))


def _turned(x, cos_sin, interleaved, back=False):
    """x [B, H, N, d], 32 bits, with its pairs turned (`back`: the other way)."""
    if cos_sin is None:
        return x
    cos, sin = cos_sin
    first, second = _halves(2 * cos.shape[-1], interleaved)
    y = x.clone()
    sin = -sin if back else sin
    y[..., first] = x[..., first] * cos - x[..., second] * sin
    y[..., second] = x[..., second] * cos + x[..., first] * sin
    return y


def _normed(x):
    """x / rms(x) over each head, and 1 / rms, in 32 bits."""
    x = x.float()
    r = (x.square().mean(-1, keepdim=True) + _EPS).rsqrt()
    return x * r, r


def _norm_turned(x, weight, cos_sin, interleaved):
    n, _ = _normed(x)
    return _turned(n if weight is None else n * weight.float(), cos_sin, interleaved).to(torch.bfloat16)


def _plain_norm(s):
    c = s["case"]
    p = s["positions"] if c["packed"] else (torch.arange(c["N"], device="cuda") + c["offset"])[None]
    cs = _angles(p, s["w"]) if c["rot"] else None
    return (_norm_turned(s["q"], s["wq"], cs, c["interleaved"]), _norm_turned(s["k"], s["wk"], cs, c["interleaved"]))


def _norm_gradient(g, x, weight, cs, interleaved):
    g = _turned(g.float(), cs, interleaved, back=True)
    n, r = _normed(x)
    u = g if weight is None else g * weight.float()
    dx = r * (u - n * (u * n).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), None if weight is None else (g * n).sum((0, 1, 2))


def _plain_norm_bwd(s):
    c = s["case"]
    p = s["positions"] if c["packed"] else (torch.arange(c["N"], device="cuda") + c["offset"])[None]
    cs = _angles(p, s["w"]) if c["rot"] else None
    dq, dwq = _norm_gradient(s["dq"], s["q"], s["wq"], cs, c["interleaved"])
    dk, dwk = _norm_gradient(s["dk"], s["k"], s["wk"], cs, c["interleaved"])
    return dq, dk, dwq, dwk


def _plain_append(s):
    c = s["case"]
    fresh = s["new"] if s["new"] is not None else torch.full_like(s["lens"], c["T"])
    t = torch.arange(c["T"], device="cuda")
    at = (s["lens"] - fresh)[:, None] + t
    live = t < fresh[:, None]
    p = at + c["offset"] + (s["shift"][:, None] if s["shift"] is not None else 0)
    cs = _angles(p, s["w"]) if c["rot"] else None
    q = _norm_turned(s["q"], s["wq"], cs, c["interleaved"])
    k = _norm_turned(s["k"], s["wk"], cs, c["interleaved"])
    s["q_out"].copy_(torch.where(live[:, None, :, None], q, s["q_out"]))
    b, i = live.nonzero(as_tuple=True)
    j = at[b, i]
    page, slot = s["table"][b, j // c["page"]].long(), j % c["page"]
    s["k_cache"][page, :, slot] = k[b, :, i]
    s["v_cache"][page, :, slot] = s["v"][b, :, i]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _gathered(pages, table):
    """[B, Hk, L, ...]: the pages of each row of the table, one after another."""
    return pages[table.clamp(min=0).long()].transpose(1, 2).flatten(2, 3)


def _plain_weights(s):
    c = s["case"]
    B, T, H, Hk, d, P = (c[x] for x in ("B", "T", "H", "Hk", "d", "page"))
    k = _gathered(s["k_cache"], s["table"]).float()
    x = (s["q"].float().view(B, Hk, -1, d) @ k.transpose(2, 3)).view(B, H, T, -1) / math.sqrt(d)
    fresh = s["new"] if s["new"] is not None else torch.full_like(s["lens"], T)
    first = (s["lens"] - fresh)[:, None, None]
    t, j = torch.arange(T, device="cuda")[:, None], torch.arange(k.shape[2], device="cuda")
    seen = (j < s["lens"][:, None, None]) & (t < fresh[:, None, None])
    if c["left"] >= 0:
        seen = seen & (j >= first + t - c["left"])
    if c["right"] >= 0:
        seen = seen & (j <= first + t + c["right"])
    seen = seen[:, None] & (s["lse"] > -math.inf)[..., None]
    p = torch.where(seen, (x - s["lse"][..., None]).exp(), torch.zeros_like(x))
    gathered = p.view(B, Hk, -1, k.shape[2]).sum(2)
    old = c["decay"] * _gathered(s["weights"], s["table"])
    gathered = gathered + torch.where(j < first, old, torch.zeros_like(old))
    b, i = ((j < s["lens"][:, None]) & (fresh > 0)[:, None]).nonzero(as_tuple=True)
    s["weights"][s["table"][b, i // P].long(), :, i % P] = gathered[b, :, i]
    return s["weights"]


def _plain_evict(s):
    c = s["case"]
    P, most = c["page"], c["budget"] + c["slack"]
    lens = s["lens"][:, None, None]
    w = _gathered(s["weights"], s["table"])
    j = torch.arange(w.shape[2], device="cuda")
    over = lens > most
    out = torch.where(over, torch.full_like(lens, c["budget"]), lens)
    held = (j < c["sinks"]) | (j >= lens - c["recent"])
    rank = torch.where(held, torch.full_like(w, math.inf), w)
    rank = torch.where(j < lens, rank, torch.full_like(w, -math.inf))
    order = rank.sort(dim=-1, descending=True, stable=True).indices  # equal weights: the lower slot first
    place = torch.empty_like(order).scatter_(-1, order, j.expand_as(order))
    keep = (place < out) & (j < lens)
    kept = torch.where(keep, j, torch.full_like(order, w.shape[2])).sort(-1).values
    kept = torch.nn.functional.pad(kept[..., :most], (0, max(0, most - w.shape[2])), value=w.shape[2])
    i = torch.arange(most, device="cuda")
    kept = torch.where(i < out, kept, torch.full_like(kept, -1))
    b, h, n = (kept >= 0).nonzero(as_tuple=True)
    src = kept[b, h, n]
    to = s["table"] if s["table_out"] is None else s["table_out"]
    from_page, from_slot = s["table"][b, src // P].long(), src % P
    to_page, to_slot = to[b, n // P].long(), n % P
    for name in ("k_cache", "v_cache", "weights"):
        s[name][to_page, h, to_slot] = s[name][from_page, h, from_slot]
    out = out.flatten()
    s["shift"] += s["lens"] - out
    return s["k_cache"], s["v_cache"], s["weights"], out, s["shift"], kept.to(torch.int32)


_PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "append": _plain_append, "weights": _plain_weights,
          "evict": _plain_evict}


def run(state):
    s, c = state, state["case"]
    if own:
        import exact_attention_19_gb300 as fa

        if c["op"] in ("norm", "norm_bwd"):
            turn = dict(q_weight=s["wq"], k_weight=s["wk"], eps=_EPS, positions=s["positions"],
                        offset=0 if c["packed"] else c["offset"], interleaved=c["interleaved"])
            if c["op"] == "norm":
                return fa.norm_rope(s["q"], s["k"], s["w"], **turn)
            return fa.norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["w"], **turn)
        if c["op"] == "append":
            fa.kv_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["w"],
                         new_lens=s["new"], offset=c["offset"], interleaved=c["interleaved"], q_out=s["q_out"],
                         eps=_EPS, q_weight=s["wq"], k_weight=s["wk"], shift=s["shift"])
            return s["q_out"], s["k_cache"], s["v_cache"]
        if c["op"] == "weights":
            return fa.kv_weights(s["q"], s["lse"], s["k_cache"], s["weights"], s["table"], s["lens"],
                                 new_lens=s["new"], window=(c["left"], c["right"]), decay=c["decay"])
        lens, kept = fa.kv_evict(s["k_cache"], s["v_cache"], s["weights"], s["table"], s["lens"], c["budget"],
                                 recent=c["recent"], sinks=c["sinks"], slack=c["slack"], table_out=s["table_out"],
                                 shift=s["shift"])
        return s["k_cache"], s["v_cache"], s["weights"], lens, s["shift"], kept
    return _PLAIN[c["op"]](s)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    c = case
    d, Hk = c["d"], c["Hk"]
    if c["op"] in ("norm", "norm_bwd"):
        n = c["B"] * c["N"] * (c["H"] + Hk) * d
        small = 4 * c["B"] * c["N"] * c["packed"] + 4 * c["rot"]
        back = c["op"] == "norm_bwd"
        return {"bytes": (6 if back else 4) * n + small, "flops": (12 if back else 7) * n}
    lens, P = _lengths(c), c["page"]
    table = 4 * sum(-(-n // P) for n in lens) + 4 * c["B"]
    if c["op"] == "append":
        n = sum(_fresh(c))
        return {"bytes": 4 * n * (c["H"] + 2 * Hk) * d + table + 4 * c["rot"], "flops": 7 * n * (c["H"] + Hk) * d}
    if c["op"] == "weights":
        fresh, left, right = _fresh(c), c["left"], c["right"]
        keys = touched = pairs = 0
        for n, m in zip(lens, fresh):
            lowest = n
            for t in range(m):
                pos = n - m + t
                lo = max(0, pos - left) if left >= 0 else 0
                hi = min(n, pos + right + 1) if right >= 0 else n
                lowest = min(lowest, lo)
                pairs += max(0, hi - lo)
            keys += n - lowest
            touched += n - lowest if c["decay"] == 1.0 else n
        rows = sum(fresh) * c["H"]
        return {"bytes": 2 * d * Hk * keys + 8 * Hk * touched + (2 * d + 4) * rows + table,
                "flops": 2 * d * c["H"] * pairs}
    most, read, moved, listed_ = c["budget"] + c["slack"], 0, 0.0, 0
    for n in lens:
        gone = n - c["budget"] if n > most else 0
        read += n if gone or c["fork"] else 0
        listed_ += n - gone
        if c["fork"]:
            moved += n - gone
        elif gone:  # the keys before the first one that goes stay where they are: where that lies on average
            free = n - c["sinks"] - c["recent"]
            moved += c["budget"] - c["sinks"] - (free - gone) / (gone + 1)
    return {"bytes": Hk * (4 * read + 4 * listed_ + moved * (8 * d + 4)) + table, "flops": Hk * read}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------
def _spun(z, p, w, interleaved, sign):
    """One sequence's z [heads, N, d], 64 bits: its pairs as complex numbers, times e^(i sign p w)."""
    if w is None:
        return z
    half = w.numel()
    x = z[..., :2 * half]
    x = x.unflatten(-1, (half, 2)) if interleaved else x.unflatten(-1, (2, half)).transpose(-1, -2)
    x = torch.view_as_complex(x.contiguous()) * torch.exp(1j * sign * torch.outer(p.double(), w))
    x = torch.view_as_real(x)
    x = x.flatten(-2) if interleaved else x.transpose(-1, -2).flatten(-2)
    return torch.cat([x, z[..., 2 * half:]], -1)


def _scaled(x, weight):
    x = x.double()
    size = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
    x = x / torch.sqrt(size * size / x.shape[-1] + _EPS)
    return x if weight is None else x * weight.double()


def _exact_norm(s, c):
    outs = []
    for x, weight in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            p = s["positions"][b] if c["packed"] else torch.arange(c["N"], device="cuda") + c["offset"]
            y[b] = _spun(_scaled(x[b], weight), p, s["w"], c["interleaved"], 1.0)
        outs.append(y)
    return tuple(outs)


def _exact_norm_bwd(s, c):
    """The gradients from the derivative of the norm written out: d(x / rms) = (I - x x^T / (d rms^2)) / rms."""
    dxs, dws = [], []
    for g, x, weight in ((s["dq"], s["q"], s["wq"]), (s["dk"], s["k"], s["wk"])):
        dx = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(c["d"], dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            p = s["positions"][b] if c["packed"] else torch.arange(c["N"], device="cuda") + c["offset"]
            back = _spun(g[b].double(), p, s["w"], c["interleaved"], -1.0)
            xb = x[b].double()
            var = (xb * xb).sum(-1, keepdim=True) / c["d"] + _EPS
            dw += (back * xb / var.sqrt()).flatten(0, 1).sum(0)
            if weight is not None:
                back = back * weight.double()
            dx[b] = back / var.sqrt() - xb * (back * xb).sum(-1, keepdim=True) / (c["d"] * var * var.sqrt())
        dxs.append(dx)
        dws.append(None if weight is None else dw)
    return (*dxs, *dws)


def _exact_append(s, c):
    q_out, kc, vc = s["q_out"].double(), s["k_cache"].double(), s["v_cache"].double()
    for b, (n, m) in enumerate(zip(_lengths(c), _fresh(c))):
        at = torch.arange(n - m, n, device="cuda")
        p = at + c["offset"] + (int(s["shift"][b]) if c["shifted"] else 0)
        page = s["table"][b][at // c["page"]].long()
        q_out[b, :, :m] = _spun(_scaled(s["q"][b, :, :m], s["wq"]), p, s["w"], c["interleaved"], 1.0)
        k = _spun(_scaled(s["k"][b, :, :m], s["wk"]), p, s["w"], c["interleaved"], 1.0)
        kc[page, :, at % c["page"]] = k.transpose(0, 1)
        vc[page, :, at % c["page"]] = s["v"][b, :, :m].double().transpose(0, 1)
    return q_out, kc, vc


def _exact_weights(s, c):
    G, P = c["H"] // c["Hk"], c["page"]
    out = s["weights"].double()
    for b, (n, m) in enumerate(zip(_lengths(c), _fresh(c))):
        j = torch.arange(n, device="cuda")
        pages = s["table"][b][j // P].long()
        pos = (n - m + torch.arange(m, device="cuda")).repeat(G)[:, None]
        lo = pos - c["left"] if c["left"] >= 0 else torch.zeros_like(pos)
        hi = pos + c["right"] if c["right"] >= 0 else torch.full_like(pos, n)
        for h in range(c["Hk"]):
            k = s["k_cache"][pages, h, j % P].double()
            group = slice(h * G, (h + 1) * G)
            x = s["q"][b, group, :m].double().reshape(G * m, -1) @ k.T / math.sqrt(c["d"])
            x = x - s["lse"][b, group, :m].double().reshape(-1, 1)
            x = torch.where((j >= lo) & (j <= hi), x, torch.full_like(x, -math.inf))
            old = out[pages, h, j % P]
            out[pages, h, j % P] = torch.where(j < n - m, c["decay"] * old, torch.zeros_like(old)) + x.exp().sum(0)
    return out


def _exact_evict(s, c):
    P, most, B, Hk = c["page"], c["budget"] + c["slack"], c["B"], c["Hk"]
    if B * Hk > 1100:
        return None
    kc, vc, w = s["k_cache"].double(), s["v_cache"].double(), s["weights"].double()
    old = [x.clone() for x in (kc, vc, w)] if c["fork"] else (kc, vc, w)
    lens, shift = _lengths(c), s["shift"].clone()
    kept = torch.full((B, Hk, most), -1, dtype=torch.int32, device="cuda")
    after = []
    to = s["table_out"] if c["fork"] else s["table"]
    for b, n in enumerate(lens):
        m = c["budget"] if n > most else n
        after.append(m)
        shift[b] += n - m
        j = torch.arange(n, device="cuda")
        pages, slots = s["table"][b][j // P].long(), j % P
        i = j[:m]
        for h in range(Hk):
            keep = torch.ones(n, dtype=torch.bool, device="cuda")
            if m < n:  # the lightest of the free ones go, of equal ones the highest slots
                free = j[c["sinks"]:n - c["recent"]].flip(0)
                by_weight = old[2][pages[free], h, slots[free]].sort(stable=True).indices
                keep[free[by_weight[:n - m]]] = False
            src = j[keep]
            kept[b, h, :m] = src.to(torch.int32)
            for a, o in zip((kc, vc, w), old):
                a[to[b][i // P].long(), h, i % P] = o[pages[src], h, slots[src]]
    return kc, vc, w, torch.tensor(after, dtype=torch.int32), shift, kept


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "append": _exact_append, "weights": _exact_weights,
            "evict": _exact_evict}[case["op"]](s, case)
