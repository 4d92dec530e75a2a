"""Measured cases of the operators around a paged cache of keys and values.

The operators (``log_domain_sinkhorn_amd``): rotary positions with a norm of each
head (``rotate_heads``, ``rotate_heads_grad``), new keys and values written into a
paged cache with both applied on the way (``cache_append``), and attention of new
tokens over such a cache (``paged_attention``).

Conventions. x [B, L, H, d]; caches [pages, page_size, Hkv, width]; key j of
sequence b lies in page page_table[b, j // page_size], slot j % page_size; query
head h reads key head h // (Hq / Hkv).
  norm:      n = x rsqrt(mean x^2 + eps) w
  rotation:  pair i of a head (elements i and i + r / 2, or 2 i and 2 i + 1) by the
             angle position f_i, times `gain`; elements from r on stay
  attention: of n new tokens of a sequence of K keys, row i is at place p = K - n + i and
             sees key j <= p; with `recent` only j > p - recent or j < first
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases
def _rotate(name, op, dtype, batch, heads_q, heads_kv, d, length, rotated=None, interleaved=False, norm=True,
            factor=1.0, start=0):
    return {"name": name, "op": op, "dtype": dtype, "batch": batch, "heads_q": heads_q, "heads_kv": heads_kv,
            "d": d, "len": length, "rotated": d if rotated is None else rotated, "interleaved": interleaved,
            "norm": norm, "factor": factor, "start": start}


def _append(name, dtype, batch, heads_q, heads_kv, d, length, cached, page, dv=None, rotated=None,
            interleaved=False, norm=False, ragged=False):
    return {"name": name, "op": "append", "dtype": dtype, "batch": batch, "heads_q": heads_q,
            "heads_kv": heads_kv, "d": d, "dv": d if dv is None else dv, "len": length, "cached": cached,
            "page": page, "rotated": d if rotated is None else rotated, "interleaved": interleaved,
            "norm": norm, "factor": 1.0, "ragged": ragged}


def _attend(name, dtype, batch, heads_q, heads_kv, d, len_q, len_k, page, dv=None, ragged=False, first=0,
            recent=0):
    return {"name": name, "op": "attend", "dtype": dtype, "batch": batch, "heads_q": heads_q,
            "heads_kv": heads_kv, "d": d, "dv": d if dv is None else dv, "len_q": len_q, "len_k": len_k,
            "page": page, "ragged": ragged, "first": first, "recent": recent}


def listed():
    return [
        # one token a sequence, far into its context: latency
        _rotate("rotate_token", "rotate", "fp16", 4, 8, 8, 64, 1, interleaved=True, norm=False, start=100000),
        # a long prompt with frequencies scaled for it, queries and keys normed
        _rotate("rotate_prompt", "rotate", "bf16", 1, 32, 8, 128, 16384, factor=8.0),
        # a training step's forward and backward
        _rotate("rotate_train", "train", "bf16", 4, 32, 8, 128, 4096),
        # the same in full precision, small and odd, half of the head rotated
        _rotate("rotate_train_odd", "train", "fp32", 2, 4, 4, 50, 333, rotated=26, interleaved=True),
        # a decoding step's keys and values into the cache, its queries on the way
        _append("append_token", "bf16", 64, 32, 8, 128, 1, 2000, 16, norm=True, ragged=True),
        # a batch of prompts into an empty cache, a quarter of the head rotated
        _append("append_prompt", "fp16", 8, 16, 16, 64, 2000, 0, 64, rotated=16, ragged=True),
        # one token against a short context, small batch: latency
        _attend("token_short", "bf16", 4, 8, 8, 64, 1, 1000, 16),
        # one token a sequence against long contexts, shared key heads
        _attend("token_long", "bf16", 16, 32, 8, 128, 1, 32768, 64, ragged=True),
        # drafted tokens, odd sizes, only the first and the recent keys visible
        _attend("tokens_few", "fp16", 3, 12, 4, 80, 5, 9001, 24, first=4, recent=2500, ragged=True),
        # a chunk of a long prompt over what came before it
        _attend("chunk_long", "bf16", 1, 32, 8, 128, 2048, 16384, 32),
        # chunks in full precision, odd sizes
        _attend("chunk_odd", "fp32", 3, 6, 2, 72, 77, 1501, 16, dv=64, ragged=True),
        # a whole prompt under a sliding window with a few first tokens
        _attend("window_prompt", "bf16", 1, 32, 8, 64, 8192, 8192, 16, first=4, recent=1024),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the listed ranges: sizes log-uniform, kept under the largest listed cost."""
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    op = rng.choice(["rotate", "train", "append", "token", "token", "chunk", "chunk"])
    heads, group = _log_int(rng, 1, 16), rng.choice([1, 1, 2, 3, 4, 8])
    while heads * group > 64:
        heads = (heads + 1) // 2
    batch = _log_int(rng, 1, 64)
    if op in ("rotate", "train"):
        d = rng.choice([32, 50, 64, 72, 80, 96, 128])
        length = _log_int(rng, 1, 16384)
        while batch * length > 16384 or batch * length * heads * (group + 1) * d > 4 * 4096 * 40 * 128:
            batch, length = (batch + 1) // 2, max(1, length // 2)
        out = _rotate("", op, dtype, batch, heads * group, heads, d, length,
                      rotated=rng.choice([d, d, d // 4 * 2]), interleaved=rng.random() < 0.5,
                      norm=rng.random() < 0.6, factor=rng.choice([1.0, 1.0, 4.0, 32.0]),
                      start=rng.choice([0, 0, _log_int(rng, 1, 500000)]))
        del out["name"]
        return out
    d = rng.choice([32, 64, 72, 80, 96, 128])
    dv = rng.choice([d, d, 64])
    page = rng.choice([8, 16, 16, 24, 32, 48, 64, 128, 256])
    ragged = rng.random() < 0.5
    if op == "append":
        length, cached = rng.choice([1, 1, _log_int(rng, 2, 2000)]), rng.choice([0, _log_int(rng, 1, 4000)])
        while batch * length > 16000 or batch * (length + cached) * heads * (d + dv) > 4.0e8:
            batch, cached = (batch + 1) // 2, cached // 2
        out = _append("", dtype, batch, heads * group, heads, d, length, cached, page, dv=dv,
                      rotated=rng.choice([d, d, d // 4 * 2]), interleaved=rng.random() < 0.5,
                      norm=rng.random() < 0.5, ragged=ragged)
        del out["name"]
        return out
    if op == "token":
        len_q, len_k = rng.choice([1, 1, 1, 2, 4, 7]), _log_int(rng, 64, 32768)
        batch = min(batch, 16)
        while batch * heads * len_k > 16 * 8 * 32768 // 3:
            batch, len_k = max(1, batch // 2), len_k // 2 + 1
    else:
        len_q, len_k = _log_int(rng, 17, 4096), _log_int(rng, 64, 16384)
        cap = 1.0e11 if dtype != "fp32" else 3.0e9  # score elements x d that a drawn case may cost
        while batch * heads * group * len_q * max(len_k, 2 * len_q) * max(d, dv) > cap \
                or batch * heads * max(len_k, 2 * len_q) * (d + dv) > 5.0e8:
            if batch > 1:
                batch = (batch + 1) // 2 if batch > 2 else 1
            elif heads * group > 8:
                heads, group = max(1, heads // 2), max(1, group // 2)
            else:
                len_q, len_k = len_q // 2 + 9, len_k // 2 + 17
    len_k = max(len_k, 2 * len_q if ragged else len_q)
    recent = rng.choice([0, 0, 0, _log_int(rng, 16, max(17, len_k // 2))])
    first = rng.choice([0, 4, 16, 100]) if recent else 0
    out = _attend("", dtype, batch, heads * group, heads, d, len_q, len_k, page, dv=dv, ragged=ragged,
                  first=first, recent=recent)
    del out["name"]
    return out


# ---------------------------------------------------------------- inputs
def _lengths(batch, n):
    """From n down to about n / 2."""
    return [max(1, n - (n * b) // (2 * batch)) for b in range(batch)]


def _frequencies(r, factor):
    """Radians a position; for a longer context slow pairs turn `factor` times more slowly
    (fewer than one turn in 8192 positions), fast ones (more than 32 turns) as before."""
    out = []
    for i in range(r // 2):
        f = 10000.0 ** (-2.0 * i / r)
        keep = 1.0 if factor == 1.0 else min(1.0, max(0.0, (8192 * f / (2 * math.pi) - 1.0) / 31.0))
        out.append(f * (keep + (1.0 - keep) / factor))
    return torch.tensor(out, dtype=torch.float64, device=DEV)


def _pages(lens, page, host):
    """Every sequence's pages, scattered over a pool: (pages, table); -1 behind the last."""
    need = [(n + page - 1) // page for n in lens]
    order = torch.randperm(sum(need) + 3, generator=host).to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return order.numel(), table.to(DEV)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))
    t = TYPES[c["dtype"]]
    B, Hq, H, d = c["batch"], c["heads_q"], c["heads_kv"], c["d"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV, dtype=t)

    def shuffled(values):
        return torch.tensor(values, dtype=torch.int32)[torch.randperm(len(values), generator=host)]

    def ints(values):
        return torch.as_tensor(values, dtype=torch.int32).to(DEV)

    st = {"op": c["op"], "dtype": t, "d": d}
    if c["op"] == "attend":
        n, m = c["len_k"], c["len_q"]
        lens = shuffled(_lengths(B, n)) if c["ragged"] else torch.full((B,), n, dtype=torch.int32)
        pages, st["table"] = _pages(lens.tolist(), c["page"], host)
        st["key_lengths"] = lens.to(DEV)
        # heads of different sharpness: the scores' deviation runs from 0.5 to 2.5
        st["q"] = normal(B, m, Hq, d) * torch.linspace(0.5, 2.5, Hq, device=DEV).to(t).view(1, 1, Hq, 1)
        st["k_cache"], st["v_cache"] = normal(pages, c["page"], H, d), normal(pages, c["page"], H, c["dv"])
        st.update(scale=1.0 / math.sqrt(d), first=c["first"], recent=c["recent"] or None)
        return st
    r = c["rotated"]
    st.update(interleaved=c["interleaved"], frequencies=_frequencies(r, c["factor"]),
              gain=1.0 if c["factor"] == 1.0 else 0.1 * math.log(c["factor"]) + 1.0, norm=EPS if c["norm"] else None)
    # the projections of the tokens, side by side in one buffer
    L = c["len"]
    dv = c.get("dv", 0)
    proj = normal(B, L, Hq * d + H * (d + dv))
    st["q"] = proj[..., :Hq * d].unflatten(2, (Hq, d))
    st["k"] = proj[..., Hq * d:(Hq + H) * d].unflatten(2, (H, d))
    for x in ("q_weight", "k_weight"):
        st[x] = 1.0 + 0.1 * torch.randn(d, generator=gen, device=DEV) if c["norm"] else None
    if c["op"] == "append":
        st["v"] = proj[..., (Hq + H) * d:].unflatten(2, (H, dv))
        before = _lengths(B, c["cached"]) if c["ragged"] and c["cached"] else [c["cached"]] * B
        new = _lengths(B, L) if c["ragged"] else [L] * B
        before, new = shuffled(before), shuffled(new)
        pages, st["table"] = _pages((before + new).tolist(), c["page"], host)
        st["cache_lengths"], st["new_lengths"] = before.to(DEV), new.to(DEV)
        st["k_cache"], st["v_cache"] = normal(pages, c["page"], H, d), normal(pages, c["page"], H, dv)
        return st
    # each sequence somewhere in its context
    st["positions"] = ints([[c["start"] + 7 * b + i for i in range(L)] for b in range(B)])
    if c["op"] == "train":
        st["dq_out"], st["dk_out"] = normal(B, L, Hq, d), normal(B, L, H, d)
    return st


# ---------------------------------------------------------------- plain forms
def _angles(st, positions):
    """cos and sin [..., 1, r / 2], angles in 64 bits, times the gain."""
    a = positions.double().unsqueeze(-1) * st["frequencies"]
    return ((x * st["gain"]).float().unsqueeze(-2) for x in (torch.cos(a), torch.sin(a)))


def _turn(st, x, cos, sin):
    """The rotation of the leading elements of x (fp32)."""
    r = 2 * st["frequencies"].numel()
    y = x.clone()
    if st["interleaved"]:
        i, j = slice(0, r, 2), slice(1, r, 2)
    else:
        i, j = slice(0, r // 2), slice(r // 2, r)
    a, b = x[..., i], x[..., j]
    y[..., i] = a * cos - b * sin
    y[..., j] = a * sin + b * cos
    return y


def _normed(st, x, weight):
    """(normed x times its weight, x hat, 1 / rms) in 32 bits."""
    x = x.float()
    if st["norm"] is None:
        return x, x, None
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + st["norm"])
    return x * rstd * weight, x * rstd, rstd


def _plain_rotate(st):
    t = st["dtype"]
    cos, sin = _angles(st, st["positions"])
    res, grads, weights = [], [], []
    for x, w, dy in (("q", "q_weight", "dq_out"), ("k", "k_weight", "dk_out")):
        n, xh, rstd = _normed(st, st[x], st[w])
        res.append(_turn(st, n, cos, sin).to(t))
        if st["op"] != "train":
            continue
        g = _turn(st, st[dy].float(), cos, -sin)
        if rstd is None:
            grads.append(g.to(t))
            continue
        weights.append((g * xh).sum((0, 1, 2)))
        u = g * st[w]
        grads.append((rstd * (u - xh * (u * xh).mean(-1, keepdim=True))).to(t))
    return tuple(res + grads + weights)


def _plain_append(st):
    t = st["dtype"]
    B, L = st["k"].shape[:2]
    before, new = st["cache_lengths"].long().view(B, 1), st["new_lengths"].long().view(B, 1)
    i = torch.arange(L, device=DEV).view(1, L)
    i = torch.where(i < new, i, torch.zeros_like(i))  # a token behind its sequence repeats the first
    place = before + i
    cos, sin = _angles(st, place)
    page = st["k_cache"].shape[1]
    slot = torch.gather(st["table"].long(), 1, place // page) * page + place % page

    def turned(x, w):
        return _turn(st, _normed(st, x, w)[0], cos, sin).to(t)

    def at(x):
        return torch.gather(x, 1, i.view(B, L, 1, 1).expand(B, L, x.shape[2], x.shape[3]))

    for x, cache in ((turned(at(st["k"]), st["k_weight"]), st["k_cache"]), (at(st["v"]), st["v_cache"])):
        cache.view(-1, *cache.shape[2:])[slot.reshape(-1)] = x.reshape(-1, *x.shape[2:])
    q = turned(st["q"], st["q_weight"])
    q = q.masked_fill((torch.arange(L, device=DEV).view(1, L) >= new).view(B, L, 1, 1), 0.0)
    return st["k_cache"], st["v_cache"], (before + new).view(B).to(torch.int32), q


def _plain_attend(st):
    q, t = st["q"].float(), st["dtype"]
    B, m, Hq, d = q.shape
    page, H = st["k_cache"].shape[1:3]
    table = st["table"].long().clamp(min=0)
    n = table.shape[1] * page
    keys = st["key_lengths"].view(B, 1, 1).long()
    p = keys - m + torch.arange(m, device=DEV).view(1, m, 1)
    j = torch.arange(n, device=DEV).view(1, 1, n)
    seen = j <= p
    if st["recent"] is not None:
        seen = seen & ((j > p - st["recent"]) | (j < st["first"]))
    gone = (j >= keys).view(B, n, 1, 1)
    k, v = (st[x][table].reshape(B, n, H, -1).float().masked_fill(gone, 0.0).permute(0, 2, 1, 3).contiguous()
            for x in ("k_cache", "v_cache"))
    q = q.reshape(B, m, H, Hq // H, d).permute(0, 2, 3, 1, 4).reshape(B, H, -1, d)
    s = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(st["scale"])
    s.view(B, H, Hq // H, m, n).masked_fill_(~seen.view(B, 1, 1, m, n), -math.inf)
    top = s.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    w = s.sub_(top).exp_()
    total = w.sum(3, keepdim=True)
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(top, -math.inf))
    w /= torch.where(total > 0, total, torch.ones_like(total))
    out = torch.matmul(w, v).reshape(B, H, Hq // H, m, -1).permute(0, 3, 1, 2, 4).reshape(B, m, Hq, -1)
    return out.to(t), lse.reshape(B, Hq, m)


# ---------------------------------------------------------------- one pass
def run(state):
    st = state
    if not own:
        return {"append": _plain_append, "attend": _plain_attend}.get(st["op"], _plain_rotate)(st)
    import log_domain_sinkhorn_amd as sk

    if st["op"] == "attend":
        return sk.paged_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["key_lengths"],
                                  scale=st["scale"], first=st["first"], recent=st["recent"])
    turn = {"frequencies": st["frequencies"], "interleaved": st["interleaved"], "gain": st["gain"],
            "norm_eps": st["norm"], "q_weight": st["q_weight"], "k_weight": st["k_weight"]}
    if st["op"] == "append":
        lengths, q = sk.cache_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"],
                                     st["cache_lengths"], new_lengths=st["new_lengths"], q=st["q"], **turn)
        return st["k_cache"], st["v_cache"], lengths, q
    res = sk.rotate_heads(st["q"], st["k"], positions=st["positions"], **turn)
    if st["op"] == "rotate":
        return res
    res += sk.rotate_heads_grad(st["dq_out"], st["dk_out"], st["q"], st["k"], positions=st["positions"], **turn)
    return res if st["norm"] is not None else res[:4]


# ---------------------------------------------------------------- work of a pass
def _visible(p, first, recent):
    """Keys that a row at place p sees."""
    if recent <= 0 or p + 1 <= recent:
        return p + 1
    return recent + min(first, p + 1 - recent)


def work(case):
    c = case
    size = 4 if c["dtype"] == "fp32" else 2
    B, Hq, H, d = c["batch"], c["heads_q"], c["heads_kv"], c["d"]
    if c["op"] == "attend":
        dv, m = c["dv"], c["len_q"]
        lens = _lengths(B, c["len_k"]) if c["ragged"] else [c["len_k"]] * B
        pairs = sum(_visible(n - m + i, c["first"], c["recent"]) for n in lens for i in range(m))
        # keys that some row sees
        keys = sum(min(n, _visible(n - 1, c["first"], c["recent"] and c["recent"] + m - 1)) for n in lens)
        return {"bytes": size * (B * m * Hq * (d + dv) + H * keys * (d + dv)) + 4 * B * m * Hq
                + 4 * (keys // c["page"] + 2 * B), "flops": 2 * Hq * pairs * (d + dv)}
    r, norm = c["rotated"], c["norm"]
    if c["op"] == "append":
        new = sum(_lengths(B, c["len"]) if c["ragged"] else [c["len"]] * B)
        return {"bytes": 2 * size * new * (Hq * d + H * (d + c["dv"])) + 16 * B + 4 * r,
                "flops": new * (Hq + H) * (3 * r + (4 * d if norm else 0))}
    rows = B * c["len"]
    n = rows * (Hq + H)
    out = {"bytes": 2 * size * n * d + 4 * rows + 4 * r, "flops": n * (3 * r + (4 * d if norm else 0))}
    if c["op"] == "train":
        out["bytes"] += size * n * d * (3 if norm else 2) + 4 * rows + 4 * r
        out["flops"] += n * (3 * r + (10 * d if norm else 0))
    return out


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_turn(x, phase, interleaved, inverse=False):
    """x [..., d] in 64 bits; phase [..., 1, r / 2] complex."""
    r = 2 * phase.shape[-1]
    head, tail = x[..., :r], x[..., r:]
    pairs = head.unflatten(-1, (r // 2, 2)) if interleaved else head.unflatten(-1, (2, r // 2)).transpose(-1, -2)
    z = torch.view_as_complex(pairs.contiguous()) * (phase.conj() if inverse else phase)
    pairs = torch.view_as_real(z)
    if not interleaved:
        pairs = pairs.transpose(-1, -2)
    return torch.cat([pairs.flatten(-2), tail], -1)


def _exact_phase(st, positions):
    a = positions.double()[..., None, None] * st["frequencies"]
    return torch.polar(torch.full_like(a, st["gain"]), a)


def _exact_norm(x, weight, eps):
    x = x.double()
    if eps is None:
        return x
    return x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + eps) * weight.double()


def _exact_rotate(st):
    phase = _exact_phase(st, st["positions"])
    args = (phase, st["interleaved"])
    y, dx, dw = [], [], []
    for x, w, dy in ((st["q"], st["q_weight"], st.get("dq_out")), (st["k"], st["k_weight"], st.get("dk_out"))):
        y.append(_exact_turn(_exact_norm(x, w, st["norm"]), *args))
        if dy is None:
            continue
        g = _exact_turn(dy.double(), *args, inverse=True)
        if st["norm"] is None:
            dx.append(g)
            continue
        x, w = x.double(), w.double()
        ms = x.square().sum(-1, keepdim=True) / x.shape[-1] + st["norm"]
        dw.append((g * x / ms.sqrt()).flatten(0, 2).sum(0))
        gw = g * w
        # d(x ms^-1/2): ms^-1/2 gw - ms^-3/2 x <gw, x> / d
        dx.append(gw / ms.sqrt() - x * (gw * x).sum(-1, keepdim=True) / (x.shape[-1] * ms * ms.sqrt()))
    return tuple(y + dx + dw)


def _exact_append(st):
    k, v = st["k_cache"].double(), st["v_cache"].double()
    B, L = st["k"].shape[:2]
    page = k.shape[1]
    before, new, table = st["cache_lengths"].tolist(), st["new_lengths"].tolist(), st["table"].tolist()
    q_out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    for b in range(B):
        phase = _exact_phase(st, torch.arange(before[b], before[b] + new[b], device=DEV))
        args = (phase, st["interleaved"])
        kb = _exact_turn(_exact_norm(st["k"][b, :new[b]], st["k_weight"], st["norm"]), *args)
        q_out[b, :new[b]] = _exact_turn(_exact_norm(st["q"][b, :new[b]], st["q_weight"], st["norm"]), *args)
        j = before[b]
        while j < before[b] + new[b]:  # a page at a time
            s = j % page
            n = min(page - s, before[b] + new[b] - j)
            at, i = table[b][j // page], j - before[b]
            k[at, s:s + n] = kb[i:i + n]
            v[at, s:s + n] = st["v"][b, i:i + n].double()
            j += n
    total = torch.tensor([x + y for x, y in zip(before, new)], dtype=torch.int32, device=DEV)
    return k, v, total, q_out


def _exact_attend(st):
    """Each query head of each sequence by itself, rows in slices."""
    B, m, Hq, _ = st["q"].shape
    page, H = st["k_cache"].shape[1:3]
    out = torch.zeros(B, m, Hq, st["v_cache"].shape[3], dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq, m), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(st["key_lengths"].tolist()):
        ids = st["table"][b, :(n + page - 1) // page].long()
        K, V = (st[x][ids].flatten(0, 1)[:n].double() for x in ("k_cache", "v_cache"))
        j = torch.arange(n, device=DEV)
        step = max(1, int(4e8 // n))
        for lo in range(0, m, step):
            p = torch.arange(lo, min(m, lo + step), device=DEV)[:, None] + (n - m)
            hidden = j > p
            if st["recent"] is not None:
                hidden |= (j <= p - st["recent"]) & (j >= st["first"])
            for h in range(Hq):
                S = st["q"][b, lo:lo + step, h].double() @ K[:, h * H // Hq].T * st["scale"]
                S[hidden] = -math.inf
                z = torch.logsumexp(S, 1)
                lse[b, h, lo:lo + step] = z
                out[b, lo:lo + step, h] = torch.exp(S - z[:, None]) @ V[:, h * H // Hq]
    return out, lse


def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend}.get(st["op"], _exact_rotate)(st)
