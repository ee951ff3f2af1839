"""The operators that fill, weigh and trim the two per-token caches: what is measured.

  rope     rotary positions on a part of every head, forward and backward
  append   new tokens into the latent and indexer-key caches (rotated, quantized)
  mass     the attention weight every cached token received, accumulated
  select   which cached tokens stay, by that weight
  compact  the tokens that stay moved together, in place or into other pages

``run`` computes the plain form with elementary torch operations, or, where ``own`` is
true, makes the calls a user of the package makes.
"""

import math

import torch

own = False

LATENT, NOPE, ROT, HEADS, D_IDX = 576, 512, 64, 128, 128
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- cases --------------------------------------------------------------------------


def listed():
    return [
        # the rope part of the queries of one sequence's two newest tokens: latency
        dict(name="rope q, 2 rows", op="rope", rows=2, heads=128, dim=64, rot_begin=0, rot=64,
             interleaved=True, dtype="bf16", scaling="yarn", far=131072, x_pad=128, out_pad=512,
             backward=False),
        # the indexer queries of an 8K prompt: half of each head rotated, the rest copied
        dict(name="rope q_idx, 8k prompt", op="rope", rows=8192, heads=64, dim=128, rot_begin=0,
             rot=64, interleaved=False, dtype="bf16", scaling="none", far=8192, x_pad=0,
             out_pad=0, backward=False),
        # the gradient of the MHA-mode queries of an odd number of tokens, in fp32
        dict(name="rope backward, fp32", op="rope", rows=1021, heads=128, dim=192, rot_begin=128,
             rot=64, interleaved=True, dtype="fp32", scaling="linear", far=65536, x_pad=0,
             out_pad=0, backward=True),
        # two new tokens of each of 128 sequences into a paged cache (one decode step)
        dict(name="append, paged decode", op="append", batch=128, q_per_seq=2, ctx_min=64,
             ctx_max=2048, paged=True, page=64, ragged=False, interleaved=True,
             idx_interleaved=False, scaling="yarn"),
        # prompts of 0 to 16384 tokens prefilled together
        dict(name="append, ragged prompts", op="append", batch=8, q_per_seq=16384, ctx_min=16384,
             ctx_max=16384, paged=False, page=64, ragged=True, interleaved=True,
             idx_interleaved=False, scaling="none"),
        # one token of one sequence of the 32K context: few rows, one long axis
        dict(name="mass, 1 row", op="mass", batch=1, q_per_seq=1, k=2048, ctx_min=32768,
             ctx_max=32768, paged=False, page=64),
        # two query rows of each of 128 sequences (one decode step)
        dict(name="mass, paged decode", op="mass", batch=128, q_per_seq=2, k=2048, ctx_min=4096,
             ctx_max=32768, paged=True, page=64),
        # the last 512 rows of a prompt, an observation window
        dict(name="mass, 512-row window", op="mass", batch=1, q_per_seq=512, k=2048,
             ctx_min=32768, ctx_max=32768, paged=False, page=64),
        # one short conversation trimmed to half
        dict(name="select, 1 short", op="select", batch=1, ctx_min=1000, ctx_max=1000, keep=500,
             sink=4, recent=64),
        # a batch of long sequences trimmed to 16K each, some of them shorter than that
        dict(name="select, 128 long", op="select", batch=128, ctx_min=4096, ctx_max=131072,
             keep=16384, sink=4, recent=1024),
        # one contiguous cache trimmed in place
        dict(name="compact, 1 in place", op="compact", batch=1, ctx_min=32768, ctx_max=32768,
             keep=16384, paged=False, page=64, in_place=True),
        # paged caches of a batch moved into fresh pages
        dict(name="compact, paged batch", op="compact", batch=48, ctx_min=4096, ctx_max=16384,
             keep=8192, paged=True, page=64, in_place=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "mass", "select", "compact"])
    paged, page = rng.random() < 0.5, rng.choice([64, 64, 128])
    if op == "rope":
        rot = rng.choice([32, 64, 64, 128])
        before, after = rng.choice([(0, 0), (0, 64), (128, 0), (16, 8)])
        heads = rng.choice([1, 4, 16, 64, 128])
        dim = before + rot + after
        return dict(op=op, rows=_log(rng, 1, min(8192, (60 << 20) // (heads * dim))), heads=heads,
                    dim=dim, rot_begin=before, rot=rot, interleaved=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    far=_log(rng, 100, 1 << 20), x_pad=rng.choice([0, 8, 128]),
                    out_pad=rng.choice([0, 8, 512]), backward=rng.random() < 0.4)
    if op == "append":
        batch = _log(rng, 1, 128)
        q = _log(rng, 1, 65536 // batch)
        ctx = q + _log(rng, 1, 2048)
        return dict(op=op, batch=batch, q_per_seq=q, ctx_min=rng.randint(q, ctx), ctx_max=ctx,
                    paged=paged, page=page, ragged=batch > 1 and rng.random() < 0.5,
                    interleaved=rng.random() < 0.7, idx_interleaved=rng.random() < 0.3,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]))
    if op == "mass":
        batch = _log(rng, 1, 64)
        q = _log(rng, 1, 256 // batch)
        ctx = _log(rng, max(300, q), 32768)
        return dict(op=op, batch=batch, q_per_seq=q, k=_log(rng, 16, 2048),
                    ctx_min=rng.randint(max(ctx // 4, q), ctx), ctx_max=ctx, paged=paged,
                    page=page)
    if op == "select":
        batch = _log(rng, 1, 64)
        ctx = _log(rng, 200, 131072)
        keep = max(100, int(ctx * rng.uniform(0.1, 0.9)))
        return dict(op=op, batch=batch, ctx_min=rng.randint(ctx // 4, ctx), ctx_max=ctx,
                    keep=keep, sink=rng.choice([0, 4, 16]),
                    recent=rng.randint(0, keep // 2))
    batch = _log(rng, 1, 32)
    ctx = _log(rng, 200, min(32768, (1 << 19) // batch))
    return dict(op=op, batch=batch, ctx_min=rng.randint(ctx // 2, ctx), ctx_max=ctx,
                keep=max(64, int(ctx * rng.uniform(0.1, 0.8))), paged=paged, page=page,
                in_place=rng.random() < 0.6)


# ---- inputs -------------------------------------------------------------------------


def _lengths(lo, hi, n):
    """n lengths spread evenly over [lo, hi] (the same for every seed, in another order)."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _query_lengths(c):
    q, n = c["q_per_seq"], c["batch"]
    return _lengths(0, q, n) if c["ragged"] else [q] * n


def frequencies(scaling, rot=ROT, base=10000.0, factor=32.0, original=4096):
    """Radians per position of each pair, and the factor on the result."""
    theta = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [t / factor for t in theta], 1.0
    if scaling == "ntk":
        b = base * factor ** (rot / (rot - 2.0))
        return [b ** (-2.0 * i / rot) for i in range(rot // 2)], 1.0
    if scaling == "yarn":
        f = []
        for t in theta:
            gamma = min(1.0, max(0.0, (original * t / (2 * math.pi) - 1.0) / 31.0))
            f.append(t / factor * (1.0 - gamma) + t * gamma)
        return f, 0.1 * math.log(factor) + 1.0
    return theta, 1.0


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return torch.empty(*shape, device="cuda", dtype=dtype).normal_(0.0, std, generator=g)


def _caches(c, g):
    """Latent rows, key codes (no NaN among them), key scales, and the block table."""
    if c["paged"]:
        per = -(-c["ctx_max"] // c["page"])
        n = c["batch"] * per
        table = torch.randperm(n, generator=g, device="cuda").int().view(c["batch"], per)
        shape = (n, c["page"])
    else:
        table, shape = None, (c["batch"], c["ctx_max"])
    kv = _normal(g, *shape, LATENT, std=0.5)
    codes = torch.randint(0, 127, (*shape, D_IDX), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.rand(*shape, generator=g, device="cuda") * 0.01 + 0.001
    return kv, codes, scale, table


def _seqlens(c, g):
    lens = torch.tensor(_lengths(c["ctx_min"], c["ctx_max"], c["batch"]), device="cuda",
                        dtype=torch.int32)
    return lens[torch.randperm(c["batch"], generator=g, device="cuda")]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "rope":
        t, h, d = c["rows"], c["heads"], c["dim"]
        dtype = TYPES[c["dtype"]]
        s["x"] = _normal(g, t, h, c["x_pad"] + d, dtype=dtype)[..., c["x_pad"]:]
        s["out"] = torch.zeros(t, h, c["out_pad"] + d, device="cuda",
                               dtype=dtype)[..., c["out_pad"]:]
        s["positions"] = torch.randint(0, c["far"], (t,), generator=g, device="cuda",
                                       dtype=torch.int32)
        f, s["magnitude"] = frequencies(c["scaling"], c["rot"])
        s["freqs"] = torch.tensor(f, device="cuda", dtype=torch.float64)
        return s
    s["seqlens"] = _seqlens(c, g)
    if c["op"] == "append":
        s["kv"], s["codes"], s["scale"], s["table"] = _caches(c, g)
        q = torch.tensor(_query_lengths(c), device="cuda")
        q = q[torch.randperm(c["batch"], generator=g, device="cuda")]
        s["q_start"] = torch.cat([q.new_zeros(1), q.cumsum(0)]).int()
        t = sum(_query_lengths(c))
        # the new latents are the last columns of a wider projection's rows
        s["latent"] = _normal(g, t, 64 + LATENT)[:, 64:]
        s["keys"] = _normal(g, t, D_IDX)
        # positions run ahead of the slots: tokens were evicted from the cache before
        s["positions"] = torch.randint(0, 1 << 17, (t,), generator=g, device="cuda",
                                       dtype=torch.int32)
        f, s["magnitude"] = frequencies(c["scaling"])
        s["freqs"] = torch.tensor(f, device="cuda", dtype=torch.float64)
        return s
    if c["op"] == "mass":
        s["kv"], _, _, s["table"] = _caches(c, g)
        b, q, k = c["batch"], c["q_per_seq"], c["k"]
        t = b * q
        s["q"] = _normal(g, t, HEADS, LATENT, std=3.0)
        seq = torch.arange(t, device="cuda") // q
        pos = s["seqlens"][seq] - q + torch.arange(t, device="cuda") % q
        # a random set of min(k, pos + 1) visible positions each, ascending, padded with -1
        r = torch.rand(t, max(c["ctx_max"], k), generator=g, device="cuda")
        r.masked_fill_(torch.arange(r.shape[1], device="cuda") > pos[:, None], -1.0)
        v, i = r.topk(k, dim=1)
        i = torch.where(v >= 0, i, 1 << 30).sort(dim=1).values
        s["idx"] = torch.where(i < (1 << 30), i, -1).int()
        s["sm_scale"] = LATENT ** -0.5
        z = _logits(s)
        s["lse"] = torch.logsumexp(z, dim=2).contiguous()
        # what a few earlier steps left
        s["mass"] = torch.rand(b, c["ctx_max"], generator=g, device="cuda") * 2e-3
        return s
    if c["op"] == "select":
        # a heavy tail, and tokens that no query ever chose
        m = torch.empty(c["batch"], c["ctx_max"], device="cuda").log_normal_(-3.0, 2.0, generator=g)
        s["mass"] = m * (torch.rand(m.shape, generator=g, device="cuda") > 0.2)
        return s
    s["kv"], s["codes"], s["scale"], s["table"] = _caches(c, g)
    b, keep = c["batch"], c["keep"]
    s["mass"] = torch.rand(b, c["ctx_max"], generator=g, device="cuda")
    r = torch.rand(b, c["ctx_max"], generator=g, device="cuda")
    at = torch.arange(c["ctx_max"], device="cuda")
    r = torch.where(at < 4, 2.0, r).masked_fill_(at >= s["seqlens"][:, None], -1.0)
    v, i = r.topk(min(keep, c["ctx_max"]), dim=1)
    i = torch.where(v >= 0, i, 1 << 30).sort(dim=1).values
    s["kept"] = torch.where(i < (1 << 30), i, -1).int()
    s["new_lens"] = s["seqlens"].clamp(max=keep)
    if not c["in_place"]:
        to = dict(c, ctx_max=keep)
        s["to_kv"], s["to_codes"], s["to_scale"], s["to_table"] = _caches(to, g)
        s["to_mass"] = torch.rand(b, keep, generator=g, device="cuda")
    return s


# ---- the plain forms ----------------------------------------------------------------


def _rotated(x, positions, freqs, magnitude, interleaved, backward=False):
    """Pairs of x's last axis turned by position times frequency, in 32 bits."""
    angle = positions.double()[:, None] * freqs
    cos, sin = (angle.cos() * magnitude).float(), (angle.sin() * magnitude).float()
    if backward:
        sin = -sin
    if x.dim() == 3:
        cos, sin = cos[:, None], sin[:, None]
    x = x.float()
    half = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    ra, rb = a * cos - b * sin, a * sin + b * cos
    return torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)


def _cache_rows(table, page, ctx, seq, slot):
    """Row of the cache arrays that holds slot `slot` of sequence `seq`."""
    if table is None:
        return seq * ctx + slot
    return table[seq, slot // page].long() * page + slot % page


def _logits(s):
    """scale q . c of every listed entry, and -inf where the list has none: [rows, heads, k]."""
    c = s["case"]
    t = s["q"].shape[0]
    seq = (torch.arange(t, device="cuda") // c["q_per_seq"])[:, None]
    slot = s["idx"].long()
    row = _cache_rows(s["table"], c["page"], c["ctx_max"], seq, slot.clamp(min=0))
    z = torch.bmm(s["q"].float(), s["kv"].view(-1, LATENT)[row].float().transpose(1, 2))
    return (z * s["sm_scale"]).masked_fill_((slot < 0)[:, None], -math.inf)


def _plain_rope(s):
    c, x = s["case"], s["x"]
    a, b = c["rot_begin"], c["rot_begin"] + c["rot"]
    y = _rotated(x[..., a:b], s["positions"], s["freqs"], s["magnitude"], c["interleaved"],
                 c["backward"])
    s["out"].copy_(torch.cat([x[..., :a], y.to(x.dtype), x[..., b:]], -1))
    return s["out"]


def _plain_append(s):
    c = s["case"]
    t = torch.arange(s["latent"].shape[0], device="cuda")
    start = s["q_start"].long()
    seq = torch.searchsorted(start, t, right=True) - 1
    slot = s["seqlens"][seq] - (start[seq + 1] - t)
    row = _cache_rows(s["table"], c["page"], c["ctx_max"], seq, slot)
    rope = _rotated(s["latent"][:, NOPE:], s["positions"], s["freqs"], s["magnitude"],
                    c["interleaved"])
    s["kv"].view(-1, LATENT)[row] = torch.cat([s["latent"][:, :NOPE], rope.bfloat16()], 1)
    key = torch.cat([_rotated(s["keys"][:, :ROT], s["positions"], s["freqs"], s["magnitude"],
                              c["idx_interleaved"]), s["keys"][:, ROT:].float()], 1)
    scale = key.abs().amax(1).clamp(min=2.0 ** -120) / 448.0
    codes = (key / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    s["codes"].view(-1, D_IDX)[row] = codes
    s["scale"].view(-1)[row] = scale
    return s["kv"], s["codes"].view(torch.float8_e4m3fn), s["scale"]


def _plain_mass(s):
    c = s["case"]
    p = (_logits(s) - s["lse"][:, :, None]).exp().mean(1)
    seq = (torch.arange(p.shape[0], device="cuda") // c["q_per_seq"])[:, None]
    at = seq * c["ctx_max"] + s["idx"].long().clamp(min=0)
    s["mass"].view(-1).index_add_(0, at.flatten(), p.flatten())
    return s["mass"]


def _plain_select(s):
    c, m = s["case"], s["mass"]
    n, at = s["seqlens"][:, None], torch.arange(c["ctx_max"], device="cuda")
    safe = (at < c["sink"]) | (at >= n - c["recent"])
    m = torch.where(safe, math.inf, m).masked_fill_(at >= n, -math.inf)
    first = m.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
    first = torch.where(first < n, first, 1 << 30).sort(dim=1).values
    kept = torch.full((c["batch"], c["keep"]), -1, device="cuda", dtype=torch.int32)
    kept[:, :first.shape[1]] = torch.where(first < (1 << 30), first, -1).int()
    return kept, s["seqlens"].clamp(max=c["keep"])


def _plain_compact(s):
    c = s["case"]
    kept = s["kept"].long()
    b, i = (kept >= 0).nonzero(as_tuple=True)
    src = _cache_rows(s["table"], c["page"], c["ctx_max"], b, kept[b, i])
    to = "" if c["in_place"] else "to_"
    ctx = c["ctx_max"] if c["in_place"] else c["keep"]
    dst = _cache_rows(s[to + "table"], c["page"], ctx, b, i)
    s[to + "kv"].view(-1, LATENT)[dst] = s["kv"].view(-1, LATENT)[src]
    s[to + "codes"].view(-1, D_IDX)[dst] = s["codes"].view(-1, D_IDX)[src]
    s[to + "scale"].view(-1)[dst] = s["scale"].view(-1)[src]
    at = torch.arange(ctx, device="cuda")
    moved = torch.zeros(c["batch"], ctx, device="cuda")
    moved[b, i] = s["mass"][b, kept[b, i]]
    s[to + "mass"].copy_(torch.where(at < s["seqlens"][:, None], moved, s[to + "mass"]))
    return (s[to + "kv"], s[to + "codes"].view(torch.float8_e4m3fn), s[to + "scale"],
            s[to + "mass"])


PLAIN = {"rope": _plain_rope, "append": _plain_append, "mass": _plain_mass,
         "select": _plain_select, "compact": _plain_compact}


# ---- the framework's calls ----------------------------------------------------------


def _layout(dsa, c, ctx, seqlens, table, cache):
    if table is None:
        return dsa.KvLayout(c["batch"], ctx, seqlens)
    return dsa.KvLayout(c["batch"], ctx, seqlens, table, c["page"], cache.shape[0])


def _own(s):
    from sparse_attention_05_b200 import dsa
    c = s["case"]
    op = c["op"]
    if op == "rope":
        f = dsa.dsa_rope_bwd if c["backward"] else dsa.dsa_rope
        return f(s["x"], s["positions"], s["freqs"], s["out"], rot_begin=c["rot_begin"],
                 interleaved=c["interleaved"], magnitude=s["magnitude"])
    if op == "select":
        return dsa.dsa_evict_select(s["mass"], dsa.KvLayout(c["batch"], c["ctx_max"],
                                                            s["seqlens"]),
                                    c["keep"], c["sink"], c["recent"])
    kv = _layout(dsa, c, c["ctx_max"], s["seqlens"], s["table"], s["kv"])
    if op == "append":
        dsa.dsa_cache_append(s["latent"], s["keys"], s["kv"], s["codes"], s["scale"], kv,
                             c["q_per_seq"], s["freqs"], s["positions"],
                             interleaved=c["interleaved"], idx_interleaved=c["idx_interleaved"],
                             magnitude=s["magnitude"],
                             q_start=s["q_start"] if c["ragged"] else None)
        return s["kv"], s["codes"].view(torch.float8_e4m3fn), s["scale"]
    if op == "mass":
        return dsa.dsa_attn_mass(s["q"], s["kv"], kv, c["q_per_seq"], s["idx"], s["sm_scale"],
                                 s["lse"], s["mass"])
    if c["in_place"]:
        dsa.dsa_cache_compact(s["kv"], s["codes"], s["scale"], kv, s["kept"], s["new_lens"],
                              mass=s["mass"])
        return s["kv"], s["codes"].view(torch.float8_e4m3fn), s["scale"], s["mass"]
    to = _layout(dsa, c, c["keep"], None, s["to_table"], s["to_kv"])
    dsa.dsa_cache_compact(s["kv"], s["codes"], s["scale"], kv, s["kept"], s["new_lens"],
                          mass=s["mass"], dst=to, dst_kv_cache=s["to_kv"],
                          dst_k_idx=s["to_codes"], dst_k_scale=s["to_scale"],
                          dst_mass=s["to_mass"])
    return (s["to_kv"], s["to_codes"].view(torch.float8_e4m3fn), s["to_scale"], s["to_mass"])


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ---- work ---------------------------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["rows"] * c["heads"]
        size = TYPES[c["dtype"]].itemsize
        return {"bytes": 2 * n * c["dim"] * size + 4 * c["rows"] + 4 * c["rot"],
                "flops": 3 * n * c["rot"]}
    if c["op"] == "append":
        t = sum(_query_lengths(c))
        return {"bytes": t * (2 * 2 * LATENT + 2 * D_IDX + 4 + D_IDX + 4) + 8 * c["batch"],
                "flops": t * (3 * 2 * ROT + 3 * D_IDX)}
    lens = _lengths(c["ctx_min"], c["ctx_max"], c["batch"])
    if c["op"] == "mass":
        q, k = c["q_per_seq"], c["k"]
        entries = sum(min(k, n - q + i + 1) for n in lens for i in range(q))
        # distinct cached rows that q independent lists of k among n name
        rows = sum(n * (1.0 - (1.0 - min(1.0, k / n)) ** q) for n in lens)
        return {"bytes": int(c["batch"] * q * (HEADS * LATENT * 2 + HEADS * 4 + 4 * k) +
                             rows * (2 * LATENT + 8)),
                "flops": entries * HEADS * LATENT * 2}
    if c["op"] == "select":
        return {"bytes": 4 * (sum(lens) + c["batch"] * (c["keep"] + 2)), "flops": sum(lens)}
    moved = sum(min(n, c["keep"]) for n in lens)
    return {"bytes": moved * (2 * (2 * LATENT + D_IDX + 4 + 4) + 4), "flops": 0}


# ---- 64 bits ------------------------------------------------------------------------


def _exact_compact(c, s):
    to = "" if c["in_place"] else "to_"
    names = ("kv", "codes", "scale")
    src = [s[n].view(torch.float8_e4m3fn).double() if n == "codes" else s[n].double()
           for n in names]
    dst = [s[to + n].view(torch.float8_e4m3fn).double() if n == "codes" else s[to + n].double()
           for n in names]
    mass = s[to + "mass"].double()

    def places(table, b, slots):
        if table is None:
            return torch.full_like(slots, b), slots
        return table[b].long()[slots // c["page"]], slots % c["page"]

    for b, n in enumerate(s["new_lens"].tolist()):
        slots = s["kept"][b, :n].long()
        new = torch.arange(n, device="cuda")
        for x, y in zip(src, dst):
            y[places(s[to + "table"], b, new)] = x[places(s["table"], b, slots)]
        mass[b, :int(s["seqlens"][b])] = 0.0
        mass[b, :n] = s["mass"][b, slots].double()
    return [*dst, mass]


def exact(case, seed):
    """The definition in 64 bits, with complex turns for the rotation."""
    c, s = case, prepare(case, seed)
    if c["op"] == "select":
        return None
    if c["op"] == "compact":
        return _exact_compact(c, s)

    def turned(x, interleaved, sign=1.0):
        turn = torch.polar(torch.full_like(s["freqs"], s["magnitude"]).expand(
            x.shape[0], -1), sign * torch.outer(s["positions"].double(), s["freqs"]))
        pair = x.double().unflatten(-1, (-1, 2) if interleaved else (2, -1))
        if not interleaved:
            pair = pair.transpose(-1, -2)
        z = torch.view_as_complex(pair.contiguous())
        z = torch.view_as_real(z * (turn[:, None] if x.dim() == 3 else turn))
        return (z if interleaved else z.transpose(-1, -2)).flatten(-2)

    if c["op"] == "rope":
        y = s["x"].double()
        part = slice(c["rot_begin"], c["rot_begin"] + c["rot"])
        y[..., part] = turned(s["x"][..., part], c["interleaved"], -1.0 if c["backward"] else 1.0)
        return y
    if c["op"] == "append":
        lat, key = s["latent"].double(), s["keys"].double()
        lat[:, NOPE:] = turned(s["latent"][:, NOPE:], c["interleaved"])
        key[:, :ROT] = turned(s["keys"][:, :ROT], c["idx_interleaved"])
        kv, scale = s["kv"].double(), s["scale"].double()
        first = s["q_start"].tolist()
        for b, n in enumerate(s["seqlens"].tolist()):
            new = slice(first[b], first[b + 1])
            at = torch.arange(n - (first[b + 1] - first[b]), n, device="cuda")
            if c["paged"]:
                where = (s["table"][b].long()[at // c["page"]], at % c["page"])
            else:
                where = (torch.full_like(at, b), at)
            kv[where] = lat[new]
            scale[where] = key[new].abs().amax(1) / 448.0
        return [kv, None, scale]
    mass = s["mass"].double()
    for b in range(c["batch"]):
        n = int(s["seqlens"][b])
        at = torch.arange(n, device="cuda")
        if c["paged"]:
            lat = s["kv"][s["table"][b].long()[at // c["page"]], at % c["page"]].double()
        else:
            lat = s["kv"][b, :n].double()
        for r in range(b * c["q_per_seq"], (b + 1) * c["q_per_seq"]):
            named = s["idx"][r][s["idx"][r] >= 0].long()
            z = s["q"][r].double() @ lat[named].T * s["sm_scale"]
            mass[b, named] += torch.exp(z - s["lse"][r].double()[:, None]).sum(0) / HEADS
    return mass
