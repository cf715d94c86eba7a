"""What the operators around an attention layer with a bounded cache are measured on:
norms and rotation of queries and keys (with the gradients), the attention weight
that cached rows gather, the choice of the rows that stay, and their moving together.

`own` False: the plain forms below (elementary torch operations, 32 bits).
`own` True: the same work through the package's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 32          # elements that share one scale in MXFP8
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # --- norms and rotation: one token of each of 16 running sequences (latency)
        dict(name="norm_step", op="norm", tokens=16, heads=64, kv=8, d=128, rot=128, norm="rms", pairs="half", src="bf16",
             far=8192, back=False),
        # a packed batch of prompts, queries and keys being slices of one projection
        dict(name="norm_prompt", op="norm", tokens=32768, heads=64, kv=8, d=128, rot=128, norm="rms", pairs="half",
             src="bf16", far=32768, back=False),
        # 32-bit carriers, few narrow heads, half of each rotated in neighbouring pairs, positions far out
        dict(name="norm_ragged", op="norm", tokens=9001, heads=20, kv=5, d=64, rot=32, norm="layer", pairs="neighbours",
             src="f32", far=1 << 20, back=False),
        # gradients of a training batch
        dict(name="back_batch", op="norm", tokens=16384, heads=32, kv=8, d=128, rot=64, norm="rms", pairs="half",
             src="bf16", far=8192, back=True),
        # gradients of a short document, one key head, layer norms with their shifts
        dict(name="back_short", op="norm", tokens=777, heads=16, kv=1, d=64, rot=64, norm="layer", pairs="half",
             src="f32", far=2048, back=True),
        # --- weight gathered by cached rows: a serving step, 64 sequences, one token each, 8-bit cache
        dict(name="weigh_step", op="weigh", seqs=64, t_lo=1, t_hi=1, s_lo=2048, s_hi=16384, heads=64, kv=8, d=128,
             prec="mxfp8", page=64, mix=8),
        # a mixed batch: chunks of odd lengths behind caches of odd lengths
        dict(name="weigh_ragged", op="weigh", seqs=6, t_lo=1, t_hi=1500, s_lo=1501, s_hi=8191, heads=32, kv=4, d=128,
             prec="fp8", page=16, mix=9),
        # a chunk of a long prompt
        dict(name="weigh_chunk", op="weigh", seqs=1, t_lo=4096, t_hi=4096, s_lo=32768, s_hi=32768, heads=64, kv=8, d=128,
             prec="bf16", page=64, mix=10),
        # --- choice of rows: caches a little over their budget, each head on its own
        dict(name="choose_step", op="choose", seqs=16, s_lo=2049, s_hi=2304, kv=8, page=64, budget=2048, sinks=4, recent=256,
             shared=False, mix=11),
        # a long prompt that has just been read, the same rows for all heads
        dict(name="choose_prompt", op="choose", seqs=3, s_lo=20000, s_hi=65536, kv=8, page=64, budget=4096, sinks=4,
             recent=1024, shared=True, mix=12),
        # --- moving the rows that stay: the caches of the step above
        dict(name="compact_step", op="compact", seqs=16, s_lo=2049, s_hi=2304, kv=8, d=128, prec="mxfp8", page=64,
             budget=2048, shared=False, mix=13),
        # long prompts, odd pages, one scale a row
        dict(name="compact_prompt", op="compact", seqs=5, s_lo=20000, s_hi=65536, kv=8, d=128, prec="bf16", page=16,
             budget=16384, shared=True, mix=14),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm of the range."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


HEADS = [(1, 4), (1, 16), (1, 64), (2, 5), (4, 8), (8, 1), (8, 8)]     # key heads, query heads to each


def draw(rng):
    op = rng.choice(["norm", "norm", "weigh", "weigh", "choose", "compact"])
    if op == "norm":
        kv, group = rng.choice(HEADS)
        d = rng.choice([64, 128])
        back = rng.random() < 0.5
        most = (1 << 30) // (10 * (kv * group + kv) * d)
        return dict(op=op, tokens=_spread(rng, 1, min(32768, most)), heads=kv * group, kv=kv, d=d,
                    rot=rng.choice([d, 32, 64]), norm=rng.choice(["rms", "layer"]), pairs=rng.choice(["half", "neighbours"]),
                    src=rng.choice(["bf16", "f32"]), far=_spread(rng, 1, 1 << 20), back=back)
    c = dict(op=op, seqs=_spread(rng, 1, 64), page=rng.choice([16, 32, 64, 128]), mix=rng.randrange(1, 1 << 30))
    top = max(64, 131072 // c["seqs"])
    if op == "weigh":
        c["prec"], c["d"] = rng.choice(["bf16", "mxfp8", "fp8"]), rng.choice([64, 128])
        c["kv"], group = rng.choice(HEADS)
        c["heads"] = c["kv"] * group
        c["s_lo"] = _spread(rng, 1, min(top, 32768))
        c["s_hi"] = _spread(rng, c["s_lo"], min(top, 32768))
        most = max(1, min(c["s_lo"], 2048 // c["seqs"]))
        c["t_lo"] = 1 if rng.random() < 0.5 else _spread(rng, 1, most)
        c["t_hi"] = _spread(rng, c["t_lo"], most) if c["t_lo"] > 1 else rng.choice([1, most])
        return c
    c["kv"] = rng.choice([1, 2, 3, 4, 8])
    c["s_lo"] = _spread(rng, 64 if op == "choose" else 1, min(top, 65536))
    c["s_hi"] = _spread(rng, c["s_lo"], min(top, 65536))
    c["budget"] = _spread(rng, 1, min(16384, 2 * c["s_hi"]))
    c["shared"] = rng.random() < 0.4
    if op == "choose":
        longest = max(s for _, s in _lengths(c))
        c["budget"] = min(c["budget"], max(1, longest // 2))          # one sequence at least has to choose
        c["sinks"] = rng.randint(0, min(8, c["budget"]))
        c["recent"] = rng.randint(0, (c["budget"] - c["sinks"]) // 2)
    else:
        c["prec"], c["d"] = rng.choice(["bf16", "mxfp8", "fp8"]), rng.choice([64, 128])
    return c


def _lengths(case):
    """(new tokens, cached tokens) of each sequence: part of the case, not of the seed."""
    rng = random.Random(case["mix"])
    out = []
    for _ in range(case["seqs"]):
        s = rng.randint(case["s_lo"], case["s_hi"])
        t = min(s, rng.randint(case["t_lo"], case["t_hi"])) if "t_lo" in case else s
        out.append((t, s))
    return out


def _row_bytes(case):
    return {"bf16": 2 * case["d"], "mxfp8": case["d"] + case["d"] // BLOCK, "fp8": case["d"] + 1}[case["prec"]]


def work(case):
    if case["op"] == "norm":
        rows = case["tokens"] * (case["heads"] + case["kv"])
        wide = case["d"] * (2 if case["src"] == "bf16" else 4)
        out = case["d"] * (2 if case["src"] == "bf16" or not case["back"] else 4)
        if case["back"]:      # inputs and gradients of the outputs read, gradients of the inputs written
            return {"bytes": rows * (wide + case["d"] * 2 + out) + 4 * case["tokens"], "flops": 14 * rows * case["d"]}
        return {"bytes": rows * (wide + out) + 4 * case["tokens"], "flops": 7 * rows * case["d"]}
    lens, kv = _lengths(case), case["kv"]
    if case["op"] == "weigh":
        rows = sum(s for _, s in lens) * kv
        tokens = sum(t for t, _ in lens)
        pairs = sum(t * (s - t) + t * (t + 1) // 2 for t, s in lens) * case["heads"]
        return {"bytes": rows * (_row_bytes(case) + 8) + tokens * case["heads"] * (2 * case["d"] + 4),
                "flops": 2 * case["d"] * pairs}
    heads = 1 if case["shared"] else kv
    kept = sum(min(s, case["budget"]) for _, s in lens)
    if case["op"] == "choose":
        rows = sum(s for _, s in lens) * kv
        return {"bytes": 4 * rows + 4 * case["seqs"] * heads * case["budget"], "flops": rows}
    return {"bytes": 2 * kept * kv * (2 * _row_bytes(case) + 4) + 4 * kept * heads, "flops": 0}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def _normal(gen, *shape, outliers=True):
    """Activations: normal, one in a hundred an outlier."""
    x = torch.randn(shape, generator=gen, device="cuda")
    if outliers:
        x *= torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.01, 8.0, 1.0)
    return x


def _prefix(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def _scale_width(case):
    return case["d"] // BLOCK if case["prec"] == "mxfp8" else 1


def _pages(case, gen, lens, names):
    """Pages that hold valid rows everywhere (slots not in use hold older rows)
    and a table that spreads the sequences' pages over them."""
    p = case["page"]
    need = [-(-s // p) for _, s in lens]
    pages = sum(need) + 3
    cache = {}
    for n in names:
        x = _normal(gen, pages, case["kv"], p, case["d"])
        if case["prec"] == "bf16":
            cache[n], cache[n + "_scale"] = x.to(torch.bfloat16), None
            continue
        b = x.reshape(pages, case["kv"], p, _scale_width(case), -1)
        e = torch.frexp(b.abs().amax(-1))[1] - 8                      # a scale that saturates nothing
        cache[n] = (b * _power(-e)[..., None]).reshape(x.shape).to(torch.float8_e4m3fn).view(torch.uint8)
        cache[n + "_scale"] = (e + 127).to(torch.uint8)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return cache, table, pages


def prepare(case, seed):
    gen = _gen(seed)
    st = dict(case=case)
    if case["op"] == "norm":
        t, h, kv, d = case["tokens"], case["heads"], case["kv"], case["d"]
        dt = torch.bfloat16 if case["src"] == "bf16" else torch.float32
        x = _normal(gen, t, h + kv, d).to(dt)                         # one projection gives both
        st["q"], st["k"] = x[:, :h], x[:, h:]
        st["pos"] = torch.randint(0, case["far"], (t,), generator=gen, device="cuda", dtype=torch.int32)
        for n in ("q", "k"):
            st[n + "_weight"] = 1 + 0.1 * _normal(gen, d, outliers=False)
            st[n + "_bias"] = 0.1 * _normal(gen, d, outliers=False) if case["norm"] == "layer" else None
        if case["back"]:
            st["dq"] = _normal(gen, t, h, d, outliers=False).to(torch.bfloat16)
            st["dk"] = _normal(gen, t, kv, d, outliers=False).to(torch.bfloat16)
        return st
    lens = _lengths(case)
    st["lens"] = lens
    names = {"weigh": ["k", "v"], "choose": [], "compact": ["k", "v"]}[case["op"]]
    st["cache"], st["table"], pages = _pages(case, gen, lens, names)
    st["cu_k"] = _prefix([s for _, s in lens])
    st["max_k"] = max(s for _, s in lens)
    # gathered so far: spread over orders of magnitude, one in twenty never looked at, some equal
    w = torch.exp(2 * torch.randn((pages, case["kv"], case["page"]), generator=gen, device="cuda") - 6)
    w = w.to(torch.bfloat16).float()
    st["weights"] = torch.where(torch.rand(w.shape, generator=gen, device="cuda") < 0.05, 0.0, w)
    if case["op"] == "weigh":
        st["cu_q"] = _prefix([t for t, _ in lens])
        st["max_q"] = max(t for t, _ in lens)
        tokens = sum(t for t, _ in lens)
        st["q"] = (2 * _normal(gen, tokens, case["heads"], case["d"], outliers=False)).to(torch.bfloat16)
        st["sm_scale"] = 1.0 / math.sqrt(case["d"])
        st["lse"] = _lse(st)
    elif case["op"] == "compact":
        n, heads = case["budget"], 1 if case["shared"] else case["kv"]
        length = torch.tensor([s for _, s in lens], device="cuda")[:, None, None]
        r = torch.rand((len(lens), heads, max(st["max_k"], n)), generator=gen, device="cuda")
        at = torch.arange(r.shape[-1], device="cuda")
        r += (at < 4) + 1.0 * (at >= length - n // 8)                 # the first and the last rows stay
        idx = torch.topk(torch.where(at < length, r, -1.0), n).indices
        idx = torch.sort(torch.where(idx < length, idx, 1 << 30)).values
        st["kept"] = torch.where(idx < length, idx, -1).to(torch.int32)
        st["kept_len"] = length.flatten().clamp_max(n).to(torch.int32)
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    c = state["case"]
    return {"norm": _run_back if c.get("back") else _run_norm, "weigh": _run_weigh, "choose": _run_choose,
            "compact": _run_compact}[c["op"]](state)


def _once(s, name, make):
    """What a user's program makes once and keeps: a handle, a workspace."""
    if name not in s:
        s[name] = make()
    return s[name]


def _handle(s):
    import sparse_attention_indexer_dsa_gb300 as dsa
    c = s["cache"]
    return _once(s, "handle", lambda: dsa.PagedCache(k=c["k"], k_scale=c["k_scale"], v=c["v"], v_scale=c["v_scale"],
                                                     prec=s["case"]["prec"]))


def _factors(s):
    """cos and sin of every token's angles, formed in 64 bits."""
    c = s["case"]
    f = 10000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
    a = s["pos"].double()[:, None] * f
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _rotate(x, cos, sin, pairs):
    """The first dimensions of x turned, a pair by an angle; the others as they are."""
    n = 2 * cos.shape[-1]
    r, rest = x[..., :n], x[..., n:]
    if pairs == "half":
        a, b = r[..., :n // 2], r[..., n // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = r[..., ::2], r[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _normed(x, norm):
    """x in 32 bits, normed and not yet weighted, and the factor that did it."""
    x = x.float()
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    inv = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * inv, inv


def _run_norm(s):
    c = s["case"]
    if own:
        import sparse_attention_indexer_dsa_gb300 as dsa
        return dsa.norm_rope(s["q"], s["k"], s["pos"], s["q_weight"], s["k_weight"], q_bias=s["q_bias"],
                             k_bias=s["k_bias"], norm=c["norm"], eps=EPS, rope_dim=c["rot"],
                             rope_interleaved=c["pairs"] == "neighbours", out_dtype=torch.bfloat16)
    cos, sin = _factors(s)
    out = []
    for n in ("q", "k"):
        y = _normed(s[n], c["norm"])[0] * s[n + "_weight"]
        if s[n + "_bias"] is not None:
            y = y + s[n + "_bias"]
        out.append(_rotate(y, cos, sin, c["pairs"]).to(torch.bfloat16))
    return tuple(out)


def _run_back(s):
    c = s["case"]
    if own:
        import sparse_attention_indexer_dsa_gb300 as dsa
        ws = _once(s, "ws", lambda: dsa.norm_rope_workspace(c["d"]))
        g = dsa.norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["pos"], s["q_weight"], s["k_weight"],
                                   norm=c["norm"], eps=EPS, rope_dim=c["rot"],
                                   rope_interleaved=c["pairs"] == "neighbours", ws=ws)
        return tuple(x for x in g if x is not None)
    cos, sin = _factors(s)
    out = []
    for n in ("q", "k"):
        g = _rotate(s["d" + n].float(), cos, -sin, c["pairs"])
        x, inv = _normed(s[n], c["norm"])
        gw = g * s[n + "_weight"]
        dx = gw - x * (gw * x).mean(-1, keepdim=True)
        if c["norm"] == "layer":
            dx = dx - gw.mean(-1, keepdim=True)
        out.append(((dx * inv).to(s[n].dtype), (g * x).sum((0, 1)), g.sum((0, 1))))
    (a, aw, ab), (b, bw, bb) = out
    return (a, b, aw, bw, ab, bb) if c["norm"] == "layer" else (a, b, aw, bw)


def _places(s, pos):
    """Page and slot of positions [sequences, ...]; page 0 behind a sequence's last."""
    p = s["case"]["page"]
    at = (pos // p).clamp(0, s["table"].shape[1] - 1)
    flat = torch.gather(s["table"].long(), 1, at.reshape(at.shape[0], -1)).reshape(at.shape)
    return flat.clamp_min(0), pos % p


def _power(e):
    """2 to whole exponents of [-126, 127], from the bits: no rounding."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _keys(s, h, page, slot):
    """Rows of key head h as 32-bit values."""
    c = s["case"]
    x = s["cache"]["k"][page, h, slot]
    if c["prec"] == "bf16":
        return x.float()
    e = s["cache"]["k_scale"][page, h, slot].int() - 127
    x = x.view(torch.float8_e4m3fn).float()
    return (x.reshape(*e.shape, -1) * _power(e)[..., None]).reshape(x.shape)


def _logits(s, h):
    """Scaled products of one key head's queries and keys, [sequences, tokens, heads to the key head, positions],
    -inf where a query does not see a key; sequences are padded to the longest."""
    c = s["case"]
    t = torch.tensor([t for t, _ in s["lens"]], device="cuda")[:, None]
    n = torch.tensor([n for _, n in s["lens"]], device="cuda")[:, None]
    i, pos = torch.arange(int(s["max_q"]), device="cuda")[None], torch.arange(s["max_k"], device="cuda")[None]
    row = (s["cu_q"][:-1, None] + i).long().clamp_max(s["q"].shape[0] - 1)
    g = c["heads"] // c["kv"]
    q = s["q"][row, h * g:(h + 1) * g].float().flatten(1, 2)
    k = _keys(s, h, *_places(s, pos.expand(len(s["lens"]), -1)))
    x = torch.bmm(q, k.transpose(1, 2)).unflatten(1, (i.shape[1], g)).mul_(s["sm_scale"])
    see = (pos[:, None] <= (n - t + i)[..., None]) & (i < t)[..., None]
    return x.masked_fill_(~see[:, :, None], -math.inf), row, i < t


def _lse(s):
    """log of the sum of exp(logit) of every query, as the attention gives it."""
    c = s["case"]
    out = torch.empty((s["q"].shape[0], c["heads"]), device="cuda")
    g = c["heads"] // c["kv"]
    for h in range(c["kv"]):
        x, row, there = _logits(s, h)
        m = x.amax(-1, keepdim=True).clamp_min(-1e30)
        v = (x.sub_(m).exp_().sum(-1).log() + m[..., 0])
        out[row[there], h * g:(h + 1) * g] = v[there]
    return out


def _run_weigh(s):
    c = s["case"]
    if own:
        import sparse_attention_indexer_dsa_gb300 as dsa
        ws = _once(s, "ws", lambda: dsa.weigh_workspace(s["q"].shape[0], len(s["lens"]), s["max_q"], c["heads"], c["kv"], c["d"]))
        dsa.cache_weigh(_handle(s), s["weights"], s["q"], s["lse"], s["cu_q"], s["cu_k"], s["table"], s["max_q"],
                        s["max_k"], sm_scale=s["sm_scale"], ws=ws)
        return s["weights"]
    g = c["heads"] // c["kv"]
    pos = torch.arange(s["max_k"], device="cuda")[None].expand(len(s["lens"]), -1)
    n = torch.tensor([n for _, n in s["lens"]], device="cuda")[:, None]
    t = torch.tensor([t for t, _ in s["lens"]], device="cuda")[:, None]
    page, slot = _places(s, pos)
    live, old = pos < n, pos < n - t
    for h in range(c["kv"]):
        x, row, there = _logits(s, h)
        lse = s["lse"][row, h * g:(h + 1) * g]
        w = x.sub_(lse[..., None]).exp_().sum((1, 2))
        w = w + torch.where(old, s["weights"][page, h, slot], 0.0)
        s["weights"][page[live], h, slot[live]] = w[live]
    return s["weights"]


def _gathered(s):
    """Weights of every sequence's rows [sequences, heads, positions], and where there are rows."""
    pos = torch.arange(s["max_k"], device="cuda")[None].expand(len(s["lens"]), -1)
    page, slot = _places(s, pos)
    w = s["weights"][page, :, slot].transpose(1, 2)
    if s["case"]["shared"]:            # the heads' sum, one after the other in 32 bits
        total = w[:, 0]
        for h in range(1, w.shape[1]):
            total = total + w[:, h]
        w = total[:, None]
    return w, pos[:, None], torch.tensor([n for _, n in s["lens"]], device="cuda")[:, None, None]


def _run_choose(s):
    c = s["case"]
    if own:
        import sparse_attention_indexer_dsa_gb300 as dsa
        ws = _once(s, "ws", dsa.cache_workspace)
        return dsa.evict_select(s["weights"], s["cu_k"], s["table"], c["budget"], s["max_k"], sinks=c["sinks"],
                                recent=c["recent"], shared=c["shared"], ws=ws)
    w, pos, n = _gathered(s)
    w = torch.where((pos < c["sinks"]) | (pos >= n - c["recent"]), math.inf, w)
    w = torch.where(pos < n, w, -math.inf)
    idx = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :c["budget"]]
    idx = torch.sort(torch.where(idx < n, idx, 1 << 30), dim=-1).values
    kept = torch.full((*idx.shape[:2], c["budget"]), -1, dtype=torch.int32, device="cuda")
    kept[..., :idx.shape[-1]] = torch.where(idx < n, idx, -1)
    return kept, n.flatten().clamp_max(c["budget"]).to(torch.int32)


def _run_compact(s):
    c = s["case"]
    out = {n: t for n, t in s["cache"].items() if t is not None} | {"weights": s["weights"]}
    if own:
        import sparse_attention_indexer_dsa_gb300 as dsa
        ws = _once(s, "ws", dsa.cache_workspace)
        dsa.cache_compact(_handle(s), s["kept"], s["kept_len"], s["table"], weights=s["weights"], ws=ws)
    else:
        src = s["kept"].long().expand(-1, c["kv"], -1)
        dst = torch.arange(c["budget"], device="cuda").expand_as(src)
        head = torch.arange(c["kv"], device="cuda")[None, :, None].expand_as(src)
        live = dst < s["kept_len"][:, None, None]
        (sp, ss), (dp, ds) = _places(s, src.clamp_min(0)), _places(s, dst)
        sp, ss, dp, ds, head = sp[live], ss[live], dp[live], ds[live], head[live]
        for t in out.values():
            t[dp, head, ds] = t[sp, head, ss]
    return {n: t.view(torch.float8_e4m3fn) if n in ("k", "v") and t.dtype == torch.uint8 else t for n, t in out.items()}


# ---------------------------------------------------------------- 64 bits

def _e4m3_64():
    """Value of every E4M3 code (1 sign, 4 exponent bits of bias 7, 3 mantissa bits)."""
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        out[c] = (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) * (-1 if c & 128 else 1)
    return torch.tensor(out, device="cuda")


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "weigh": _exact_weigh, "choose": _exact_choose, "compact": _exact_compact}[case["op"]](s)


def _turn_64(x, s, sign):
    """Pairs as complex numbers, times e^(i sign angle)."""
    c = s["case"]
    n = c["rot"]
    step = torch.tensor([math.pow(10000.0, -2 * j / n) for j in range(n // 2)], dtype=torch.float64, device="cuda")
    a = sign * s["pos"].double()[:, None, None] * step
    u = torch.complex(torch.cos(a), torch.sin(a))
    y = x.clone()
    at = (slice(0, n // 2), slice(n // 2, n)) if c["pairs"] == "half" else (slice(0, n, 2), slice(1, n, 2))
    z = torch.complex(x[..., at[0]].contiguous(), x[..., at[1]].contiguous()) * u
    y[..., at[0]], y[..., at[1]] = z.real, z.imag
    return y


def _exact_norm(s):
    c, out = s["case"], []
    d = c["d"]
    for n in ("q", "k"):
        x, w = s[n].double(), s[n + "_weight"].double()
        mean = x.sum(-1, keepdim=True) / d if c["norm"] == "layer" else 0.0
        x = x - mean
        std = torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)
        if not c["back"]:
            y = x / std * w
            out.append(_turn_64(y if s[n + "_bias"] is None else y + s[n + "_bias"].double(), s, 1.0))
            continue
        g = _turn_64(s["d" + n].double(), s, -1.0)
        gw = g * w
        dx = gw / std - x * (gw * x).sum(-1, keepdim=True) / (d * std ** 3)
        if c["norm"] == "layer":
            dx = dx - (gw / std).sum(-1, keepdim=True) / d
        out.append((dx, (g * x / std).flatten(0, 1).sum(0), g.flatten(0, 1).sum(0)))
    if not c["back"]:
        return tuple(out)
    got = tuple(x for pair in zip(*out) for x in pair)
    return got if c["norm"] == "layer" else got[:4]


def _exact_weigh(s):
    c = s["case"]
    if work(c)["flops"] > 6e12:
        return None
    g, at, p = c["heads"] // c["kv"], 0, c["page"]
    out = s["weights"].double()
    codes = _e4m3_64()
    for i, (t, n) in enumerate(s["lens"]):
        pages = s["table"][i, :-(-n // p)].long()
        for h in range(c["kv"]):
            k = s["cache"]["k"][pages, h].reshape(-1, c["d"])[:n]
            if c["prec"] == "bf16":
                k = k.double()
            else:
                e = s["cache"]["k_scale"][pages, h].reshape(-1, _scale_width(c))[:n].double() - 127
                k = codes[k.long()] * torch.exp2(e).repeat_interleave(c["d"] // e.shape[1], dim=1)
            whole = out[pages, h].reshape(-1)
            whole[n - t:n] = 0.0
            step = max(1, int(2e8) // (g * n))
            for j in range(0, t, step):
                m = min(step, t - j)
                q = s["q"][at + j:at + j + m, h * g:(h + 1) * g].double() * s["sm_scale"]
                a = torch.exp(torch.einsum("mgd,sd->mgs", q, k) - s["lse"][at + j:at + j + m, h * g:(h + 1) * g, None].double())
                last = torch.arange(n - t + j, n - t + j + m, device="cuda")
                a *= (torch.arange(n, device="cuda") <= last[:, None])[:, None]
                whole[:n] += a.sum((0, 1))
            out[pages, h] = whole.reshape(-1, p)
        at += t
    return out


def _exact_choose(s):
    c = s["case"]
    heads = 1 if c["shared"] else c["kv"]
    weights, table = s["weights"].cpu().numpy(), s["table"].cpu().numpy()
    kept = np.full((len(s["lens"]), heads, c["budget"]), -1, np.int32)
    for i, (_, n) in enumerate(s["lens"]):
        pages = table[i, :-(-n // c["page"])]
        w = np.moveaxis(weights[pages], 1, 0).reshape(c["kv"], -1)[:, :n]
        if c["shared"]:                # (defined as the sum in 32 bits, head after head)
            total = np.zeros(n, np.float32)
            for row in w:
                total = total + row
            w = total[None]
        for h in range(heads):
            must = np.arange(n)
            must = (must < c["sinks"]) | (must >= n - c["recent"])
            order = np.lexsort((np.arange(n), -w[h].astype(np.float64), ~must))
            best = np.sort(order[:c["budget"]])
            kept[i, h, :len(best)] = best
    lens = np.array([min(n, c["budget"]) for _, n in s["lens"]], np.int32)
    return torch.from_numpy(kept).cuda(), torch.from_numpy(lens).cuda()


def _exact_compact(s):
    c, codes = s["case"], _e4m3_64()
    out = {n: t.clone() for n, t in s["cache"].items() if t is not None} | {"weights": s["weights"].clone()}
    for i in range(len(s["lens"])):
        pages, m = s["table"][i].long(), int(s["kept_len"][i])
        pages = pages[pages >= 0]
        for h in range(c["kv"]):
            src = s["kept"][i, 0 if c["shared"] else h, :m].long()
            for t in out.values():
                rows = t[pages, h].flatten(0, 1)
                rows[:m] = rows[src]
                t[pages, h] = rows.reshape(len(pages), c["page"], *rows.shape[1:])
    return {n: t if "scale" in n else codes[t.long()] if t.dtype == torch.uint8 else t.double() for n, t in out.items()}
