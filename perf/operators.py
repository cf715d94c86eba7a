"""What the paged-cache operators are measured on: writing a quantised cache,
reading it back, attention of new tokens over it, and attention over the rows
that the indexer selected.

`own` False: the plain forms below (elementary torch operations, 32 bits).
`own` True: the same work through the package's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 32          # elements that share one scale in MXFP8
FAR = 32768         # the longest document of the workloads


# ---------------------------------------------------------------- cases

def listed():
    return [
        # --- cache_write: one token of each of 16 running sequences (latency)
        dict(name="write_step", op="write", seqs=16, t_lo=1, t_hi=1, s_lo=500, s_hi=8192, kv=8, d=128, prec="mxfp8",
             page=64, src="bf16", values=True, mix=1),
        # a whole prompt enters the cache in MXFP8, K and V slices of one projection
        dict(name="write_prompt", op="write", seqs=1, t_lo=32768, t_hi=32768, s_lo=32768, s_hi=32768, kv=8, d=128,
             prec="mxfp8", page=64, src="bf16", values=True, mix=2),
        # a packed batch of ragged chunks from FP32 carriers, one scale a row, narrow heads, small pages
        dict(name="write_ragged", op="write", seqs=9, t_lo=100, t_hi=6000, s_lo=6000, s_hi=9001, kv=5, d=64,
             prec="fp8", page=16, src="f32", values=True, mix=3),
        # --- cache_read: index keys of a few short sequences (latency)
        dict(name="read_short", op="read", seqs=5, s_lo=1, s_hi=130, kv=1, d=128, prec="mxfp8", page=64, values=False,
             to="operands", mix=4),
        # index keys of eight long documents as the operands of the scoring kernel
        dict(name="read_index_keys", op="read", seqs=8, s_lo=20000, s_hi=65536, kv=1, d=128, prec="mxfp8", page=64,
             values=False, to="operands", mix=5),
        # keys and values back as BF16, for a consumer that has no 8-bit path
        dict(name="read_bf16", op="read", seqs=7, s_lo=511, s_hi=8191, kv=8, d=128, prec="fp8", page=32, values=True,
             to="bf16", mix=6),
        # --- paged_attention: the first tokens of one small sequence (latency)
        dict(name="attend_first", op="attend", seqs=1, t_lo=1, t_hi=1, s_lo=17, s_hi=17, heads=16, kv=4, d=64,
             prec="bf16", page=16, topk=0, mix=7),
        # a serving step: 64 sequences, one token each, 8-bit cache
        dict(name="attend_step", op="attend", seqs=64, t_lo=1, t_hi=1, s_lo=2048, s_hi=16384, heads=64, kv=8, d=128,
             prec="mxfp8", page=64, topk=0, mix=8),
        # a mixed batch: chunks of odd lengths behind caches of odd lengths
        dict(name="attend_ragged", op="attend", seqs=6, t_lo=1, t_hi=1500, s_lo=1501, s_hi=8191, heads=32, kv=4, d=128,
             prec="fp8", page=16, topk=0, mix=9),
        # a chunk of a long prompt
        dict(name="attend_chunk", op="attend", seqs=1, t_lo=4096, t_hi=4096, s_lo=32768, s_hi=32768, heads=64, kv=8,
             d=128, prec="bf16", page=64, topk=0, mix=10),
        # --- attention over the indexer's rows: a serving step, one latent key head
        dict(name="selected_step", op="attend", seqs=32, t_lo=1, t_hi=1, s_lo=4000, s_hi=32768, heads=64, kv=1, d=128,
             prec="mxfp8", page=64, topk=2048, mix=11),
        # a chunk of a long prompt, every query with its own 2048 keys
        dict(name="selected_chunk", op="attend", seqs=1, t_lo=4096, t_hi=4096, s_lo=32768, s_hi=32768, heads=64, kv=1,
             d=128, prec="bf16", page=64, topk=2048, mix=12),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm of the range."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "selected", "selected"])
    c = dict(op="attend" if op == "selected" else op, d=rng.choice([64, 128]), prec=rng.choice(["bf16", "mxfp8", "fp8"]),
             page=rng.choice([16, 32, 64, 128]), mix=rng.randrange(1, 1 << 30))
    if op in ("write", "read"):
        c["seqs"] = _spread(rng, 1, 64)
        top = max(1, 32768 // c["seqs"])
        c["s_lo"] = _spread(rng, 1, top)
        c["s_hi"] = _spread(rng, c["s_lo"], top)
        c["kv"] = rng.choice([1, 2, 3, 4, 8])
        c["values"] = rng.random() < 0.7
        if op == "write":
            c["t_lo"] = _spread(rng, 1, c["s_lo"])
            c["t_hi"] = _spread(rng, c["t_lo"], c["s_hi"])
            c["src"] = rng.choice(["bf16", "f32"])
        else:
            c["to"] = rng.choice(["operands", "bf16"])
        return c
    c["kv"], group = rng.choice([(1, 4), (1, 16), (1, 32), (1, 64), (2, 5), (4, 4), (4, 8), (8, 1), (8, 8)])
    c["heads"] = c["kv"] * group
    c["topk"] = rng.choice([32, 256, 700, 2048]) if op == "selected" else 0
    c["seqs"] = _spread(rng, 1, 64)
    top = max(64, 65536 // c["seqs"])
    c["s_lo"] = _spread(rng, 1, min(top, FAR))
    c["s_hi"] = _spread(rng, c["s_lo"], min(top, FAR))
    most = max(1, min(c["s_lo"], 2048 // c["seqs"]))
    c["t_lo"] = 1 if rng.random() < 0.5 else _spread(rng, 1, most)
    c["t_hi"] = _spread(rng, c["t_lo"], most) if c["t_lo"] > 1 else rng.choice([1, most])
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


def _listed_keys(case):
    """Keys that each sequence's queries attend to, summed."""
    total = 0
    for t, s in _lengths(case):
        k = case["topk"] or s
        first = s - t + 1                      # visible keys of the first query
        full = max(0, min(t, s - max(k, first) + 1)) if k < s else 0     # queries that see k or more
        grow = t - full
        total += full * k + grow * first + grow * (grow - 1) // 2
    return total


def work(case):
    lens = _lengths(case)
    kv, d = case["kv"], case["d"]
    row = {"bf16": 2 * d, "mxfp8": d + d // BLOCK, "fp8": d + 1}[case["prec"]]      # bytes of a cached row
    if case["op"] == "write":
        rows = sum(t for t, _ in lens) * kv * (2 if case["values"] else 1)
        return {"bytes": rows * (row + d * (2 if case["src"] == "bf16" else 4)), "flops": 3 * rows * d}
    if case["op"] == "read":
        rows = sum(s for _, s in lens) * kv * (2 if case["values"] else 1)
        return {"bytes": rows * (row + (row if case["to"] == "operands" else 2 * d)), "flops": rows * d}
    h = case["heads"]
    rows = sum(min(s, t * case["topk"]) if case["topk"] else s for t, s in lens) * kv * 2
    tokens = sum(t for t, _ in lens)
    return {"bytes": rows * row + tokens * (4 * h * d + 4 * case["topk"]), "flops": 4 * h * d * _listed_keys(case)}


# ---------------------------------------------------------------- inputs

def _values(shape, gen, dtype, scale=1.0):
    """Activations: normal, one in a hundred an outlier."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.01, 8.0 * scale, scale)
    return x.to(dtype)


def _scale_width(case):
    return case["d"] // BLOCK if case["prec"] == "mxfp8" else 1


def _cache(case, gen, lens):
    """Pages that hold valid rows everywhere (slots not in use hold older rows)
    and a table that spreads the sequences' pages over them."""
    p = case["page"]
    need = [-(-s // p) for _, s in lens]
    pages = sum(need) + 3
    shape = (pages, case["kv"], p, case["d"])
    names = ["k", "v"] if case.get("values", True) else ["k"]
    cache = {}
    for n in names:
        if case["prec"] == "bf16":
            cache[n] = _values(shape, gen, torch.bfloat16)
            cache[n + "_scale"] = None
        else:
            code = torch.randint(0, 0x78, shape, generator=gen, device="cuda", dtype=torch.uint8)
            code |= torch.randint(0, 2, shape, generator=gen, device="cuda", dtype=torch.uint8) << 7
            code[torch.rand(shape, generator=gen, device="cuda") < 0.3] &= 0x87      # the small half of the range
            cache[n] = code
            cache[n + "_scale"] = torch.randint(118, 121, shape[:3] + (_scale_width(case),), generator=gen,
                                                device="cuda", dtype=torch.uint8)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return cache, table


def _prefix(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def _select(case, gen, lens):
    """Each query's rows as the indexer gives them: ascending, -1 behind the
    last, every visible key while there are no more than topk."""
    rows = []
    for t, s in lens:
        for i0 in range(0, t, 512):
            n = min(512, t - i0)
            last = torch.arange(s - t + i0, s - t + i0 + n, device="cuda")[:, None]
            key = torch.arange(s, device="cuda")[None, :]
            r = torch.rand((n, s), generator=gen, device="cuda")
            r += 0.5 * (key > last - 1024)                        # recent keys are picked more often
            r = torch.where(key <= last, r, -1.0)
            k = min(case["topk"], s)
            v, idx = torch.topk(r, k, dim=1)
            idx = torch.where(v >= 0, idx, s)
            idx = torch.sort(idx, dim=1).values
            idx = torch.where(idx == s, -1, idx).to(torch.int32)
            if k < case["topk"]:
                idx = torch.nn.functional.pad(idx, (0, case["topk"] - k), value=-1)
            rows.append(idx)
    idx = torch.cat(rows)
    return idx, (idx >= 0).sum(1).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    lens = _lengths(case)
    cache, table = _cache(case, gen, lens)
    t_total, s_total = sum(t for t, _ in lens), sum(s for _, s in lens)
    st = dict(case=case, lens=lens, cache=cache, table=table, cu_q=_prefix([t for t, _ in lens]),
              cu_k=_prefix([s for _, s in lens]), s_total=s_total)
    if case["op"] == "write":
        dt = torch.bfloat16 if case["src"] == "bf16" else torch.float32
        n = 2 * case["kv"] if case["values"] else case["kv"]
        kv = _values((t_total, n, case["d"]), gen, dt)            # one projection gives both
        st["new_k"] = kv[:, :case["kv"]]
        st["new_v"] = kv[:, case["kv"]:] if case["values"] else None
    elif case["op"] == "attend":
        st["q"] = _values((t_total, case["heads"], case["d"]), gen, torch.bfloat16)
        st["sm_scale"] = 1.0 / math.sqrt(case["d"])
        if case["topk"]:
            st["topk_idx"], st["topk_len"] = _select(case, gen, lens)
    if own:
        import sparse_attention_indexer_dsa_gb300 as dsa
        st["handle"] = dsa.PagedCache(k=cache["k"], k_scale=cache["k_scale"], v=cache.get("v"),
                                      v_scale=cache.get("v_scale"), prec=case["prec"])
        if case["op"] == "attend":
            st["max_q"], st["max_k"] = max(t for t, _ in lens), max(s for _, s in lens)
            st["ws"] = dsa.attention_workspace(t_total, len(lens), st["max_q"], case["heads"], case["kv"], case["d"],
                                               topk_width=case["topk"])
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    c = state["case"]
    return {"write": _run_write, "read": _run_read, "attend": _run_attend}[c["op"]](state)


def _codes(x):
    """8-bit codes as the numbers they stand for."""
    return x if x is None or x.dtype != torch.uint8 else x.view(torch.float8_e4m3fn)


def _run_write(s):
    cache = s["cache"]
    if own:
        import sparse_attention_indexer_dsa_gb300 as dsa
        dsa.cache_write(s["handle"], s["new_k"], s["new_v"], s["cu_q"], s["cu_k"], s["table"])
    else:
        page, slot = _places(s, new_only=True)
        for n in ("k", "v"):
            x = s["new_" + n]
            if x is None:
                continue
            y, e = _quantise(x.float(), s["case"])
            cache[n][page, :, slot] = y
            if e is not None:
                cache[n + "_scale"][page, :, slot] = e
    return {n: _codes(t) if "scale" not in n else t for n, t in cache.items() if t is not None}


def _run_read(s):
    c = s["case"]
    if own:
        import sparse_attention_indexer_dsa_gb300 as dsa
        got = dsa.cache_read(s["handle"], s["cu_k"], s["table"], s["s_total"],
                             out_prec=None if c["to"] == "operands" else "bf16")
        out = dict(zip(("k", "k_scale", "v", "v_scale"), got))
    else:
        page, slot = _places(s)
        out = {}
        for n, t in s["cache"].items():
            if t is None:
                continue
            if c["to"] == "operands":
                out[n] = t[page, :, slot]
            elif "scale" not in n:
                out[n] = _rows(s, n, page, slot).to(torch.bfloat16)
    return {n: _codes(t) if "scale" not in n else t for n, t in out.items() if t is not None}


def _run_attend(s):
    c = s["case"]
    if own:
        import sparse_attention_indexer_dsa_gb300 as dsa
        return dsa.paged_attention(s["q"], s["handle"], s["cu_q"], s["cu_k"], s["table"], s["max_q"], s["max_k"],
                                   sm_scale=s["sm_scale"], topk_idx=s.get("topk_idx"), topk_len=s.get("topk_len"),
                                   ws=s["ws"])
    out = torch.empty_like(s["q"])
    page, slot = _places(s)
    k, v = _rows(s, "k", page, slot), _rows(s, "v", page, slot)
    tq = sk = 0
    for t, n in s["lens"]:
        kd, vd = k[sk:sk + n], v[sk:sk + n]
        step = max(1, int(2e9) // (c["heads"] * (n if not c["topk"] else c["topk"] * (1 + 2 * c["d"] // c["heads"])) * 4))
        for i in range(0, t, step):
            m = min(step, t - i)
            q = s["q"][tq + i:tq + i + m].float().reshape(m, c["kv"], -1, c["d"])
            pos = torch.arange(n - t + i, n - t + i + m, device="cuda")
            if c["topk"]:
                idx = s["topk_idx"][tq + i:tq + i + m].long()
                off = (idx < 0) | (idx > pos[:, None])
                idx = idx.clamp(0, n - 1)
                lg = torch.matmul(q, kd[idx].permute(0, 2, 3, 1)) * s["sm_scale"]         # [m, kv, group, topk]
                p = _softmax(lg, off[:, None, None, :])
                o = torch.matmul(p, vd[idx].permute(0, 2, 1, 3))
            else:
                lg = torch.matmul(q.permute(1, 2, 0, 3).reshape(c["kv"], -1, c["d"]), kd.permute(1, 2, 0))
                lg = (lg * s["sm_scale"]).reshape(c["kv"], -1, m, n)
                off = torch.arange(n, device="cuda")[None, :] > pos[:, None]
                p = _softmax(lg, off).reshape(c["kv"], -1, n)
                o = torch.matmul(p, vd.permute(1, 0, 2)).reshape(c["kv"], -1, m, c["d"]).permute(2, 0, 1, 3)
            out[tq + i:tq + i + m] = o.reshape(m, c["heads"], c["d"]).to(out.dtype)
        tq, sk = tq + t, sk + n
    return out


def _places(s, new_only=False):
    """Page and slot of every cached (or newly written) position, packed."""
    p = s["case"]["page"]
    page, slot = [], []
    for i, (t, n) in enumerate(s["lens"]):
        pos = torch.arange(n - t if new_only else 0, n, device="cuda")
        page.append(s["table"][i, pos // p].long())
        slot.append(pos % p)
    return torch.cat(page), torch.cat(slot)


def _rows(s, name, page, slot):
    """Cached rows as 32-bit values, [positions, kv heads, d]."""
    x = s["cache"][name][page, :, slot]
    if s["case"]["prec"] == "bf16":
        return x.float()
    e = s["cache"][name + "_scale"][page, :, slot].int() - 127
    x = x.view(torch.float8_e4m3fn).float()
    return (x.reshape(*x.shape[:2], e.shape[-1], -1) * _power(e)[..., None]).reshape(x.shape)


def _quantise(x, case):
    """Codes and scale bytes (None for BF16): the smallest exponent that
    saturates no element, then round to nearest even."""
    if case["prec"] == "bf16":
        return x.to(torch.bfloat16), None
    b = x.reshape(*x.shape[:2], _scale_width(case), -1)
    amax = b.abs().amax(-1)
    m, e = torch.frexp(amax)                              # amax = m 2^e, 448 = 0.875 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(-127, 127)
    e = torch.where(amax == 0, -127, e)
    y = (b * _power(-e)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return y.reshape(x.shape), (e + 127).to(torch.uint8)


def _power(e):
    """2 to whole exponents of [-127, 127], from the bits: no rounding."""
    e = e.to(torch.int32)
    return torch.where(e < -126, 1 << 22, (e + 127) << 23).to(torch.int32).view(torch.float32)


def _softmax(x, off):
    x = x.masked_fill_(off, -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    return x / x.sum(-1, keepdim=True).clamp_min(1e-30)


# ---------------------------------------------------------------- 64 bits

def _e4m3_64():
    """Value of every E4M3 code (1 sign, 4 exponent bits of bias 7, 3 mantissa bits)."""
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        out[c] = (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) * (-1 if c & 128 else 1)
    return torch.tensor(out, device="cuda")


def _stored_64(cache, name, case, d_idx, h, r):
    """Rows of one head, from the page list of one sequence, in 64 bits."""
    x = cache[name][d_idx, h].reshape(-1, case["d"])[:r]
    if case["prec"] == "bf16":
        return x.double()
    sc = cache[name + "_scale"][d_idx, h].reshape(-1, _scale_width(case))[:r]
    val = _e4m3_64()[x.long()]
    return val * _power_64(sc.long() - 127).repeat_interleave(case["d"] // _scale_width(case), dim=1)


def _power_64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _format_64(x, case):
    """The definition of the stored format: exponent by search, payload by rounding to the format's spacing."""
    if case["prec"] == "bf16":
        _, e = torch.frexp(x)
        step = _power_64((e - 8).clamp_min(-133))
        return torch.round(x / step) * step, None
    w = _scale_width(case)
    b = x.reshape(*x.shape[:-1], w, -1)
    top = b.abs().amax(-1)
    rough = torch.floor(torch.log2(torch.where(top > 0, top, 1.0) / 448)) - 1
    e = torch.where(top > 0, rough, -127.0).clamp_min(-127)
    for _ in range(4):
        e = torch.where(top > 448 * _power_64(e), e + 1, e)
    y = b / _power_64(e)[..., None]
    _, ye = torch.frexp(y)
    step = _power_64((ye - 4).clamp_min(-9))
    return (torch.round(y / step) * step).reshape(x.shape), (e + 127).to(torch.uint8)


def exact(case, seed):
    if case["op"] == "attend" and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    cache, page, kv, d = s["cache"], case["page"], case["kv"], case["d"]
    lists = [s["table"][i, :-(-n // page)].long() for i, (_, n) in enumerate(s["lens"])]
    if case["op"] == "write":
        out = {}
        for name in ("k", "v"):
            if name not in cache:
                continue
            w = _scale_width(case)
            old = cache[name].double() if case["prec"] == "bf16" else _e4m3_64()[cache[name].long()]
            esc = None if case["prec"] == "bf16" else cache[name + "_scale"].clone()
            at = 0
            for (t, n), pages in zip(s["lens"], lists):
                y, e = _format_64(s["new_" + name][at:at + t].double(), case)
                for h in range(kv):
                    whole = old[pages, h].reshape(-1, d)
                    whole[n - t:n] = y[:, h]
                    old[pages, h] = whole.reshape(-1, page, d)
                    if e is not None:
                        ew = esc[pages, h].reshape(-1, w)
                        ew[n - t:n] = e[:, h]
                        esc[pages, h] = ew.reshape(-1, page, w)
                at += t
            out[name] = old
            if esc is not None:
                out[name + "_scale"] = esc
        return {n: out[n] for n in cache if n in out}
    if case["op"] == "read":
        out = {}
        for name in ("k", "v"):
            if name not in cache:
                continue
            if case["to"] == "bf16" or case["prec"] == "bf16":
                # BF16 holds E4M3 times a power of two exactly
                out[name] = torch.cat([torch.stack([_stored_64(cache, name, case, p, h, n) for h in range(kv)], 1)
                                       for p, (_, n) in zip(lists, s["lens"])])
            else:
                val = _e4m3_64()
                for nm in (name, name + "_scale"):
                    x = torch.cat([torch.stack([cache[nm][p, h].reshape(-1, cache[nm].shape[-1])[:n]
                                                for h in range(kv)], 1) for p, (_, n) in zip(lists, s["lens"])])
                    out[nm] = val[x.long()] if nm == name else x
        return {n: out[n] for n in cache if n in out}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group, at = case["heads"] // kv, 0
    for (t, n), pages in zip(s["lens"], lists):
        for h in range(kv):
            k, v = _stored_64(cache, "k", case, pages, h, n), _stored_64(cache, "v", case, pages, h, n)
            step = max(1, int(3e8) // (group * (case["topk"] * (1 + 2 * d // group) if case["topk"] else n)))
            for i in range(0, t, step):
                m = min(step, t - i)
                q = s["q"][at + i:at + i + m, h * group:(h + 1) * group].double() * s["sm_scale"]
                last = torch.arange(n - t + i, n - t + i + m, device="cuda")
                if case["topk"]:
                    idx = s["topk_idx"][at + i:at + i + m].long()
                    see = ((idx >= 0) & (idx <= last[:, None]))[:, None]
                    idx = idx.clamp_min(0)
                    a = torch.einsum("mgd,mwd->mgw", q, k[idx])
                else:
                    see = (torch.arange(n, device="cuda") <= last[:, None])[:, None]
                    a = torch.einsum("mgd,sd->mgs", q, k)
                a = torch.where(see, a, -math.inf)
                a = torch.exp(a - a.amax(-1, keepdim=True))
                a = torch.where(see, a, 0.0)
                z = a.sum(-1, keepdim=True)
                o = torch.einsum("mgw,mwd->mgd", a, v[idx]) if case["topk"] else torch.einsum("mgs,sd->mgd", a, v)
                out[at + i:at + i + m, h * group:(h + 1) * group] = o / z
        at += t
    return out
