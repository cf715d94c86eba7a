"""Plain 64-bit forms of the paged-cache operators and the random batches their
tests share (numpy; the formats come from the oracle)."""
import numpy as np
import torch

import oracle.dsa_oracle as O

BF16_HALF = 2.0 ** -8        # a BF16 rounding is off by at most half a step, relative
F32_STEP = 2.0 ** -23        # FP32 sums may truncate: a whole step per addition


def scale_width(prec, D):
    return {"bf16": 0, "mxfp8": D // 32, "fp8": 1}[prec]


def pow2(e):
    return np.ldexp(1.0, np.asarray(e, np.int64))


def quantise(x, prec, rule="nosat"):
    """float64 [..., D] -> (stored array, scale bytes or None): BF16 bit patterns or E4M3 codes."""
    x = np.asarray(x, np.float64)
    if prec == "bf16":
        return O.float_to_bf16_bits(O.round_bf16(x)), None
    D = x.shape[-1]
    rows = x.reshape(-1, D)
    n = scale_width(prec, D)
    blocks = rows.reshape(-1, D // n)
    e = O.mx_block_exponents(np.abs(blocks).max(1), rule)
    codes = O.e4m3_encode(O.round_e4m3_sat(blocks / pow2(e)[:, None]))
    return codes.reshape(x.shape).astype(np.uint8), (e + 127).astype(np.uint8).reshape(x.shape[:-1] + (n,))


def values(stored, scales, prec):
    """Stored rows as float64 values."""
    if prec == "bf16":
        return O.bf16_bits_to_float(stored).astype(np.float64)
    v = O.e4m3_decode(stored.reshape(-1)).reshape(stored.shape).astype(np.float64)
    n = scales.shape[-1]
    b = v.reshape(v.shape[:-1] + (n, -1)) * pow2(scales.astype(np.int64) - 127)[..., None]
    return b.reshape(v.shape)


class Batch:
    """Sequences of (new, cached) tokens over randomly placed pages.  Slots that no
    sequence uses hold NaN (BF16) or the NaN code with the largest scale; page
    table entries behind a sequence's last page hold a page that does not exist."""

    def __init__(self, rng, lens, n_kv, D, page, prec, values_too=True, extra_pages=2, std=1.0, pad_q=0):
        self.lens, self.n_kv, self.D, self.page, self.prec = lens, n_kv, D, page, prec
        need = [-(-s // page) for _, s in lens]
        self.num_pages = sum(need) + extra_pages
        self.max_pages = max(1, max(need)) + 1
        order = rng.permutation(self.num_pages)
        self.table = np.full((len(lens), self.max_pages), 1 << 30, np.int32)
        at = 0
        for d, n in enumerate(need):
            self.table[d, :n] = order[at:at + n]
            at += n
        self.cu_q = np.concatenate([[0], np.cumsum([t for t, _ in lens])]).astype(np.int32)
        self.cu_k = np.concatenate([[0], np.cumsum([s for _, s in lens])]).astype(np.int32)
        self.total_q = int(self.cu_q[-1]) + pad_q
        self.total_k = int(self.cu_k[-1])
        self.names = ["k", "v"] if values_too else ["k"]
        self.rows, self.pages, self.scales = {}, {}, {}
        n = scale_width(prec, D)
        for nm in self.names:
            x = rng.standard_normal((self.total_k, n_kv, D)) * std
            st, sc = quantise(x, prec)
            self.rows[nm] = values(st, sc, prec)
            shape = (self.num_pages, n_kv, page, D)
            self.pages[nm] = np.full(shape, 0x7FC0, np.uint16) if prec == "bf16" else np.full(shape, 0x7F, np.uint8)
            self.scales[nm] = None if n == 0 else np.full(shape[:3] + (n,), 254, np.uint8)
            for d in range(len(lens)):
                for pos in range(lens[d][1]):
                    pg, sl = self.table[d, pos // page], pos % page
                    self.pages[nm][pg, :, sl] = st[self.cu_k[d] + pos]
                    if n:
                        self.scales[nm][pg, :, sl] = sc[self.cu_k[d] + pos]

    def cache(self, dsa):
        """The pages on the GPU."""
        def up(a):
            if a is None:
                return None
            t = torch.from_numpy(np.ascontiguousarray(a.view(np.int16) if a.dtype == np.uint16 else a)).cuda()
            return t.view(torch.bfloat16) if a.dtype == np.uint16 else t
        return dsa.PagedCache(up(self.pages["k"]), up(self.scales["k"]), up(self.pages.get("v")),
                              up(self.scales.get("v")), self.prec)

    def dev(self, name):
        return torch.from_numpy(getattr(self, name)).cuda()


def attention(b, q, group, sm_scale, sel=None, sel_len=None):
    """out, lse and the error bound of a kernel that multiplies exactly,
    accumulates in FP32 and rounds the weights and the result to BF16 once.

    With w the softmax weights and A = sum w |v|: a logit is off by at most
    dl = scale (D + 2) 2^-23 sum |q k| + 2^-22 |logit - max| (the sum, the scaling and the
    argument of the exponential), a weight by exp(2 dl) - 1 <= 4 dl relative in
    numerator and denominator together plus 2^-8 (its rounding) and 2^-21 (the
    exponential), the sums over n keys by 2 n 2^-23, the result by 2^-8."""
    T, H, D = q.shape
    out, lse, tol, ltol = np.zeros((T, H, D)), np.full((T, H), -np.inf), np.zeros((T, H, D)), np.zeros((T, H))
    K, V = b.rows["k"], b.rows["v"]
    for d, (t, s) in enumerate(b.lens):
        for i in range(t):
            r = b.cu_q[d] + i
            pos = s - t + i
            keys = np.arange(pos + 1)
            if sel is not None:
                keys = sel[r] if sel_len is None else sel[r][:max(0, sel_len[r])]
                keys = keys[(keys >= 0) & (keys <= pos)]
            if len(keys) == 0:
                continue
            for h in range(H):
                k, v = K[b.cu_k[d] + keys, h // group], V[b.cu_k[d] + keys, h // group]
                lg = sm_scale * (k @ q[r, h])
                mag = sm_scale * (np.abs(k) @ np.abs(q[r, h]))
                m = lg.max()
                w = np.exp(lg - m)
                z = w.sum()
                w /= z
                out[r, h] = w @ v
                lse[r, h] = m + np.log(z)
                dl = ((D + 2) * F32_STEP * mag + 2.0 ** -22 * (np.abs(lg - m) + 8 + np.abs(m))).max()
                A = w @ np.abs(v)
                rel = 4 * dl + 2.0 ** -21 + 2 * len(keys) * F32_STEP
                tol[r, h] = (rel + BF16_HALF) * A * 1.01 + BF16_HALF * np.abs(out[r, h])
                ltol[r, h] = rel + 2.0 ** -22 * (abs(lse[r, h]) + 8)
    return out, lse, tol + 1e-30, ltol
