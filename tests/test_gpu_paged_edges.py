"""Attention over the paged cache where a kernel kind, a plan or a limit changes.
The reference and its derived bound are those of tests/paged_ref.py."""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_dsa_gb300 as dsa
from sparse_attention_indexer_dsa_gb300 import _abi
from tests.gpu_util import dev, host
from tests.paged_ref import Batch, attention, quantise, values
from tests.test_gpu_paged_attention import _close, _queries, _run, _selection

pytestmark = pytest.mark.gpu

# (tokens, cached): pairs of query tiles, single tiles, listed keys
KINDS = {"pair": ([(300, 900)], 0), "solo": ([(1, 900), (1, 300)], 0), "list": ([(3, 900)], 400)}


@pytest.mark.parametrize("heads", [8, 24])   # narrow tiles, tiles of 128 rows
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
def test_a_withheld_tile_times_out_and_the_next_call_is_clean(prec, kind, heads):
    rng = np.random.default_rng(51)
    lens, W = KINDS[kind]
    b = Batch(rng, lens, 1, 128, 64, prec)
    sel, _ = _selection(rng, b, W, "sorted") if W else (None, None)
    q, qd = _queries(rng, b.total_q, heads, 128)
    max_q, max_k = max(t for t, _ in lens), max(s for _, s in lens)
    ws = dsa.attention_workspace(b.total_q, len(lens), max_q, heads, 1, 128, W)
    lib = _abi.load()
    args = (qd, b.cache(dsa), b.dev("cu_q"), b.dev("cu_k"), b.dev("table"), max_q, max_k)
    lst = None if sel is None else dev(sel)
    try:
        lib.dsa_idx_test_set_timeout_ns(50_000_000)
        lib.dsa_idx_test_set_fault_inject(1)
        dsa.paged_attention(*args, topk_idx=lst, ws=ws)
        assert dsa.read_status(ws) == _abi.DSA_ERR_TIMEOUT
    finally:
        lib.dsa_idx_test_set_fault_inject(0)
        lib.dsa_idx_test_set_timeout_ns(2_000_000_000)
    out = dsa.paged_attention(*args, topk_idx=lst, ws=ws)
    assert dsa.read_status(ws) == 0
    want, _, tol, _ = attention(b, q, heads, 128 ** -0.5, sel)
    _close(host(out.double()), want, tol)


@pytest.mark.parametrize("page", [8, 16, 256, 1024])
@pytest.mark.parametrize("prec,D", [("bf16", 64), ("mxfp8", 64), ("mxfp8", 128), ("fp8", 128)])
def test_small_and_large_pages(prec, D, page):
    rng = np.random.default_rng(52)
    b = Batch(rng, [(1, 391), (70, 300), (0, 3), (2, 2), (1, 1040)], 2, D, page, prec)
    _run(b, rng, 8, 4)
    sel, lens = _selection(rng, b, 150, "wild")
    _run(b, rng, 8, 4, sel, lens)


@pytest.mark.parametrize("group", [32, 33, 65, 100, 128])
@pytest.mark.parametrize("prec,D", [("bf16", 128), ("mxfp8", 128), ("fp8", 64)])
def test_heads_to_a_key_head(prec, D, group):
    """A tile of 128 rows holds 4 tokens .. 1, its last rows unused; above 64 rows an 8-bit
    cache of 128 elements leaves room for one stream only."""
    rng = np.random.default_rng(53)
    b = Batch(rng, [(3, 200), (1, 385), (9, 9)], 2, D, 32, prec)
    _run(b, rng, 2 * group, group)
    sel, lens = _selection(rng, b, 170, "wild")
    _run(b, rng, 2 * group, group, sel, lens)


@pytest.mark.parametrize("group,lens", [(4, [(2, 5000)] + [(1, 3)] * 40), (1, [(200, 2600), (1, 1), (40, 40)]),
                                        (16, [(1, 9000), (0, 0), (0, 700)])])
@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
def test_one_long_sequence_among_short_ones(prec, group, lens):
    rng = np.random.default_rng(54)
    b = Batch(rng, lens, 1, 64, 128, prec)
    _run(b, rng, group, group)


@pytest.mark.parametrize("kw", [dict(), dict(W=2100)])
@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
def test_the_same_call_gives_the_same_bits(prec, kw):
    rng = np.random.default_rng(55)
    b = Batch(rng, [(2, 6000), (1, 2500)], 2, 128, 64, prec)
    sel = _selection(rng, b, kw["W"], "sorted")[0] if kw else None
    first = _run(b, np.random.default_rng(56), 16, 8, sel)
    for _ in range(3):
        again = _run(b, np.random.default_rng(56), 16, 8, sel)
        assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.parametrize("prec", ["mxfp8", "fp8"])
@pytest.mark.parametrize("W", [0, 140])
@pytest.mark.parametrize("k_shift", [-90, 7, 60])
def test_scales_over_their_range(prec, W, k_shift):
    """Keys times 2^k_shift (queries times its inverse), values of every row times another power:
    a factor of two steps in the widening, codes whose values are subnormal in BF16."""
    rng = np.random.default_rng(57)
    b = Batch(rng, [(2, 260), (20, 150)], 1, 128, 16, prec)
    shifts = rng.choice([-126, -60, 0, 8, 9, 50, 100], b.total_k)
    for d, (_, s) in enumerate(b.lens):
        for pos in range(s):
            pg, sl, r = b.table[d, pos // 16], pos % 16, b.cu_k[d] + pos
            for nm, e in (("k", k_shift), ("v", int(shifts[r]))):
                was = b.scales[nm][pg, :, sl].astype(int)
                now = np.clip(was + e, 0, 254)
                b.scales[nm][pg, :, sl] = now
                step = (now - was)[0]
                b.rows[nm][r] *= np.repeat(np.ldexp(1.0, step), 128 // len(step))
    q, qd = _queries(rng, b.total_q, 4, 128)
    q, qd = q * 2.0 ** -k_shift, qd * 2.0 ** -k_shift
    sel = _selection(rng, b, W, "sorted")[0] if W else None
    out = dsa.paged_attention(qd, b.cache(dsa), b.dev("cu_q"), b.dev("cu_k"), b.dev("table"), 20, 260,
                              topk_idx=None if sel is None else dev(sel))
    want, _, tol, _ = attention(b, q, 4, 128 ** -0.5, sel)
    _close(host(out.double()), want, tol)


def test_a_falling_prefix_computes_nothing():
    rng = np.random.default_rng(58)
    b = Batch(rng, [(2, 30), (3, 40), (2, 9)], 1, 64, 16, "bf16")
    _, qd = _queries(rng, 7, 4, 64)
    out = torch.full((7, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    for cu in ([0, 6, 3, 7], [-2, 2, 5, 7]):
        ws = dsa.attention_workspace(7, 3, 6, 4, 1, 64)
        dsa.paged_attention(qd, b.cache(dsa), dev(np.array(cu, np.int32)), b.dev("cu_k"), b.dev("table"), 6, 40, out=out, ws=ws)
        assert dsa.read_status(ws) == _abi.DSA_ERR_INVALID_ARG
        assert (out == 3).all()


def test_an_empty_batch_with_a_list():
    rng = np.random.default_rng(59)
    b = Batch(rng, [(0, 5), (0, 0)], 2, 64, 16, "mxfp8")
    empty = lambda shape, dt: torch.empty(shape, dtype=dt, device="cuda")
    out, lse = dsa.paged_attention(empty((0, 4, 64), torch.bfloat16), b.cache(dsa), b.dev("cu_q"), b.dev("cu_k"),
                                   b.dev("table"), 0, 5, topk_idx=empty((0, 32), torch.int32),
                                   topk_len=empty((0,), torch.int32), return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_captured_calls_that_share_a_workspace():
    """One workspace, sized for the larger call, in two graphs replayed in turn."""
    rng = np.random.default_rng(60)
    big, small = Batch(rng, [(3, 2000), (1, 700)], 2, 128, 64, "mxfp8"), Batch(rng, [(1, 4000)], 2, 128, 64, "mxfp8")
    ws = dsa.attention_workspace(4, 2, 3, 16, 2, 128)
    runs = []
    for b in (big, small):
        q, qd = _queries(rng, b.total_q, 16, 128)
        out = torch.zeros((b.total_q, 16, 128), dtype=torch.bfloat16, device="cuda")
        args = (qd, b.cache(dsa), b.dev("cu_q"), b.dev("cu_k"), b.dev("table"), max(t for t, _ in b.lens), 4000)
        dsa.paged_attention(*args, out=out, ws=ws)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            dsa.paged_attention(*args, out=out, ws=ws)
        runs.append((g, out, args, attention(b, q, 8, 128 ** -0.5)))
    for _ in range(3):
        for g, out, _, _ in runs:
            out.zero_()
            g.replay()
    torch.cuda.synchronize()
    for _, out, _, (want, _, tol, _) in runs:
        _close(host(out.double()), want, tol)


@pytest.mark.parametrize("group", [1, 4, 5])
@pytest.mark.parametrize("prec,D,page", [("bf16", 128, 16), ("mxfp8", 128, 32), ("fp8", 128, 8), ("mxfp8", 64, 32)])
def test_tiles_of_few_rows(prec, D, page, group):
    """A few tokens of few heads each: at most 16 rows to a tile, of several tokens."""
    rng = np.random.default_rng(61)
    b = Batch(rng, [(3, 700), (2, 129), (0, 5), (1, 1), (3, 3), (3, 257)], 2, D, page, prec)
    _run(b, rng, 2 * group, group)
    sel, lens = _selection(rng, b, 300, "wild")
    _run(b, rng, 2 * group, group, sel, lens)


@pytest.mark.parametrize("step", [0.05, -0.05, 0.4])
@pytest.mark.parametrize("group", [4, 16, 24])
def test_rising_and_falling_logits_of_few_rows(group, step):
    """Keys whose logits grow (or fall) along the sequence by 2 ** 0.5 .. 2 ** 5 in every one: the
    running maximum is raised over and over while products are in flight, within split ranges too."""
    rng = np.random.default_rng(62)
    b = Batch(rng, [(1, 1500), (1, 640), (1, 90)], 1, 128, 16, "bf16")
    for d, (_, s) in enumerate(b.lens):
        for pos in range(s):
            bits, _ = quantise(np.concatenate([[step * pos], 0.2 * rng.standard_normal(127)])[None], "bf16")
            b.pages["k"][b.table[d, pos // 16], 0, pos % 16] = bits
            b.rows["k"][b.cu_k[d] + pos, 0] = values(bits, None, "bf16")
    q, qd = _queries(rng, 3, group, 128)
    q[:, :, 0], qd[:, :, 0] = 8.0, 8.0
    for sel in (None, np.stack([np.concatenate([rng.permutation(s)[:80], np.full(max(0, 80 - s), -1)]) for _, s in b.lens]).astype(np.int32)):
        out, lse = dsa.paged_attention(qd, b.cache(dsa), b.dev("cu_q"), b.dev("cu_k"), b.dev("table"), 1, 1500, sm_scale=1.0,
                                       topk_idx=None if sel is None else dev(sel), return_lse=True)
        want, wl, tol, ltol = attention(b, q, group, 1.0, sel)
        _close(host(out.double()), want, tol)
        _close(host(lse.double()), wl, ltol)
