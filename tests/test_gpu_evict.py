"""A paged cache of bounded length: gathered attention weights, the choice of rows and their moving, against the
formulas in 64 bits (tests/evict_ref.py, whose bound of the FP32 sums is the tolerance) and together as they are used."""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_dsa_gb300 as dsa
from sparse_attention_indexer_dsa_gb300 import _abi
from tests import evict_ref as E
from tests.gpu_util import bf16_dev, dev, host
from tests.paged_ref import Batch, quantise, values

pytestmark = pytest.mark.gpu


def queries(rng, T, H, D, std=1.0):
    bits, _ = quantise(rng.standard_normal((T, H, D)) * std, "bf16")
    return values(bits, None, "bf16"), bf16_dev(bits)


def true_lse(b, q, group, scale):
    out = np.full(q.shape[:2], -np.inf)
    for d, (t, s) in enumerate(b.lens):
        for i in range(t):
            for hh in range(q.shape[1]):
                lg = scale * (b.rows["k"][b.cu_k[d]:b.cu_k[d] + s - t + i + 1, hh // group] @ q[b.cu_q[d] + i, hh])
                out[b.cu_q[d] + i, hh] = lg.max() + np.log(np.exp(lg - lg.max()).sum())
    return out.astype(np.float32)


def weigh(b, c, w, qd, lse, scale, max_q=None, max_k=None, ws=None, status=0):
    max_q = max(t for t, _ in b.lens) if max_q is None else max_q
    max_k = max(s for _, s in b.lens) if max_k is None else max_k
    if ws is None:
        ws = dsa.weigh_workspace(qd.shape[0], len(b.lens), max_q, qd.shape[1], b.n_kv, b.D)
    dsa.cache_weigh(c, w, qd, lse, b.dev("cu_q"), b.dev("cu_k"), b.dev("table"), max_q, max_k, sm_scale=scale, ws=ws)
    assert dsa.read_status(ws) == status
    return w


def close(got, want, tol, what=""):
    got = host(got.double())
    over = np.abs(got - want) - tol
    assert np.isfinite(got).all() and (over <= 0).all(), (what, np.unravel_index(over.argmax(), over.shape), float(over.max()))


def check_weigh(b, rng, group, std=2.0, scale=None, pad_q=0):
    scale = b.D ** -0.5 if scale is None else scale
    q, qd = queries(rng, b.total_q, b.n_kv * group, b.D, std)
    lse = true_lse(b, q, group, scale)
    w = E.random_weights(rng, b)
    got = weigh(b, b.cache(dsa), dev(w), qd, dev(lse), scale)
    want, tol = E.weigh(b, q, lse.astype(np.float64), w, group, scale)
    close(got, want, tol)
    return got


LENS = {
    "one": [(1, 1)],
    "steps": [(1, 1), (1, 31), (1, 32), (0, 9), (1, 33), (1, 600)],
    "chunk": [(33, 33), (0, 0), (17, 300), (1, 260), (130, 131)],
    "prompt": [(257, 257)],
}


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("kv,group", [(1, 1), (2, 8), (1, 64), (3, 5)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prec", ["bf16", "mxfp8", "fp8"])
def test_weigh(lens, kv, group, D, prec):
    rng = np.random.default_rng([sorted(LENS).index(lens), kv, group, D, len(prec)])
    b = Batch(rng, LENS[lens], kv, D, 16, prec)
    check_weigh(b, rng, group)


@pytest.mark.parametrize("page", [8, 64, 1024])
@pytest.mark.parametrize("lens", [[(1, 700), (3, 64), (1, 1025)], [(200, 900)], [(70, 70), (1, 2000), (0, 40), (40, 400)]])
def test_weigh_pages(page, lens):
    rng = np.random.default_rng([page, len(lens)])
    b = Batch(rng, lens, 2, 128, page, "mxfp8", values_too=False, pad_q=5)
    check_weigh(b, rng, 4)


@pytest.mark.parametrize("prec", ["bf16", "mxfp8", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 128])
def test_weigh_rows_of_a_page_together(prec, D, page):
    """Pages of less than a step's rows and of more, last rows anywhere in a page whose other slots hold NaN."""
    rng = np.random.default_rng([len(prec), D, page])
    for group, lens in ((8, [(1, 1), (1, 31), (1, 33), (1, 130), (1, 511)]), (5, [(3, 65), (1, 200), (4, 4)])):
        check_weigh(Batch(rng, lens, 2, D, page, prec), rng, group)


@pytest.mark.parametrize("group,T", [(128, 9), (1, 300), (7, 41), (2, 520)])
def test_weigh_groups(group, T):
    rng = np.random.default_rng([group, T])
    b = Batch(rng, [(T, T + 77), (1, 300)], 1, 64, 32, "bf16", values_too=False)
    check_weigh(b, rng, group)


@pytest.mark.parametrize("prec,D,page", [("bf16", 128, 64), ("mxfp8", 128, 16), ("fp8", 64, 8)])
@pytest.mark.parametrize("kv,group,lens", [(1, 8, [(640, 700), (0, 5), (90, 95)]), (2, 5, [(1, 9), (900, 900)]),
                                           (1, 128, [(40, 3000)])])
def test_weigh_divided(kv, group, lens, prec, D, page):
    """Few units of keys with many query rows: their tokens are divided and the parts joined."""
    rng = np.random.default_rng([kv, group, D])
    check_weigh(Batch(rng, lens, kv, D, page, prec, values_too=False, pad_q=3), rng, group)


def test_weigh_other_rows_of_a_tile():
    """A tile's last rows may be another sequence's tokens, or padding, that hold anything."""
    rng = np.random.default_rng(37)
    b = Batch(rng, [(70, 150), (20, 20), (65, 65)], 1, 64, 16, "bf16", values_too=False, pad_q=40)
    q, qd = queries(rng, b.total_q, 4, 64)
    lse = true_lse(b, q, 4, 0.1)
    lse[155:] = np.nan
    qd[155:] = float("nan")
    qd[70:90] = float("nan")
    w = E.random_weights(rng, b)
    got = weigh(b, b.cache(dsa), dev(w), qd, dev(lse), 0.1)
    want, tol = E.weigh(b, q, lse.astype(np.float64), w, 4, 0.1)
    page, slot = E.rows_of(b, 1)
    mine = np.ones(w.shape, bool)
    mine[page, :, slot] = False
    assert host(got)[page, :, slot].size and np.isnan(host(got)[page, :, slot]).all()
    close(got[torch.from_numpy(mine).cuda()], want[mine], tol[mine])


def test_weigh_a_wait_that_runs_out():
    rng = np.random.default_rng(38)
    b = Batch(rng, [(70, 150)], 1, 128, 16, "mxfp8", values_too=False)
    q, qd = queries(rng, b.total_q, 4, 128)
    lse = dev(true_lse(b, q, 4, 0.1))
    w = E.random_weights(rng, b)
    lib = _abi.load()
    try:
        lib.dsa_idx_test_set_timeout_ns(50_000_000)
        lib.dsa_idx_test_set_fault_inject(1)
        weigh(b, b.cache(dsa), dev(w), qd, lse, 0.1, status=_abi.DSA_ERR_TIMEOUT)
    finally:
        lib.dsa_idx_test_set_fault_inject(0)
        lib.dsa_idx_test_set_timeout_ns(2_000_000_000)
    got = weigh(b, b.cache(dsa), dev(w), qd, lse, 0.1)
    close(got, *E.weigh(b, q, host(lse).astype(np.float64), w, 4, 0.1))


def test_weigh_far_scales():
    """8-bit rows whose scales are far from one: the widened values span BF16's range."""
    rng = np.random.default_rng(31)
    for prec in ("mxfp8", "fp8"):
        b = Batch(rng, [(1, 90), (40, 70)], 1, 128, 16, prec, std=3e5)
        check_weigh(b, rng, 2, std=1e-6)


@pytest.mark.parametrize("prec", ["bf16", "mxfp8", "fp8"])
@pytest.mark.parametrize("T", [1, 5])
def test_weigh_queries_of_wide_range(prec, T):
    """Query elements that span up to 2^100, far from one altogether (the scale brings the logits back)."""
    rng = np.random.default_rng([39, T])
    b = Batch(rng, [(T, 77)], 1, 128, 16, prec)
    for spread, shift in ((1, 0), (20, 80), (31, 0), (31, -100), (33, 0), (60, 0), (100, 80), (100, -100)):
        x = rng.standard_normal((T, 4, 128)) * 2.0 ** (shift + rng.uniform(-spread, 0, (T, 4, 128)))
        x[:, 3, ::2] = 0
        bits, _ = quantise(x, "bf16")
        q, qd = values(bits, None, "bf16"), bf16_dev(bits)
        scale = float(np.float32(0.09 * 2.0 ** -shift))
        lse = true_lse(b, q, 4, scale)
        w = E.random_weights(rng, b)
        got = weigh(b, b.cache(dsa), dev(w), qd, dev(lse), scale)
        close(got, *E.weigh(b, q, lse.astype(np.float64), w, 4, scale), (spread, shift))


def test_weigh_lost_bits():
    """One huge query element against zeros of every key: the others' products must not suffer."""
    rng = np.random.default_rng(40)
    for prec in ("mxfp8", "fp8"):
        b = Batch(rng, [(1, 64)], 1, 64, 16, prec)
        for nm in ("k",):
            b.rows[nm][..., 7] = 0
            b.pages[nm][..., 7] = 0
        x = rng.standard_normal((1, 2, 64))
        x[..., 7] = 1e12
        bits, _ = quantise(x, "bf16")
        q, qd = values(bits, None, "bf16"), bf16_dev(bits)
        lse = true_lse(b, q, 2, 0.5)
        w = np.zeros((b.num_pages, 1, 16), np.float32)
        got = weigh(b, b.cache(dsa), dev(w), qd, dev(lse), 0.5)
        close(got, *E.weigh(b, q, lse.astype(np.float64), w, 2, 0.5))


def test_weigh_strange_lse():
    """Rows that saw nothing add nothing; scale 0 weighs every row alike."""
    rng = np.random.default_rng(32)
    b = Batch(rng, [(2, 40), (80, 100)], 2, 64, 16, "bf16", values_too=False)
    q, qd = queries(rng, b.total_q, 4, 64)
    lse = true_lse(b, q, 2, 0.125)
    lse[1] = -np.inf
    lse[30:40, 1] = -np.inf
    w = E.random_weights(rng, b)
    got = weigh(b, b.cache(dsa), dev(w), qd, dev(lse), 0.125)
    close(got, *E.weigh(b, q, lse.astype(np.float64), w, 2, 0.125))
    lse = true_lse(b, q, 2, 0.0)
    got = weigh(b, b.cache(dsa), dev(w), qd, dev(lse), 0.0)
    close(got, *E.weigh(b, q, lse.astype(np.float64), w, 2, 0.0))


def test_weigh_leaves_other_slots_and_repeats():
    rng = np.random.default_rng(33)
    b = Batch(rng, [(1, 50), (0, 33), (90, 131)], 2, 128, 16, "mxfp8", pad_q=7)
    q, qd = queries(rng, b.total_q, 16, 128)
    lse = true_lse(b, q, 8, 0.1)
    w = E.random_weights(rng, b)
    used = np.zeros(w.shape, bool)
    for d in (0, 2):
        used[E.rows_of(b, d)[0], :, E.rows_of(b, d)[1]] = True
    w[~used] = np.nan
    got = [host(weigh(b, b.cache(dsa), dev(w), qd, dev(lse), 0.1)) for _ in range(3)]
    assert np.isnan(got[0][~used]).all() and np.isfinite(got[0][used]).all()
    assert all(np.array_equal(got[0], g, equal_nan=True) for g in got[1:])
    # a token adds its number of heads in all
    added = got[0].astype(np.float64)
    page, slot = E.rows_of(b, 0)
    old = w[page, :, slot].astype(np.float64)
    old[49:] = 0
    assert np.allclose((added[page, :, slot] - old).sum(0), 8, atol=1e-4)


def test_weigh_with_strided_queries_and_the_attentions_lse():
    rng = np.random.default_rng(34)
    b = Batch(rng, [(1, 500), (60, 333)], 2, 128, 32, "fp8")
    wide = torch.randn(b.total_q, 8 + 3, 128, device="cuda").bfloat16()
    qd = wide[:, :8]
    c = b.cache(dsa)
    _, lse = dsa.paged_attention(qd, c, b.dev("cu_q"), b.dev("cu_k"), b.dev("table"), 60, 500, return_lse=True)
    w = dsa.paged_weights(c)
    weigh(b, c, w, qd, lse, None)
    want, tol = E.weigh(b, host(qd.double()), host(lse).astype(np.float64), np.zeros(w.shape, np.float32), 4, 128 ** -0.5)
    close(w, want, tol)


def test_weigh_reports():
    rng = np.random.default_rng(35)
    b = Batch(rng, [(1, 40), (3, 50)], 1, 64, 16, "bf16", values_too=False)
    q, qd = queries(rng, b.total_q, 2, 64)
    lse = dev(true_lse(b, q, 2, 0.1))
    w = E.random_weights(rng, b)
    c = b.cache(dsa)
    want, tol = E.weigh(b, q, host(lse).astype(np.float64), w, 2, 0.1)
    # a page that does not exist: its rows are left out
    t = b.table[1, 1]
    b.table[1, 1] = b.num_pages
    got = weigh(b, c, dev(w), qd, lse, 0.1, status=1)
    other = np.ones(w.shape, bool)
    other[t] = False
    assert np.array_equal(host(got)[t], w[t])
    close(got, np.where(other, want, w), tol)
    b.table[1, 1] = t
    # a bound that is too small: that sequence is not computed
    got = host(weigh(b, c, dev(w), qd, lse, 0.1, max_k=45, status=1))
    page, slot = E.rows_of(b, 1)
    assert np.array_equal(got[page, :, slot], w[page, :, slot])
    # a prefix that falls: nothing is
    for name, bad in (("cu_q", [0, 3, 1]), ("cu_k", [0, 50, 40])):
        keep = getattr(b, name)
        setattr(b, name, np.array(bad, np.int32))
        assert np.array_equal(host(weigh(b, c, dev(w), qd, lse, 0.1, status=1)), w)
        setattr(b, name, keep)
    # more new tokens than rows, more tokens than there are
    for name, bad in (("cu_k", [0, 40, 42]), ("cu_q", [0, 1, 9])):
        keep = getattr(b, name)
        setattr(b, name, np.array(bad, np.int32))
        got = host(weigh(b, c, dev(w), qd, lse, 0.1, status=1))
        assert np.array_equal(got[page, :, slot], w[page, :, slot])
        setattr(b, name, keep)


def test_weigh_empty():
    rng = np.random.default_rng(36)
    b = Batch(rng, [(0, 10), (0, 0)], 1, 64, 8, "bf16", values_too=False)
    w = E.random_weights(rng, b)
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    got = weigh(b, b.cache(dsa), dev(w), q, torch.empty(0, 4, device="cuda"), 1.0)
    assert np.array_equal(host(got), w)


# ---------------------------------------------------------------- choice

def check_select(b, w, budget, sinks, recent, shared, max_k=None):
    ws = dsa.cache_workspace()
    max_k = max(s for _, s in b.lens) if max_k is None else max_k
    kept, n = dsa.evict_select(dev(w), b.dev("cu_k"), b.dev("table"), budget, max_k, sinks=sinks, recent=recent,
                               shared=shared, ws=ws)
    assert dsa.read_status(ws) == 0
    want, wn = E.select(b, w, budget, sinks, recent, shared)
    assert np.array_equal(host(n), wn) and np.array_equal(host(kept), want)


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (64, 4, 16), (100, 0, 100), (127, 100, 27), (1500, 3, 0)])
def test_select(ties, shared, budget, sinks, recent):
    rng = np.random.default_rng([ties, shared, budget, sinks, recent])
    b = Batch(rng, [(0, s) for s in (0, 1, 63, 64, 65, 127, 1023, 1025, 2100)], 3, 64, 16, "bf16", values_too=False)
    check_select(b, E.random_weights(rng, b, ties), budget, sinks, recent, shared)


@pytest.mark.parametrize("page", [8, 1024])
def test_select_long(page):
    """More rows than shared memory holds."""
    rng = np.random.default_rng(page)
    b = Batch(rng, [(0, 70001), (0, 300)], 1, 64, page, "fp8", values_too=False)
    w = E.random_weights(rng, b)
    for budget in (200, 4096, 70000):
        check_select(b, w, budget, 4, 64, False)
    check_select(b, E.random_weights(rng, b, True), 5000, 0, 0, True)


@pytest.mark.parametrize("lens", [[20000], [5000, 41, 9000], [3000] * 70, [400000]])
def test_select_clusters(lens):
    """From one block to a head to eight, and more rows than eight hold."""
    rng = np.random.default_rng(len(lens))
    b = Batch(rng, [(0, s) for s in lens], 1, 64, 1024, "fp8", values_too=False)
    w = E.random_weights(rng, b, True)
    for budget in (33, 2500):
        check_select(b, w, budget, 3, 10, False)


def test_select_strange_weights():
    rng = np.random.default_rng(41)
    b = Batch(rng, [(0, 400), (0, 90)], 2, 64, 8, "bf16", values_too=False)
    w = E.random_weights(rng, b)
    flat = w.reshape(-1)
    for v in (np.nan, -np.nan, np.inf, -np.inf, -0.0, 0.0, 1e-45, -1e-45, np.finfo(np.float32).max, np.finfo(np.float32).min):
        flat[rng.random(flat.size) < 0.06] = v
    for budget in (1, 5, 30, 80, 380):
        check_select(b, w, budget, 1 if budget > 1 else 0, 2 if budget > 4 else 0, False)
    for v in (0.0, np.nan, np.inf, -1.0):      # all alike: the first ones
        check_select(b, np.full_like(w, v), 37, 2, 5, False)


def test_select_wide_table_and_outputs():
    rng = np.random.default_rng(42)
    b = Batch(rng, [(0, 50), (0, 20)], 2, 64, 8, "bf16", values_too=False)
    w = E.random_weights(rng, b)
    check_select(b, w, 10, 1, 1, False, max_k=1 << 20)       # a bound far above the lengths
    out = (torch.full((2, 2, 10), 9, dtype=torch.int32, device="cuda"), torch.full((2,), 9, dtype=torch.int32, device="cuda"))
    got = dsa.evict_select(dev(w), b.dev("cu_k"), b.dev("table"), 10, 50, out=out)
    assert got[0] is out[0] and np.array_equal(host(out[0]), E.select(b, w, 10, 0, 0, False)[0])


def test_select_reports():
    rng = np.random.default_rng(43)
    b = Batch(rng, [(0, 50), (0, 40)], 1, 64, 8, "bf16", values_too=False)
    w = E.random_weights(rng, b)
    want, _ = E.select(b, w, 10, 0, 0, False)
    ws = dsa.cache_workspace()

    def run(max_k=50):
        kept, n = dsa.evict_select(dev(w), b.dev("cu_k"), b.dev("table"), 10, max_k, ws=ws)
        assert dsa.read_status(ws) == 1
        return host(kept), host(n)

    kept, n = run(max_k=45)
    assert (kept[0] == -1).all() and np.array_equal(kept[1], want[1]) and list(n) == [0, 10]
    keep, b.cu_k = b.cu_k, np.array([0, 50, 45], np.int32)
    kept, n = run()
    assert (kept[1] == -1).all() and np.array_equal(kept[0], want[0]) and list(n) == [10, 0]
    b.cu_k = keep
    b.table[0, 2] = -7
    kept, n = run()
    assert not ((kept[0] >= 16) & (kept[0] < 24)).any() and list(n) == [10, 10]


# ---------------------------------------------------------------- moving

def tensors_of(b, w=None):
    t = {}
    for nm in b.names:
        t[nm] = b.pages[nm]
        if b.scales[nm] is not None:
            t[nm + "_scale"] = b.scales[nm]
    if w is not None:
        t["weights"] = w
    return t


def as_bits(t):
    return host(t.view(torch.int16)).view(np.uint16) if t.dtype == torch.bfloat16 else host(t)


def check_compact(b, rng, kept, kept_len, w=None, status=0):
    c, ws = b.cache(dsa), dsa.cache_workspace()
    wd = None if w is None else dev(w)
    dsa.cache_compact(c, dev(kept), dev(kept_len), b.dev("table"), weights=wd, ws=ws)
    assert dsa.read_status(ws) == status
    want = E.compact(b, tensors_of(b, w), kept, kept_len)
    got = {"k": c.k, "k_scale": c.k_scale, "v": c.v, "v_scale": c.v_scale, "weights": wd}
    for name, x in want.items():
        assert np.array_equal(as_bits(got[name]), x), name


def some_rows(rng, b, heads, width, part=0.5):
    kept = np.full((len(b.lens), heads, width), -1, np.int32)
    n = np.array([min(width, int(round(s * part))) for _, s in b.lens], np.int32)
    for d, (_, s) in enumerate(b.lens):
        for h in range(heads):
            kept[d, h, :n[d]] = np.sort(rng.choice(s, n[d], replace=False))
    return kept, n


@pytest.mark.parametrize("prec", ["bf16", "mxfp8", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv,heads", [(1, 1), (3, 3), (3, 1)])
@pytest.mark.parametrize("part", [0.1, 0.9, 1.0])
def test_compact(prec, D, kv, heads, part):
    rng = np.random.default_rng([len(prec), D, kv, heads, int(10 * part)])
    b = Batch(rng, [(0, 0), (0, 1), (0, 17), (0, 700), (0, 2500)], kv, D, 16, prec)
    kept, n = some_rows(rng, b, heads, 2600, part)
    check_compact(b, rng, kept, n, E.random_weights(rng, b))


@pytest.mark.parametrize("page", [8, 1024])
@pytest.mark.parametrize("prec,values_too,weights", [("bf16", False, False), ("mxfp8", False, True), ("fp8", True, False)])
def test_compact_parts(page, prec, values_too, weights):
    rng = np.random.default_rng([page, len(prec)])
    b = Batch(rng, [(0, 9000), (0, 1300)], 1, 128, page, prec, values_too=values_too)
    kept, n = some_rows(rng, b, 1, 5000, 0.8)
    check_compact(b, rng, kept, n, E.random_weights(rng, b) if weights else None)


def test_compact_many_sequences():
    rng = np.random.default_rng(51)
    b = Batch(rng, [(0, int(s)) for s in rng.integers(0, 90, 300)], 4, 64, 8, "mxfp8")
    kept, n = some_rows(rng, b, 4, 40)
    check_compact(b, rng, kept, n, E.random_weights(rng, b))


def test_compact_again_and_again():
    """Many chunks by blocks of threads that are not in step, the same bits every time."""
    rng = np.random.default_rng(54)
    for lens, kv, D, prec in (([30000], 2, 128, "bf16"), ([9000] * 3, 8, 128, "mxfp8"), ([2000] * 60, 4, 64, "fp8")):
        b = Batch(rng, [(0, s) for s in lens], 1, D, 64, prec)
        kept, n = some_rows(rng, b, 1, max(lens), 0.7)
        base = b.cache(dsa)
        full = [None if t is None else t.expand(-1, kv, -1, -1) for t in (base.k, base.k_scale, base.v, base.v_scale)]
        w = torch.arange(b.num_pages * 64, device="cuda").float().view(-1, 1, 64).expand(-1, kv, -1)
        want = E.compact(b, tensors_of(b, host(w[:, :1].contiguous())), kept, n)
        for _ in range(6):
            c = dsa.PagedCache(*[None if t is None else t.contiguous() for t in full], prec)
            wd = w.contiguous()
            dsa.cache_compact(c, dev(kept), dev(n), b.dev("table"), weights=wd)
            for name, t in (("k", c.k), ("k_scale", c.k_scale), ("v", c.v), ("v_scale", c.v_scale), ("weights", wd)):
                if t is not None:
                    first = as_bits(t[:, :1].contiguous())
                    assert np.array_equal(first, want[name]), (name, lens)
                    assert torch.equal(t.view(torch.uint8) if t.dtype == torch.bfloat16 else t,
                                       (t[:, :1].view(torch.uint8) if t.dtype == torch.bfloat16 else t[:, :1]).expand_as(
                                           t.view(torch.uint8) if t.dtype == torch.bfloat16 else t))


@pytest.mark.parametrize("sequences", [10, 14, 18, 22, 28, 36, 50])
def test_compact_sequences_in_between(sequences):
    """Numbers of sequences that give a head three to eight blocks, not powers of two alone; ragged last chunks."""
    rng = np.random.default_rng([55, sequences])
    b = Batch(rng, [(0, int(s)) for s in rng.integers(300, 1500, sequences)], 2, 64, 16, "mxfp8")
    kept, n = some_rows(rng, b, 2, 1400, 0.9)
    check_compact(b, rng, kept, n, E.random_weights(rng, b))


def test_compact_shifts_by_one():
    """Every row but one stays: each chunk reads what the one before it has to leave alone."""
    rng = np.random.default_rng(52)
    for gone in (0, 1, 255, 256, 2999):
        b = Batch(rng, [(0, 3000)], 2, 128, 64, "mxfp8")
        kept = np.delete(np.arange(3000, dtype=np.int32), gone)[None, None]
        check_compact(b, rng, kept, np.array([2999], np.int32), E.random_weights(rng, b))


def test_compact_reports():
    rng = np.random.default_rng(53)
    b = Batch(rng, [(0, 100), (0, 80)], 2, 64, 8, "fp8")
    kept, n = some_rows(rng, b, 2, 50)
    good = E.compact(b, tensors_of(b), kept, n)
    page1 = E.rows_of(b, 1)
    for bad in ("falls", "twice", "behind", "before", "length", "width"):
        k, m = kept.copy(), n.copy()
        if bad == "falls":
            k[0, 0, 10], k[0, 0, 20] = k[0, 0, 20], k[0, 0, 10]
        elif bad == "twice":
            k[0, 0, 11] = k[0, 0, 10]
        elif bad == "behind":
            k[0, 0, int(m[0]) - 1] = 1 << 29
        elif bad == "before":
            k[0, 0, 0] = -5
        elif bad == "length":
            m[0] = -1
        else:
            m[0] = 51
        c, ws = b.cache(dsa), dsa.cache_workspace()
        dsa.cache_compact(c, dev(k), dev(m), b.dev("table"), ws=ws)
        assert dsa.read_status(ws) == 1, bad
        for nm, t in (("k", c.k), ("v", c.v), ("v_scale", c.v_scale)):
            got, start = as_bits(t), tensors_of(b)[nm]
            assert np.array_equal(got[page1[0], :, page1[1]], good[nm][page1[0], :, page1[1]]), bad
            outside = np.ones(start.shape[0], bool)
            outside[b.table[0, :13]] = outside[b.table[1, :10]] = False
            assert np.array_equal(got[outside], start[outside]), bad


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
@pytest.mark.parametrize("shared", [False, True])
def test_a_bounded_cache_step_by_step(prec, shared):
    """A prompt in chunks, then single tokens, through norm_rope, cache_write, paged_attention, cache_weigh and, over
    the budget, evict_select and cache_compact, with an index cache that keeps the same rows where the choice is shared:
    the rows that a cache holds are those that a plain run of the choices keeps, bit for bit."""
    torch.manual_seed(7)
    kv, group, D, page, budget, B = 2, 4, 128, 16, 96, 3
    pages = B * 12
    table = torch.randperm(pages, device="cuda").to(torch.int32).view(B, 12)
    cache = dsa.paged_cache(pages, page, kv, D, prec)
    index = dsa.paged_cache(pages, page, 1, D, "bf16", values=False)
    weights = dsa.paged_weights(cache)
    lens = [0] * B
    held = [[[] for _ in range(kv)] for _ in range(B)]        # positions of the rows that each head holds
    qw, kw = torch.rand(D, device="cuda") + 0.5, torch.rand(D, device="cuda") + 0.5
    seen = [0] * B
    keys = [torch.empty(0, kv, D, device="cuda") for _ in range(B)]    # of every position, as written
    for step in range(12):
        new = [70, 33, 1] if step == 0 else ([40, 50, 64] if step == 1 else [1, 1, 1])
        T = sum(new)
        cu_q = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
        for d in range(B):
            lens[d] += new[d]
        cu_k = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        pos = torch.cat([torch.arange(seen[d], seen[d] + new[d]) for d in range(B)]).to(torch.int32).cuda()
        x = torch.randn(T, (group + 2) * kv, D, device="cuda").bfloat16()
        q, k = dsa.norm_rope(x[:, :group * kv], x[:, group * kv:group * kv + kv], pos, qw, kw)
        dsa.cache_write(cache, k, x[:, group * kv + kv:], cu_q, cu_k, table)
        dsa.cache_write(index, k[:, :1], None, cu_q, cu_k, table)
        max_q, max_k = max(new), max(lens)
        out, lse = dsa.paged_attention(q, cache, cu_q, cu_k, table, max_q, max_k, return_lse=True)
        dsa.cache_weigh(cache, weights, q, lse, cu_q, cu_k, table, max_q, max_k)
        at = 0
        for d in range(B):
            keys[d] = torch.cat([keys[d], k[at:at + new[d]].float()])
            at += new[d]
            for h in range(kv):
                held[d][h] += range(seen[d], seen[d] + new[d])
            seen[d] += new[d]
        before = host(weights)
        kept, n = dsa.evict_select(weights, cu_k, table, budget, max_k, sinks=2, recent=8, shared=shared)
        dsa.cache_compact(cache, kept, n, table, weights=weights)
        if shared:
            dsa.cache_compact(index, kept, n, table)
        rows, m = host(kept), host(n)
        for d in range(B):
            for h in range(kv):
                mine = rows[d, 0 if shared else h, :m[d]]
                w = np.concatenate([before[p] for p in host(table)[d]], axis=1)[h] if not shared else None
                if not shared and lens[d] > budget:      # the lightest that stays is no lighter than the heaviest that goes
                    gone = np.setdiff1d(np.arange(2, lens[d] - 8), mine)
                    free = mine[(mine >= 2) & (mine < lens[d] - 8)]
                    assert w[free].min() >= w[gone].max()
                held[d][h] = [held[d][h][i] for i in mine]
            lens[d] = int(m[d])
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        got, _, _, _ = dsa.cache_read(cache, cu, table, sum(lens), out_prec="bf16")
        idx, _, _, _ = dsa.cache_read(index, cu, table, sum(lens))
        at = 0
        for d in range(B):
            for h in range(kv):
                want = keys[d][held[d][h], h]
                have = got[at:at + lens[d], h].float()
                if prec == "bf16":
                    assert torch.equal(have, want)
                else:       # half a step of E4M3 relative, or of its smallest under the block's scale
                    amax = want.view(-1, D // 32, 32).abs().amax(-1, keepdim=True).expand(-1, -1, 32).reshape(want.shape)
                    assert ((have - want).abs() <= torch.maximum(want.abs() * 2.0 ** -4, amax * 2.0 ** -16)).all()
            if shared:
                assert torch.equal(idx[at:at + lens[d], 0].float(), keys[d][held[d][0], 0])
            at += lens[d]
    assert lens == [96, 93, 75]


def test_streams_and_graphs():
    rng = np.random.default_rng(61)
    b = Batch(rng, [(1, 300), (70, 200)], 2, 64, 16, "mxfp8")
    q, qd = queries(rng, b.total_q, 8, 64)
    lse = dev(true_lse(b, q, 4, 0.1))
    w0 = E.random_weights(rng, b)
    args = [b.dev(n) for n in ("cu_q", "cu_k", "table")]
    ws = dsa.weigh_workspace(b.total_q, 2, 70, 8, 2, 64)
    cw = dsa.cache_workspace()

    def run(c, w):
        dsa.cache_weigh(c, w, qd, lse, *args, 70, 300, sm_scale=0.1, ws=ws)
        kept, n = dsa.evict_select(w, args[1], args[2], 128, 300, sinks=1, recent=9, ws=cw)
        dsa.cache_compact(c, kept, n, args[2], weights=w, ws=cw)
        return kept, n

    c1, w1 = b.cache(dsa), dev(w0)
    kept, n = run(c1, w1)
    c2, w2 = b.cache(dsa), dev(w0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = run(c2, w2)
        w2.copy_(dev(w0))          # nothing ran at capture
        graph.replay()
    s.synchronize()
    assert torch.equal(got[0], kept) and torch.equal(got[1], n) and torch.equal(w1, w2)
    assert torch.equal(c1.k, c2.k) and torch.equal(c1.v, c2.v) and torch.equal(c1.k_scale, c2.k_scale)


def test_two_calls_at_once():
    """Two streams with caches and workspaces of their own, steps and tiles in one call."""
    rng = np.random.default_rng(62)
    b = Batch(rng, [(1, 900), (300, 2000), (40, 700)], 2, 128, 16, "mxfp8")
    q, qd = queries(rng, b.total_q, 16, 128)
    lse = dev(true_lse(b, q, 8, 0.1))
    w0 = E.random_weights(rng, b)
    args = [b.dev(n) for n in ("cu_q", "cu_k", "table")]
    streams = [torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()]
    state = [(b.cache(dsa), dev(w0), dsa.weigh_workspace(b.total_q, 3, 300, 16, 2, 128), dsa.cache_workspace()) for _ in streams]
    torch.cuda.synchronize()
    got = []
    for (c, w, ws, cw), s in zip(state, streams):
        with torch.cuda.stream(s):
            for _ in range(3):
                dsa.cache_weigh(c, w, qd, lse, *args, 300, 2000, sm_scale=0.1, ws=ws)
            got.append(dsa.evict_select(w, args[1], args[2], 500, 2000, sinks=2, recent=30, ws=cw))
            dsa.cache_compact(c, *got[-1], args[2], weights=w, ws=cw)
        if s is streams[0]:
            torch.cuda.synchronize()      # the first alone, the others beside one another
    torch.cuda.synchronize()
    for i in (1, 2):
        assert torch.equal(got[i][0], got[0][0]) and torch.equal(got[i][1], got[0][1])
        assert torch.equal(state[i][1], state[0][1]) and all(
            torch.equal(getattr(state[i][0], n), getattr(state[0][0], n)) for n in ("k", "v", "k_scale", "v_scale"))


@pytest.mark.parametrize("prec,pages", [("bf16", 150000), ("mxfp8", 300000)])
def test_rows_behind_four_gigabytes(prec, pages):
    """The same sequences at the end of a cache whose keys are more than 2^32 bytes: the same bits."""
    rng = np.random.default_rng(63)
    b = Batch(rng, [(1, 400), (90, 700)], 2, 128, 64, prec)
    q, qd = queries(rng, b.total_q, 16, 128)
    lse = dev(true_lse(b, q, 8, 0.1))
    w0 = dev(E.random_weights(rng, b))
    cu_q, cu_k, table = (b.dev(n) for n in ("cu_q", "cu_k", "table"))

    def run(c, w, table):
        dsa.cache_weigh(c, w, qd, lse, cu_q, cu_k, table, 90, 700, sm_scale=0.1)
        kept = dsa.evict_select(w, cu_k, table, 150, 700, sinks=1, recent=20)
        dsa.cache_compact(c, *kept, table, weights=w)
        return kept

    small, w = b.cache(dsa), w0.clone()
    n = small.k.shape[0]
    far = dsa.paged_cache(pages, 64, 2, 128, prec)
    fw = dsa.paged_weights(far)
    names = [x for x in ("k", "v", "k_scale", "v_scale") if getattr(small, x) is not None]
    for x in names:
        getattr(far, x)[-n:] = getattr(small, x)
    assert far.k[:-n].numel() * far.k.element_size() > 2 ** 32
    fw[-n:] = w
    want, got = run(small, w, table), run(far, fw, torch.where(table >= 0, table + (pages - n), table))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(fw[-n:], w)
    assert not fw[:-n].any()
    for x in names:
        a, e = getattr(far, x)[-n:], getattr(small, x)
        assert torch.equal(a.view(torch.uint8), e.view(torch.uint8)), x   # (unused slots hold NaN)


# ---------------------------------------------------------------- parts of a batch

def part_of(b, lo, hi):
    """Sequences lo .. hi - 1 as parts of the batch's prefixes and table: the prefixes begin where the part does."""
    return b.dev("cu_q")[lo:hi + 1], b.dev("cu_k")[lo:hi + 1], b.dev("table")[lo:hi]


@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
@pytest.mark.parametrize("lens", [[(1, 1000), (1, 100), (1, 200)], [(2, 37), (1, 40), (3, 333), (0, 12), (1, 5)],
                                  [(1, 600), (60, 300), (1, 90), (130, 131)]])
def test_weigh_parts_of_a_batch(lens, prec):
    """Every part by itself: its sequences' weights, and no bit of the others'."""
    rng = np.random.default_rng([71, len(lens), len(prec)])
    b = Batch(rng, lens, 2, 128, 16, prec, values_too=False)
    q, qd = queries(rng, b.total_q, 16, 128)
    lse = true_lse(b, q, 8, 0.1)
    w = E.random_weights(rng, b)
    want, tol = E.weigh(b, q, lse.astype(np.float64), w, 8, 0.1)
    c, ws = b.cache(dsa), dsa.weigh_workspace(b.total_q, len(lens), max(t for t, _ in lens), 16, 2, 128)
    for lo in range(len(lens)):
        for hi in (lo + 1, len(lens)):
            got = dev(w)
            cq, ck, table = part_of(b, lo, hi)
            dsa.cache_weigh(c, got, qd, dev(lse), cq, ck, table, max(t for t, _ in lens), max(s for _, s in lens), sm_scale=0.1, ws=ws)
            assert dsa.read_status(ws) == 0
            mine = np.zeros(w.shape, bool)
            for d in range(lo, hi):
                page, slot = E.rows_of(b, d)
                mine[page, :, slot] = True
            assert np.array_equal(host(got)[~mine], w[~mine]), (lo, hi)
            close(got[torch.from_numpy(mine).cuda()], want[mine], tol[mine], (lo, hi))


def test_select_parts_of_a_batch():
    rng = np.random.default_rng(72)
    b = Batch(rng, [(0, 1000), (0, 100), (0, 333)], 2, 64, 16, "bf16", values_too=False)
    w = E.random_weights(rng, b)
    want, n = E.select(b, w, 64, 2, 9, False)
    for lo, hi in ((1, 3), (2, 3), (1, 2)):
        _, ck, table = part_of(b, lo, hi)
        kept, got = dsa.evict_select(dev(w), ck, table, 64, 1000, sinks=2, recent=9)
        assert np.array_equal(host(kept), want[lo:hi]) and np.array_equal(host(got), n[lo:hi])


# ---------------------------------------------------------------- the scale

@pytest.mark.parametrize("T", [1, 40])      # a step, a chunk
@pytest.mark.parametrize("D", [64, 128])
def test_weigh_takes_the_scale_as_given(D, T):
    """One product to a logit, 2^14 and exact, under a scale whose product with log2(e) is 1 in FP32: a weight is
    2^(2^14 - B) with B = lse log2(e) rounded to FP32, as near as its own arithmetic is (two roundings of at most 2^-24 of an
    exponent below 2, ex2 at 2^-21, a sum of at most 5 x 40 at 2^-24 each).  One step more of the scale would be 2^-9 off."""
    group = 5
    rng = np.random.default_rng([73, D, T])
    b = Batch(rng, [(T, T + 9)], 1, D, 16, "bf16", values_too=False)
    b.pages["k"][:] = 0
    b.pages["k"][..., 3] = 0x4300                       # 128
    scale = float(np.float32(np.log(2.0)))
    log2e = np.float32(1.4426950408889634)
    assert np.float32(scale) * log2e == np.float32(1.0)
    q = torch.zeros(T, group, D, dtype=torch.bfloat16, device="cuda")
    q[..., 3] = 128.0
    lse = (16384 * np.log(2.0) + rng.uniform(-1, 1, (T, group))).astype(np.float32)
    w = np.zeros((b.num_pages, 1, 16), np.float32)
    got = weigh(b, b.cache(dsa), dev(w), q, dev(lse), scale)
    each = np.exp2(16384.0 - (lse * log2e).astype(np.float32).astype(np.float64)).sum(1)
    want = np.zeros(w.shape)
    page, slot = E.rows_of(b, 0)
    want[page, 0, slot] = [each[max(0, s - 9):].sum() for s in range(T + 9)]
    close(got, want, want * (2.0 ** -20 + 200 * 2.0 ** -24))


# ---------------------------------------------------------------- pages that do not exist

@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("where", ["sinks", "recent", "between", "within the budget", "last page"])
@pytest.mark.parametrize("page", [-7, 1 << 30])
def test_select_reports_every_missing_page(shared, where, page):
    """A row that has to stay, or a sequence that keeps all its rows, on a page that does not exist: reported like any
    other, and the choice is the same as with a page."""
    rng = np.random.default_rng(74)
    b = Batch(rng, [(0, 400), (0, 37), (0, 90)], 2, 64, 8, "bf16", values_too=False)
    w = E.random_weights(rng, b)
    ws = dsa.cache_workspace()

    def run():
        kept, n = dsa.evict_select(dev(w), b.dev("cu_k"), b.dev("table"), 64, 400, sinks=8, recent=16, shared=shared, ws=ws)
        return host(kept), host(n), dsa.read_status(ws)

    want, n, status = run()
    assert status == 0
    d, i = {"sinks": (0, 0), "recent": (0, 49), "between": (2, 5), "within the budget": (1, 2), "last page": (1, 4)}[where]
    b.table[d, i] = page
    kept, got, status = run()
    assert status == 1 and np.array_equal(got, n)
    if where == "between":      # as NaN: those rows go first
        assert not ((kept[2] >= 40) & (kept[2] < 48)).any()
        kept[2] = want[2]
    assert np.array_equal(kept, want)


def test_select_reports_a_missing_page_of_a_long_sequence():
    """Rows by several blocks of a cluster; one page missing under the recent rows, which other blocks hold than report."""
    rng = np.random.default_rng(75)
    b = Batch(rng, [(0, 20000)], 1, 64, 64, "fp8", values_too=False)
    w = E.random_weights(rng, b)
    ws = dsa.cache_workspace()
    for at in (0, 312, None):
        t = b.table.copy()
        if at is not None:
            b.table[0, at] = b.num_pages
        for budget in (4000, 20000):
            dsa.evict_select(dev(w), b.dev("cu_k"), b.dev("table"), budget, 20000, sinks=64, recent=64, ws=ws)
            assert dsa.read_status(ws) == (0 if at is None else 1), (at, budget)
        b.table = t


# ---------------------------------------------------------------- clusters of eight, rows read again

class Long:
    """Sequences' table and weights alone: what the choice reads."""

    def __init__(self, rng, lens, n_kv, page):
        need = [-(-s // page) for s in lens]
        self.lens, self.n_kv, self.page, self.num_pages = [(0, s) for s in lens], n_kv, page, sum(need) + 2
        order, at = rng.permutation(self.num_pages), 0
        self.table = np.full((len(lens), max(need)), -1, np.int32)
        for d, n in enumerate(need):
            self.table[d, :n] = order[at:at + n]
            at += n
        self.cu_k = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)

    def dev(self, name):
        return torch.from_numpy(getattr(self, name)).cuda()


def choice(b, w, budget, sinks, recent, shared):
    """As E.select, for weights without NaN, by a sort of arrays."""
    heads = 1 if shared else b.n_kv
    kept = np.full((len(b.lens), heads, budget), -1, np.int32)
    for d, (_, s) in enumerate(b.lens):
        page, slot = E.rows_of(b, d)
        x = np.stack([w[page, h, slot] for h in range(b.n_kv)])
        if shared:
            total = x[0]
            for h in range(1, b.n_kv):
                total = (total + x[h]).astype(np.float32)
            x = total[None]
        i = np.arange(s)
        may = ~((i < sinks) | (i >= s - recent))
        for h in range(heads):
            best = np.sort(np.lexsort((i, -x[h], may))[:budget])
            kept[d, h, :len(best)] = best
    return kept, np.array([min(s, budget) for _, s in b.lens], np.int32)


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("lens,kv,shared", [([40000], 5, False), ([40000, 33000, 17, 36000, 9000, 40961], 1, True),
                                            ([330000, 5000], 5, False), ([700000], 2, True)])
def test_select_of_eight_blocks_and_of_rows_read_again(lens, kv, shared, ties):
    """Five heads or more with over 32768 rows: eight blocks to each (fewer heads have sixteen).  Over 327680 rows on
    eight blocks, or 655360 on sixteen, are not held in shared memory: every pass reads the weights again."""
    rng = np.random.default_rng([76, len(lens), kv, ties])
    b = Long(rng, lens, kv, 1024)
    w = E.random_weights(rng, b, ties)
    ws = dsa.cache_workspace()
    for budget, sinks, recent in ((1, 0, 0), (3000, 4, 256), (39999, 0, 7)):
        kept, n = dsa.evict_select(dev(w), b.dev("cu_k"), b.dev("table"), budget, max(lens), sinks=sinks, recent=recent,
                                   shared=shared, ws=ws)
        assert dsa.read_status(ws) == 0
        want, wn = choice(b, w, budget, sinks, recent, shared)
        assert np.array_equal(host(n), wn) and np.array_equal(host(kept), want), (budget, sinks, recent)


# ---------------------------------------------------------------- far queries against far keys

@pytest.mark.parametrize("prec", ["mxfp8", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("far", [-112, -100, -60, 60, 100, 112])
def test_weigh_far_queries_and_far_keys(prec, D, far):
    """Query elements around 2^far, keys around 2^-far: their products, and the logits, are ordinary numbers."""
    rng = np.random.default_rng([77, D, 200 + far])
    b = Batch(rng, [(1, 130)], 1, D, 16, prec, values_too=False, std=2.0 ** -far)
    check_weigh(b, rng, 4, std=2.0 ** far, scale=0.1)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prec", ["bf16", "fp8"])
def test_weights_of_the_attentions_lse_add_up_to_the_heads(D, prec):
    """Logits around 25 under the lse that paged_attention returns: whatever the sums of products lose, logits and lse lose
    alike, so the weights of all tokens add up to their heads.

    A row's sum is off by one factor: the roundings of lse (2^-24 |lse|), of lse log2(e) (as much) and of the attention's own
    scaled maximum (as much), any sign, evenly spread at most: a variance of (3 2^-24 lse)^2 / 3.  The mean over N rows is held
    to six standard deviations, and what does not average out: ex2 here and in the attention 2^-22 each, its log 2^-22."""
    T, S, kv, group, page = 512, 4096, 2, 8, 64
    gen = torch.Generator(device="cuda")
    gen.manual_seed(D)

    def rows(*shape):
        x = torch.randn(shape, generator=gen, device="cuda")
        return x * torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.01, 8.0, 1.0)
    c = dsa.paged_cache(S // page, page, kv, D, prec)
    table = torch.randperm(S // page, generator=gen, device="cuda").to(torch.int32)[None]
    cu = [torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (S, T)]
    dsa.cache_write(c, rows(S, kv, D), rows(S, kv, D), cu[0], cu[0], table)
    q = (2 * rows(T, kv * group, D)).bfloat16()
    _, lse = dsa.paged_attention(q, c, cu[1], cu[0], table, T, S, return_lse=True)
    w = dsa.paged_weights(c)
    dsa.cache_weigh(c, w, q, lse, cu[1], cu[0], table, T, S)
    off = float(w.double().sum() / (T * kv * group)) - 1
    deviation = 2.0 ** -24 * float(3 * lse.double().square().mean() / (T * kv * group)) ** 0.5
    assert abs(off) < 3 * 2.0 ** -22 + 6 * deviation, (off, deviation)
