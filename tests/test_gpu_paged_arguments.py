"""The paged-cache entry points on the arguments at their limits: refused with an
error and nothing written, or taken with the documented result."""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_dsa_gb300 as dsa
from sparse_attention_indexer_dsa_gb300 import _abi
from tests.gpu_util import dev, host
from tests.paged_ref import Batch, attention, quantise, values
from tests.test_gpu_paged_attention import _close, _queries, _run, _selection
from tests.test_gpu_paged_cache import _check_pages

pytestmark = pytest.mark.gpu


def test_expanded_tokens_are_refused():
    rng = np.random.default_rng(71)
    b = Batch(rng, [(5, 40), (3, 9)], 2, 64, 16, "bf16")
    c = b.cache(dsa)
    args = (b.dev("cu_q"), b.dev("cu_k"), b.dev("table"))
    _, one = _queries(rng, 1, 2, 64)
    with pytest.raises(ValueError):
        dsa.cache_write(c, one.expand(8, 2, 64), one.expand(8, 2, 64), *args)
    _, q = _queries(rng, 1, 4, 64)
    with pytest.raises(ValueError):
        dsa.paged_attention(q.expand(8, 4, 64), c, *args, 5, 40)
    torch.cuda.synchronize()
    _check_pages(c, b, b.pages, b.scales)


@pytest.mark.parametrize("prec", ["bf16", "mxfp8", "fp8"])
def test_no_tokens_at_all(prec):
    """Empty tensors in every form that a call takes: nothing is refused, nothing is touched."""
    b = Batch(np.random.default_rng(72), [(0, 5), (0, 0)], 1, 128, 16, prec)
    c, ws = b.cache(dsa), dsa.cache_workspace()
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    args = (none, none, b.dev("table"))
    rows = lambda dt: torch.empty((0, 1, 128), dtype=dt, device="cuda")
    for dt in (torch.float32, torch.bfloat16):
        dsa.cache_write(c, rows(dt), rows(dt), *args, ws=ws)
        assert dsa.read_status(ws) == 0
    if prec != "bf16":
        sc = torch.empty((0, 1, 4 if prec == "mxfp8" else 1), dtype=torch.uint8, device="cuda")
        dsa.cache_write(c, rows(torch.uint8), rows(torch.uint8), *args, k_scale=sc, v_scale=sc, ws=ws)
        assert dsa.read_status(ws) == 0
    for to in (None, "bf16"):
        k, ks, v, vs = dsa.cache_read(c, *args[1:], 0, out_prec=to, ws=ws)
        assert dsa.read_status(ws) == 0 and k.shape == v.shape == (0, 1, 128)
        assert (ks is None) == (vs is None) == (prec == "bf16" or to == "bf16")
    _check_pages(c, b, b.pages, b.scales)


# (cu_q, cu_k) of three sequences that hold 30, 40 and 9 cached tokens; the last one is good
FALLING = [([0, 6, 3, 7], [0, 30, 70, 79]), ([-2, 2, 5, 7], [0, 30, 70, 79]), ([0, 2, 5, 7], [0, 30, 20, 29]),
           ([0, 2, 2, 2], [0, 30, 20, 79])]


@pytest.mark.parametrize("cu", FALLING)
def test_a_write_under_a_falling_prefix_is_reported(cu):
    """Nothing but the sequences' own last positions is touched, and the same workspace's next call is clean."""
    rng = np.random.default_rng(73)
    b = Batch(rng, [(2, 30), (3, 40), (2, 9)], 2, 64, 16, "bf16")
    c, ws, tb = b.cache(dsa), dsa.cache_workspace(), b.dev("table")
    x = torch.ones((7, 2, 64), device="cuda")
    cu_q, cu_k = (dev(np.array(a, np.int32)) for a in cu)
    dsa.cache_write(c, x, x, cu_q, cu_k, tb, ws=ws)
    assert dsa.read_status(ws) == _abi.DSA_ERR_INVALID_ARG
    free = np.ones((b.num_pages, 16), bool)           # slots that no sequence's new tokens can have
    for d, (_, s) in enumerate(b.lens):
        for pos in range(max(0, s - 7), s):
            free[b.table[d, pos // 16], pos % 16] = False
    for n in b.names:
        got = getattr(c, n).view(torch.int16).cpu().numpy().view(np.uint16)
        np.testing.assert_array_equal(got.transpose(0, 2, 1, 3)[free], b.pages[n].transpose(0, 2, 1, 3)[free])
    dsa.cache_write(c, x, x, b.dev("cu_q"), b.dev("cu_k"), tb, ws=ws)
    assert dsa.read_status(ws) == 0


@pytest.mark.parametrize("cu", [[0, 30, 20, 29], [-3, 30, 70, 79], [0, 30, 20, 79]])
def test_a_read_under_a_falling_prefix_is_reported(cu):
    rng = np.random.default_rng(74)
    b = Batch(rng, [(2, 30), (3, 40), (2, 9)], 2, 64, 16, "mxfp8")
    c, ws, tb = b.cache(dsa), dsa.cache_workspace(), b.dev("table")
    out = (torch.full((90, 2, 64), 7, dtype=torch.uint8, device="cuda"),
           torch.full((90, 2, 2), 9, dtype=torch.uint8, device="cuda"), None, None)
    dsa.cache_read(c, dev(np.array(cu, np.int32)), tb, 90, out=out, ws=ws)
    assert dsa.read_status(ws) == _abi.DSA_ERR_INVALID_ARG
    assert bool((out[0][max(cu):] == 7).all()) and bool((out[1][max(cu):] == 9).all())   # behind every sequence
    dsa.cache_read(c, b.dev("cu_k"), tb, 90, out=out, ws=ws)
    assert dsa.read_status(ws) == 0


def test_many_sequences_prefixes_are_looked_at_to_the_end():
    """A fall between any two neighbours of a prefix longer than one block has threads."""
    rng = np.random.default_rng(75)
    n = 1000
    b = Batch(rng, [(1, 3)] * n, 1, 64, 8, "bf16")
    c, ws, tb, ck = b.cache(dsa), dsa.cache_workspace(), b.dev("table"), b.dev("cu_k")
    x = torch.zeros((n, 1, 64), device="cuda")
    for at in (0, 255, 256, 600, n - 2, None):
        cu = b.cu_q.copy()
        if at is not None:
            cu[at + 1] += 2                            # above its right neighbour
        dsa.cache_write(c, x, x, dev(cu), ck, tb, ws=ws)
        assert dsa.read_status(ws) == (0 if at is None else _abi.DSA_ERR_INVALID_ARG), at


# (tokens, cached) of the first sequence, heads to a key head, width of the lists: pairs of query tiles,
# single tiles, lists over tiles of 128 rows and narrow ones
NAN_KINDS = {"pair": ((300, 700), 8, 0), "solo": ((1, 700), 8, 0), "list": ((3, 700), 24, 300), "narrow": ((3, 700), 4, 300)}


@pytest.mark.parametrize("how", ["written", "stored", "scale 255"])
@pytest.mark.parametrize("kind", list(NAN_KINDS))
@pytest.mark.parametrize("prec", ["bf16", "mxfp8", "fp8"])
def test_a_nan_stays_a_nan(prec, kind, how):
    """A NaN in a row that every query of sequence 0 sees: written with the new tokens, or among the
    stored rows.  In K the results of its key head's queries are NaN, in V those of the element; the
    other key head and the other sequence have their own results, bit by bit within the bound."""
    if how == "scale 255" and prec == "bf16":
        pytest.skip("no scales")
    rng = np.random.default_rng(76)
    (t, s), group, W = NAN_KINDS[kind]
    b = Batch(rng, [(t, s), (1, 200)], 2, 128, 16, prec)
    sel = None
    if W:
        sel = _selection(rng, b, W, "sorted")[0]
        sel[:t, 0] = s - t
    q, qd = _queries(rng, b.total_q, 2 * group, 128)
    cu_q, cu_k, tb = b.dev("cu_q"), b.dev("cu_k"), b.dev("table")
    pos, dim = s - t, 70                       # the first new token: visible to all of them
    pg, sl = int(b.table[0, pos // 16]), pos % 16
    for n in b.names:
        c = b.cache(dsa)
        if how == "written":
            new = {m: np.concatenate([b.rows[m][e - u:e] for e, (u, _) in zip(b.cu_k[1:], b.lens)]) for m in b.names}
            new[n][0, 1, dim] = np.nan
            dsa.cache_write(c, dev(new["k"].astype(np.float32)), dev(new["v"].astype(np.float32)), cu_q, cu_k, tb)
        elif prec == "bf16":
            getattr(c, n)[pg, 1, sl, dim] = float("nan")
        elif how == "stored":
            getattr(c, n)[pg, 1, sl, dim] = 0xFF
            getattr(c, n + "_scale")[pg, 1, sl] = 248
        else:
            getattr(c, n + "_scale")[pg, 1, sl] = 255
        back = dsa.cache_read(c, cu_k, tb, b.total_k, out_prec="bf16")[0 if n == "k" else 2]
        gone = torch.isnan(back)
        assert bool(gone[pos, 1, dim]) and not bool(gone[:, 0].any()) and int(gone[:, 1].any(1).sum()) == 1
        out, lse = dsa.paged_attention(qd, c, cu_q, cu_k, tb, t, s, topk_idx=None if sel is None else dev(sel),
                                       return_lse=True)
        want, wl, tol, ltol = attention(b, q, group, 128 ** -0.5, sel)
        got, gl = host(out.double()), host(lse.double())
        if n == "k":
            assert np.isnan(got[:t, group:]).all() and np.isnan(gl[:t, group:]).all()
        else:
            assert np.isnan(got[:t, group:, dim]).all()
            _close(gl[:t, group:], wl[:t, group:], ltol[:t, group:])
        _close(got[:, :group], want[:, :group], tol[:, :group])
        _close(got[t:], want[t:], tol[t:])
        _close(gl[:, :group], wl[:, :group], ltol[:, :group])


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -126, 2.0 ** -140])
@pytest.mark.parametrize("kind", list(NAN_KINDS))
@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
def test_the_smallest_scales_on_the_largest_logits(prec, kind, scale):
    """Products of +-2^126: a scale of 0 gives every seen key the same weight, one of 2^-126 the
    logits +-1, one below FP32's normal numbers next to none."""
    rng = np.random.default_rng(77)
    (t, s), group, W = NAN_KINDS[kind]
    b = Batch(rng, [(t, s)], 1, 128, 16, prec)
    row = np.zeros((s, 1, 128))
    row[:, 0, 0] = rng.choice([-1.0, 1.0], s) * 2.0 ** 63
    st, sc = quantise(row, prec)
    b.rows["k"] = values(st, sc, prec)
    for pos in range(s):
        b.pages["k"][b.table[0, pos // 16], :, pos % 16] = st[pos]
        if sc is not None:
            b.scales["k"][b.table[0, pos // 16], :, pos % 16] = sc[pos]
    q = np.zeros((t, group, 128))
    q[:, :, 0] = 2.0 ** 63
    sel = _selection(rng, b, W, "sorted")[0] if W else None
    out, lse = dsa.paged_attention(dev(q.astype(np.float32)).to(torch.bfloat16), b.cache(dsa), b.dev("cu_q"), b.dev("cu_k"),
                                   b.dev("table"), t, s, sm_scale=scale, topk_idx=None if sel is None else dev(sel),
                                   return_lse=True)
    want, wl, tol, ltol = attention(b, q, group, scale, sel)
    _close(host(out.double()), want, tol)
    _close(host(lse.double()), wl, ltol)


@pytest.mark.parametrize("kind", ["chunk", "steps", "list"])
def test_a_call_without_a_workspace_allocates_its_own_alone(kind):
    """Where the plan divides no key range that is the status header; the results are those of a call
    with a workspace for every smaller one."""
    rng = np.random.default_rng(78)
    lens, W = {"chunk": ([(6000, 6400)], 0), "steps": ([(1, 200)] * 40, 0), "list": ([(700, 900)], 96)}[kind]
    c = dsa.paged_cache(200, 64, 4, 128)
    c.k.normal_()
    c.v.normal_()
    t, s = np.array(lens).T
    cu_q, cu_k = (dev(np.concatenate([[0], np.cumsum(x)]).astype(np.int32)) for x in (t, s))
    need = [-(-x // 64) for x in s]
    table = np.full((len(lens), max(need)), -1, np.int32)
    for d, n in enumerate(need):
        table[d, :n] = rng.permutation(200)[:n]
    T = int(t.sum())
    q = torch.randn((T, 16, 128), device="cuda").to(torch.bfloat16)
    sel = dev(rng.integers(0, 100, (T, W)).astype(np.int32)) if W else None
    args = (q, c, cu_q, cu_k, dev(table), int(t.max()), int(s.max()))
    out = torch.empty_like(q)
    ws = dsa.attention_workspace(T, len(lens), int(t.max()), 16, 4, 128, W)
    want = dsa.paged_attention(*args, topk_idx=sel, ws=ws)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    dsa.paged_attention(*args, topk_idx=sel, out=out)
    assert torch.cuda.max_memory_allocated() - before <= 16384
    assert torch.equal(out, want)


@pytest.mark.parametrize("prec", ["bf16", "mxfp8", "fp8"])
def test_a_chunk_beside_single_tokens(prec):
    """One long chunk makes the call's tiles pairs; the single tokens beside it take a pair each, whose
    second tile is empty."""
    rng = np.random.default_rng(79)
    b = Batch(rng, [(1, 1), (400, 900), (1, 300), (0, 70), (1, 1290)] + [(1, int(n)) for n in rng.integers(1, 500, 9)],
              2, 128, 32, prec)
    _run(b, rng, 16, 8)


def test_two_host_threads():
    """Calls from two threads at once, each with its stream, workspace and cache: the results are those
    of the same calls one after the other, and an error is its own thread's."""
    import threading
    rng = np.random.default_rng(80)
    jobs = []
    for prec, lens, W in (("mxfp8", [(1, 3000), (1, 70)], 0), ("bf16", [(20, 600), (3, 90)], 64)):
        b = Batch(rng, lens, 2, 128, 16, prec)
        sel = dev(_selection(rng, b, W, "sorted")[0]) if W else None
        _, qd = _queries(rng, b.total_q, 16, 128)
        ws = dsa.attention_workspace(b.total_q, 2, max(t for t, _ in lens), 16, 2, 128, W)
        args = (qd, b.cache(dsa), b.dev("cu_q"), b.dev("cu_k"), b.dev("table"), max(t for t, _ in lens), max(s for _, s in lens))
        jobs.append((args, dict(topk_idx=sel, ws=ws)))
    want = [dsa.paged_attention(*a, **k) for a, k in jobs]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            args, kw = jobs[i]
            with torch.cuda.stream(torch.cuda.Stream()):
                out = torch.empty_like(want[i])
                for n in range(100):
                    dsa.paged_attention(*args, out=out, **kw)
                    if n % 10 == 0:
                        with pytest.raises(dsa.DsaError) as e:
                            dsa.paged_attention(*args, topk_idx=kw["topk_idx"], out=out, ws=kw["ws"][:256 * (i + 1)])
                        assert f"workspace {256 * (i + 1)} bytes" in str(e.value)
                assert dsa.read_status(kw["ws"]) == 0
                assert torch.equal(out, want[i])
        except BaseException as e:   # noqa: B902 (reported by the test's thread)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
