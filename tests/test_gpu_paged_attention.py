"""Attention over the paged cache against its formula in 64 bits.

The tolerance is the derived bound of tests/paged_ref.py: every product is
exact, sums are FP32, the softmax weights and the result are rounded to BF16
once each."""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_dsa_gb300 as dsa
from sparse_attention_indexer_dsa_gb300 import _abi
from tests.gpu_util import bf16_dev, dev, host
from tests.paged_ref import Batch, attention, quantise, values

pytestmark = pytest.mark.gpu


def _queries(rng, T, H, D, std=1.0):
    bits, _ = quantise(rng.standard_normal((T, H, D)) * std, "bf16")
    return values(bits, None, "bf16"), bf16_dev(bits)


def _close(got, want, tol, what=""):
    err = np.abs(got - want) - tol
    assert not np.isnan(got).any(), what
    assert (err <= 0).all(), (what, np.unravel_index(err.argmax(), err.shape), float(err.max()))


def _run(b, rng, H, group, sel=None, sel_len=None, std=2.0, scale=None, **kw):
    q, qd = _queries(rng, b.total_q, H, b.D, std)
    scale = b.D ** -0.5 if scale is None else scale
    c = b.cache(dsa)
    max_q, max_k = max(t for t, _ in b.lens), max(s for _, s in b.lens)
    ws = dsa.attention_workspace(b.total_q, len(b.lens), max_q, H, H // group, b.D, 0 if sel is None else sel.shape[1])
    out, lse = dsa.paged_attention(qd, c, b.dev("cu_q"), b.dev("cu_k"), b.dev("table"), max_q, max_k, sm_scale=scale,
                                   topk_idx=None if sel is None else dev(sel),
                                   topk_len=None if sel_len is None else dev(sel_len), return_lse=True, ws=ws, **kw)
    assert dsa.read_status(ws) == 0
    n = int(b.cu_q[-1])
    want, wl, tol, ltol = attention(b, q[:n], group, scale, sel, sel_len)
    _close(host(out.double())[:n], want, tol, "out")
    g = host(lse.double())[:n]
    dead = np.isinf(wl)
    assert (g[dead] == -np.inf).all()
    _close(g[~dead], wl[~dead], ltol[~dead], "lse")
    return out, lse


LENS = {
    "one": [(1, 1)],
    "steps": [(1, 1), (1, 127), (1, 128), (0, 9), (1, 129), (1, 600)],
    "chunk": [(33, 33), (0, 0), (17, 300), (1, 260), (130, 131)],
    "prompt": [(257, 257)],
}


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("kv,group", [(1, 1), (2, 8), (1, 64), (3, 5)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prec", ["bf16", "mxfp8", "fp8"])
def test_every_visible_key(prec, D, kv, group, lens):
    rng = np.random.default_rng(31)
    page = {"one": 8, "steps": 64, "chunk": 16, "prompt": 128}[lens]
    b = Batch(rng, LENS[lens], kv, D, page, prec)
    _run(b, rng, kv * group, group)


def _selection(rng, b, W, kind):
    T = b.total_q
    sel = np.full((T, W), -1, np.int32)
    lens = np.zeros(T, np.int32)
    for d, (t, s) in enumerate(b.lens):
        for i in range(t):
            r, pos = b.cu_q[d] + i, s - t + i
            if kind == "sorted":
                n = min(W, pos + 1)
                sel[r, :n] = np.sort(rng.permutation(pos + 1)[:n])
                lens[r] = n
            else:   # any order, gaps, positions not visible, repeats, rows with nothing
                sel[r] = rng.integers(-3, s + 40, W)
                lens[r] = rng.integers(-1, W + 3)
                if r % 5 == 0:
                    sel[r] = -1
                if r % 7 == 3:
                    sel[r] = pos + 1
    return sel, lens


@pytest.mark.parametrize("kind", ["sorted", "wild"])
@pytest.mark.parametrize("W", [1, 40, 129, 300])
@pytest.mark.parametrize("kv,group", [(1, 16), (1, 64), (2, 5)])
@pytest.mark.parametrize("D,prec", [(128, "bf16"), (64, "bf16"), (128, "mxfp8"), (64, "mxfp8"), (128, "fp8")])
def test_selected_keys(D, prec, kv, group, W, kind):
    rng = np.random.default_rng(32)
    b = Batch(rng, [(1, 1), (9, 350), (0, 5), (20, 20), (1, 128)], kv, D, 16, prec)
    sel, lens = _selection(rng, b, W, kind)
    _run(b, rng, kv * group, group, sel, lens)
    _run(b, rng, kv * group, group, sel)


def test_selection_of_everything_equals_no_selection():
    rng = np.random.default_rng(33)
    b = Batch(rng, [(40, 200)], 2, 128, 16, "bf16")
    sel = np.broadcast_to(np.arange(200, dtype=np.int32), (40, 200)).copy()
    q, _ = _run(b, np.random.default_rng(34), 16, 8)
    s, _ = _run(b, np.random.default_rng(34), 16, 8, sel)
    _close(host(q.double()), host(s.double()), 2 * 2.0 ** -8 * (np.abs(host(q.double())) + 0.5))


@pytest.mark.parametrize("scale,std", [(0.0, 1.0), (1e-3, 1.0), (3.0, 3.0)])
def test_flat_and_peaked_weights(scale, std):
    rng = np.random.default_rng(35)
    b = Batch(rng, [(3, 500), (200, 300)], 1, 128, 32, "bf16", std=std)
    _run(b, rng, 8, 8, std=std, scale=scale)


def test_rising_logits_rescale_the_sums():
    """Keys whose logits grow along the sequence: the running maximum moves in every tile."""
    rng = np.random.default_rng(36)
    b = Batch(rng, [(2, 900), (150, 700)], 1, 64, 16, "bf16")
    for d, (t, s) in enumerate(b.lens):
        for pos in range(s):
            bits, _ = quantise(np.concatenate([[0.05 * pos], 0.2 * rng.standard_normal(63)])[None], "bf16")
            b.pages["k"][b.table[d, pos // 16], 0, pos % 16] = bits
            b.rows["k"][b.cu_k[d] + pos, 0] = values(bits, None, "bf16")
    q, qd = _queries(rng, b.total_q, 4, 64)
    q[:, :, 0], qd[:, :, 0] = 8.0, 8.0
    want, wl, tol, ltol = attention(b, q, 4, 1.0)
    out, lse = dsa.paged_attention(qd, b.cache(dsa), b.dev("cu_q"), b.dev("cu_k"), b.dev("table"), 150, 900, sm_scale=1.0,
                                   return_lse=True)
    _close(host(out.double()), want, tol)
    _close(host(lse.double()), wl, ltol)


def test_padded_batch_and_strided_queries():
    rng = np.random.default_rng(37)
    b = Batch(rng, [(5, 70), (20, 33)], 2, 128, 16, "mxfp8", pad_q=4)
    fused, fd = _queries(rng, b.total_q, 16 + 4, 128)
    qd = fd[:, 2:18]
    out = torch.full((b.total_q, 16, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.total_q, 16), 5.0, device="cuda")
    dsa.paged_attention(qd, b.cache(dsa), b.dev("cu_q"), b.dev("cu_k"), b.dev("table"), 20, 70, return_lse=True,
                        out=(out, lse))
    n = int(b.cu_q[-1])
    want, wl, tol, ltol = attention(b, fused[:n, 2:18], 8, 128 ** -0.5)
    _close(host(out.double())[:n], want, tol)
    _close(host(lse.double())[:n], wl, ltol)
    assert bool((out[n:] == 3).all()) and bool((lse[n:] == 5).all())


@pytest.mark.parametrize("lens,group", [([(1, 5000)], 4), ([(1, 3000), (1, 10), (1, 7000)], 8), ([(40, 4000)], 16),
                                        ([(200, 3500), (1, 900)], 16)])
def test_long_key_ranges(lens, group):
    """Few rows over many keys: the range is divided and joined."""
    rng = np.random.default_rng(38)
    b = Batch(rng, lens, 1, 128, 64, "mxfp8")
    _run(b, rng, group, group)
    again = [_run(b, np.random.default_rng(39), group, group)[0] for _ in range(2)]
    assert torch.equal(again[0], again[1])


def test_many_sequences():
    rng = np.random.default_rng(40)
    lens = [(int(rng.integers(0, 3)), int(rng.integers(3, 60))) for _ in range(700)]
    b = Batch(rng, lens, 1, 64, 16, "bf16")
    _run(b, rng, 4, 4)


def test_page_order_does_not_matter_beyond_32_bits():
    """Rows of a cache whose byte offsets pass 2^32."""
    pages, page, D = 9000, 1024, 128                  # 9000 * 2 * 1024 rows of 256 bytes = 4.7 GB for each of k and v
    c = dsa.paged_cache(pages, page, 2, D)
    rng = np.random.default_rng(41)
    b = Batch(rng, [(3, 1500)], 2, D, page, "bf16", extra_pages=0)
    far = np.array([pages - 1, pages - 2], np.int32)
    small = b.cache(dsa)
    for i, pg in enumerate(b.table[0, :2]):
        c.k[int(far[i])] = small.k[int(pg)]
        c.v[int(far[i])] = small.v[int(pg)]
    q, qd = _queries(rng, 3, 8, D)
    out = dsa.paged_attention(qd, c, b.dev("cu_q"), b.dev("cu_k"), dev(far[None]), 3, 1500)
    want, _, tol, _ = attention(b, q, 4, D ** -0.5)
    _close(host(out.double()), want, tol)
    new, newd = _queries(rng, 3, 2, D)
    dsa.cache_write(c, newd, newd, b.dev("cu_q"), b.dev("cu_k"), dev(far[None]))
    k, _, v, _ = dsa.cache_read(c, b.dev("cu_k"), dev(far[None]), 1500)
    np.testing.assert_array_equal(host(k.double())[1497:], new)
    np.testing.assert_array_equal(host(v.double())[:1497], b.rows["v"][:1497])


def test_what_the_device_finds_wrong():
    rng = np.random.default_rng(42)
    b = Batch(rng, [(4, 20), (3, 40)], 2, 64, 16, "bf16")
    q, qd = _queries(rng, b.total_q, 4, 64)
    want, _, tol, _ = attention(b, q, 2, 0.125)
    ws = dsa.attention_workspace(b.total_q, 2, 4, 4, 2, 64)
    c = b.cache(dsa)
    args = (b.dev("cu_q"), b.dev("cu_k"))
    for bad in (-1, b.num_pages, 1 << 30):
        table = b.table.copy()
        table[0, 0] = bad
        out = dsa.paged_attention(qd, c, *args, dev(table), 4, 40, ws=ws)
        assert dsa.read_status(ws) == _abi.DSA_ERR_INVALID_ARG
        _close(host(out.double())[4:], want[4:], tol[4:])            # the other sequence
    for cu_q, cu_k, mq, mk in (([0, 4, 7], [0, 3, 43], 4, 40), ([0, 4, 47], [0, 20, 60], 64, 64),
                               ([0, 4, 7], [0, 20, 60], 3, 40), ([0, 4, 7], [0, 20, 60], 4, 39),
                               ([0, 4, 7], [0, 20, 400], 4, 400)):
        w2 = dsa.attention_workspace(b.total_q, 2, mq, 4, 2, 64)
        dsa.paged_attention(qd, c, dev(np.array(cu_q, np.int32)), dev(np.array(cu_k, np.int32)), b.dev("table"), mq, mk,
                            ws=w2)
        assert dsa.read_status(w2) == _abi.DSA_ERR_INVALID_ARG
    out = dsa.paged_attention(qd, c, *args, b.dev("table"), 4, 40, ws=ws)
    assert dsa.read_status(ws) == 0
    _close(host(out.double()), want, tol)


def test_nothing_new():
    rng = np.random.default_rng(43)
    b = Batch(rng, [(0, 5), (0, 0)], 2, 64, 16, "fp8")
    out = dsa.paged_attention(torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda"), b.cache(dsa), b.dev("cu_q"),
                              b.dev("cu_k"), b.dev("table"), 0, 5)
    assert out.shape == (0, 4, 64)


def test_graphs_and_streams():
    """Captured on another stream and replayed with new contents and lengths; two
    calls with a workspace each run at the same time."""
    rng = np.random.default_rng(44)
    b = Batch(rng, [(1, 700), (1, 90)], 2, 128, 16, "mxfp8")
    c = b.cache(dsa)
    q, qd = _queries(rng, 2, 16, 128)
    cu_q, cu_k, table = b.dev("cu_q"), b.dev("cu_k"), b.dev("table")
    ws = [dsa.attention_workspace(2, 2, 1, 16, 2, 128) for _ in range(2)]
    outs = [torch.zeros((2, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for i in range(2):
        streams[i].wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            dsa.paged_attention(qd, c, cu_q, cu_k, table, 1, 700, out=outs[i], ws=ws[i])
        graphs.append(g)
    for lens in ([(1, 700), (1, 90)], [(1, 650), (1, 1)]):
        short = b
        if lens != b.lens:
            short = Batch(np.random.default_rng(44), [(1, 700), (1, 90)], 2, 128, 16, "mxfp8")
            keep = np.concatenate([np.arange(s) + short.cu_k[d] for d, (_, s) in enumerate(lens)])
            short.rows = {n: r[keep] for n, r in short.rows.items()}
            short.lens = lens
            short.cu_k = np.array([0, 650, 651], np.int32)
            cu_k.copy_(dev(short.cu_k))
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        want, _, tol, _ = attention(short, q, 8, 128 ** -0.5)
        for o in outs:
            _close(host(o.double()), want, tol)


def test_a_serving_step():
    """The run these operators are for: new tokens are preprocessed and stored, the
    index keys come back as the scoring operand, the selected rows are attended to.
    The pieces agree with the same calls without a cache."""
    rng = np.random.default_rng(45)
    lens = [(5, 300), (1, 77), (64, 64)]
    H, D, kv, topk = 16, 128, 2, 48
    Sk, Tq = sum(s for _, s in lens), sum(t for t, _ in lens)
    cu_q = np.concatenate([[0], np.cumsum([t for t, _ in lens])]).astype(np.int32)
    cu_k = np.concatenate([[0], np.cumsum([s for _, s in lens])]).astype(np.int32)
    new = np.concatenate([np.arange(cu_k[d + 1] - t, cu_k[d + 1]) for d, (t, _) in enumerate(lens)])
    old = np.setdiff1d(np.arange(Sk), new)
    iq = dev(rng.standard_normal((Sk, H, D)).astype(np.float32))
    ik = dev(rng.standard_normal((Sk, D)).astype(np.float32))
    w = dev(rng.standard_normal((Tq, H)).astype(np.float32))
    q_op, q_sc, k_op, k_sc = dsa.preprocess(iq, ik, dev(cu_k), 300, rope_dim=64, out_prec="mxfp8")
    q_op = q_op.view(Sk, H, D)[new].reshape(-1, D).contiguous()
    q_sc = q_sc.view(Sk, H, 4)[new].reshape(-1, 4).contiguous()
    K, V = (dev(rng.standard_normal((Sk, kv, D)).astype(np.float32)) for _ in range(2))
    qd = dev(rng.standard_normal((Tq, H, D)).astype(np.float32)).to(torch.bfloat16)
    page = 32
    need = [-(-s // page) for _, s in lens]
    table = np.full((3, max(need)), -1, np.int32)
    order, at = rng.permutation(sum(need)), 0
    for d, n in enumerate(need):
        table[d, :n] = order[at:at + n]
        at += n
    index_cache = dsa.paged_cache(sum(need), page, 1, D, "mxfp8", values=False)
    kv_cache = dsa.paged_cache(sum(need), page, kv, D, "mxfp8")
    tb, ck, cq = dev(table), dev(cu_k), dev(cu_q)
    before = [s - t for t, s in lens]
    cu_b = dev(np.concatenate([[0], np.cumsum(before)]).astype(np.int32))
    o = dev(old)
    # what is there already: a chunk of its own; then the new tokens
    dsa.cache_write(index_cache, k_op[o][:, None].contiguous(), None, cu_b, cu_b, tb, k_scale=k_sc[o][:, None].contiguous())
    dsa.cache_write(kv_cache, K[o], V[o], cu_b, cu_b, tb)
    n = dev(new)
    dsa.cache_write(index_cache, k_op[n][:, None].contiguous(), None, cq, ck, tb, k_scale=k_sc[n][:, None].contiguous())
    dsa.cache_write(kv_cache, K[n], V[n], cq, ck, tb)
    keys, scales, _, _ = dsa.cache_read(index_cache, ck, tb, Sk)
    assert torch.equal(keys[:, 0], k_op) and torch.equal(scales[:, 0], k_sc)
    idx, sc, ln = dsa.score_topk_kv(q_op, q_sc, keys[:, 0], scales[:, 0], w, cq, ck, 64, 300, H, topk, "mxfp8")
    idx2, sc2, ln2 = dsa.score_topk_kv(q_op, q_sc, k_op, k_sc, w, cq, ck, 64, 300, H, topk, "mxfp8")
    assert torch.equal(idx, idx2) and torch.equal(sc, sc2) and torch.equal(ln, ln2)
    out = dsa.paged_attention(qd, kv_cache, cq, ck, tb, 64, 300, topk_idx=idx, topk_len=ln)
    b = Batch(rng, lens, kv, D, page, "mxfp8")
    for nm, x in (("k", K), ("v", V)):
        st, s8 = quantise(host(x.double()), "mxfp8")
        b.rows[nm] = values(st, s8, "mxfp8")
    want, _, tol, _ = attention(b, host(qd.double()), H // kv, D ** -0.5, host(idx), host(ln))
    _close(host(out.double()), want, tol)
