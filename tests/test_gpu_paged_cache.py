"""Cache write and read-back against the oracle's quantisers, bit for bit."""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_dsa_gb300 as dsa
from sparse_attention_indexer_dsa_gb300 import _abi
from tests.gpu_util import bf16_dev, dev, host
from tests.paged_ref import Batch, quantise, scale_width, values

pytestmark = pytest.mark.gpu

LENS = {
    "one": [(1, 1)],
    "steps": [(1, 1), (1, 64), (1, 65), (0, 7), (1, 200)],
    "ragged": [(37, 37), (0, 0), (5, 131), (64, 64), (130, 259), (0, 3)],
}


def _stored(t):
    a = t.view(torch.int16) if t.dtype == torch.bfloat16 else t
    a = host(a)
    return a.view(np.uint16) if a.dtype == np.int16 else a


def _expect_write(b, new, rule="nosat"):
    """Pages and scales after the new rows {name: float64 [T, n_kv, D]} are stored."""
    pages = {n: b.pages[n].copy() for n in b.names}
    scales = {n: None if b.scales[n] is None else b.scales[n].copy() for n in b.names}
    for n in b.names:
        st, sc = quantise(new[n], b.prec, rule)
        for d, (t, s) in enumerate(b.lens):
            for i in range(t):
                pos = s - t + i
                pg, sl = b.table[d, pos // b.page], pos % b.page
                pages[n][pg, :, sl] = st[b.cu_q[d] + i]
                if sc is not None:
                    scales[n][pg, :, sl] = sc[b.cu_q[d] + i]
    return pages, scales


def _check_pages(c, b, pages, scales):
    for n in b.names:
        np.testing.assert_array_equal(_stored(getattr(c, n)), pages[n])
        if scales[n] is not None:
            np.testing.assert_array_equal(host(getattr(c, n + "_scale")), scales[n])


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("src", ["f32", "bf16"])
@pytest.mark.parametrize("prec", ["bf16", "mxfp8", "fp8"])
def test_write(prec, src, D, lens):
    rng = np.random.default_rng(21)
    n_kv, page = {"one": (1, 8), "steps": (8, 64), "ragged": (3, 16)}[lens]
    b = Batch(rng, LENS[lens], n_kv, D, page, prec, pad_q=3)
    new, args = {}, []
    for n in b.names:
        x = rng.standard_normal((b.total_q, n_kv, D)) * np.exp2(rng.integers(-20, 20, (b.total_q, n_kv, 1)))
        x[0] = 0.0
        x = x.astype(np.float32)
        if src == "bf16":
            bits = (x.view(np.uint32) >> 16).astype(np.uint16)
            args.append(bf16_dev(bits))
            x = values(bits, None, "bf16")
        else:
            args.append(dev(x))
        new[n] = x.astype(np.float64)
    c = b.cache(dsa)
    ws = dsa.cache_workspace()
    dsa.cache_write(c, *args, b.dev("cu_q"), b.dev("cu_k"), b.dev("table"), ws=ws)
    assert dsa.read_status(ws) == 0
    _check_pages(c, b, *_expect_write(b, new))


def test_write_floor_rule_strides_and_keys_alone():
    rng = np.random.default_rng(22)
    b = Batch(rng, LENS["ragged"], 2, 128, 32, "mxfp8")
    qkv = torch.from_numpy(rng.standard_normal((b.total_q, 7, 128)).astype(np.float32)).cuda().to(torch.bfloat16)
    k, v = qkv[:, 3:5], qkv[:, 5:7]
    c = b.cache(dsa)
    dsa.cache_write(c, k, v, b.dev("cu_q"), b.dev("cu_k"), b.dev("table"), scale_rule="floor")
    new = {n: host(t.double()) for n, t in (("k", k), ("v", v))}
    _check_pages(c, b, *_expect_write(b, new, "floor"))
    b1 = Batch(rng, LENS["steps"], 1, 128, 64, "fp8", values_too=False)
    x = rng.standard_normal((b1.total_q, 1, 128)).astype(np.float32)
    c1 = b1.cache(dsa)
    dsa.cache_write(c1, dev(x), None, b1.dev("cu_q"), b1.dev("cu_k"), b1.dev("table"))
    _check_pages(c1, b1, *_expect_write(b1, {"k": x.astype(np.float64)}))


@pytest.mark.parametrize("prec", ["mxfp8", "fp8"])
def test_write_operands_as_they_are(prec):
    """Codes and scales of a preprocess call enter the cache unchanged, every code included."""
    rng = np.random.default_rng(23)
    b = Batch(rng, LENS["ragged"], 1, 128, 16, prec)
    n = scale_width(prec, 128)
    codes = {m: rng.integers(0, 256, (b.total_q, 1, 128)).astype(np.uint8) for m in b.names}
    sc = {m: rng.integers(0, 256, (b.total_q, 1, n)).astype(np.uint8) for m in b.names}
    c = b.cache(dsa)
    dsa.cache_write(c, dev(codes["k"]), dev(codes["v"]), b.dev("cu_q"), b.dev("cu_k"), b.dev("table"),
                    k_scale=dev(sc["k"]), v_scale=dev(sc["v"]))
    pages, scales = {m: b.pages[m].copy() for m in b.names}, {m: b.scales[m].copy() for m in b.names}
    for d, (t, s) in enumerate(b.lens):
        for i in range(t):
            pos = s - t + i
            for m in b.names:
                pages[m][b.table[d, pos // 16], :, pos % 16] = codes[m][b.cu_q[d] + i]
                scales[m][b.table[d, pos // 16], :, pos % 16] = sc[m][b.cu_q[d] + i]
    _check_pages(c, b, pages, scales)


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prec,to", [("bf16", None), ("mxfp8", None), ("fp8", None), ("mxfp8", "bf16"), ("fp8", "bf16")])
def test_read(prec, to, D, lens):
    rng = np.random.default_rng(24)
    n_kv, page = {"one": (1, 8), "steps": (1, 64), "ragged": (5, 16)}[lens]
    b = Batch(rng, LENS[lens], n_kv, D, page, prec, values_too=lens != "steps")
    c = b.cache(dsa)
    ws = dsa.cache_workspace()
    k, ks, v, vs = dsa.cache_read(c, b.dev("cu_k"), b.dev("table"), b.total_k, out_prec=to, ws=ws)
    assert dsa.read_status(ws) == 0
    assert (v is None) == ("v" not in b.names)
    for n, t, s in (("k", k, ks), ("v", v, vs)):
        if t is None:
            continue
        if to is None and prec != "bf16":
            np.testing.assert_array_equal(values(host(t), host(s), prec), b.rows[n])
        else:
            assert s is None
            np.testing.assert_array_equal(host(t.double()), b.rows[n])


def test_read_every_code_and_scale_to_bf16():
    """All finite codes under every scale byte, against a correct rounding to BF16."""
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)
    codes = np.resize(codes, (256, 1, 2, 128))
    codes[:, :, 1] = np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)[-128:]
    scales = np.broadcast_to(np.arange(256, dtype=np.uint8)[:, None, None, None], (256, 1, 2, 1)).copy()
    scales[255] = 254
    c8, s8 = np.zeros((256, 1, 8, 128), np.uint8), np.full((256, 1, 8, 1), 127, np.uint8)
    c8[:, :, :2], s8[:, :, :2] = codes, scales
    c = dsa.PagedCache(dev(c8), dev(s8), None, None, "fp8")
    cu = dev(np.array([0, 2048], np.int32))
    table = dev(np.arange(256, dtype=np.int32)[None])
    got = host(dsa.cache_read(c, cu, table, 2048, out_prec="bf16")[0].double()).reshape(256, 8, 128)
    want = values(c8, s8, "fp8").reshape(256, 8, 128)
    want = torch.from_numpy(want).to(torch.float32).to(torch.bfloat16).double().numpy()   # FP32 holds them all
    big = np.abs(want) == np.inf
    assert not big[:240].any()
    np.testing.assert_array_equal(got, want)


def test_rows_behind_the_last_sequence_stay():
    rng = np.random.default_rng(25)
    b = Batch(rng, LENS["ragged"], 2, 64, 16, "mxfp8", pad_q=9)
    c = b.cache(dsa)
    out = (torch.full((b.total_k + 6, 2, 64), 7, dtype=torch.uint8, device="cuda"),
           torch.full((b.total_k + 6, 2, 2), 9, dtype=torch.uint8, device="cuda"), None, None)
    dsa.cache_read(c, b.dev("cu_k"), b.dev("table"), b.total_k + 6, out=out)
    assert bool((out[0][b.total_k:] == 7).all()) and bool((out[1][b.total_k:] == 9).all())
    np.testing.assert_array_equal(values(host(out[0][:b.total_k]), host(out[1][:b.total_k]), "mxfp8"), b.rows["k"])


def test_what_the_device_finds_wrong():
    """Pages and lengths that do not fit are reported; the good rows are still written."""
    rng = np.random.default_rng(26)
    b = Batch(rng, [(4, 20), (3, 40)], 2, 64, 16, "bf16")
    x = {n: rng.integers(-3, 4, (b.total_q, 2, 64)).astype(np.float32) for n in b.names}
    pages, scales = _expect_write(b, {n: v.astype(np.float64) for n, v in x.items()})
    for bad in (-1, b.num_pages, 1 << 30):
        c = b.cache(dsa)
        table = b.table.copy()
        table[0, 1] = bad                      # positions 16..19 of sequence 0: its four new tokens
        ws = dsa.cache_workspace()
        dsa.cache_write(c, dev(x["k"]), dev(x["v"]), b.dev("cu_q"), b.dev("cu_k"), dev(table), ws=ws)
        assert dsa.read_status(ws) == _abi.DSA_ERR_INVALID_ARG
        for n in b.names:
            want = pages[n].copy()
            want[b.table[0, 1]] = b.pages[n][b.table[0, 1]]
            np.testing.assert_array_equal(_stored(getattr(c, n)), want)
        dsa.cache_read(c, b.dev("cu_k"), dev(table), b.total_k, ws=ws)
        assert dsa.read_status(ws) == _abi.DSA_ERR_INVALID_ARG
    c = b.cache(dsa)
    ws = dsa.cache_workspace()
    for cu_q, cu_k in (([0, 4, 47], [0, 20, 60]),      # more new tokens than cached ones; more than the tensor holds
                       ([0, 4, 7], [0, 3, 43]),        # sequence 0: 4 new, 3 cached
                       ([0, 4, 7], [0, 20, 400])):     # behind the page table
        dsa.cache_write(c, dev(x["k"]), dev(x["v"]), dev(np.array(cu_q, np.int32)), dev(np.array(cu_k, np.int32)),
                        b.dev("table"), ws=ws)
        assert dsa.read_status(ws) == _abi.DSA_ERR_INVALID_ARG
    dsa.cache_read(c, b.dev("cu_k"), b.dev("table"), b.total_k - 1, ws=ws)
    assert dsa.read_status(ws) == _abi.DSA_ERR_INVALID_ARG
    dsa.cache_read(c, b.dev("cu_k"), b.dev("table"), b.total_k, ws=ws)      # a later good call clears it
    assert dsa.read_status(ws) == 0


def test_nothing_new():
    rng = np.random.default_rng(27)
    b = Batch(rng, [(0, 5), (0, 0)], 2, 64, 16, "fp8")
    c = b.cache(dsa)
    ws = dsa.cache_workspace()
    e = torch.empty((0, 2, 64), device="cuda")
    dsa.cache_write(c, e, e, b.dev("cu_q"), b.dev("cu_k"), b.dev("table"), ws=ws)
    assert dsa.read_status(ws) == 0
    _check_pages(c, b, b.pages, b.scales)


def test_write_and_read_in_a_graph_on_another_stream():
    rng = np.random.default_rng(28)
    b = Batch(rng, LENS["ragged"], 2, 128, 16, "mxfp8")
    c = b.cache(dsa)
    cu_q, cu_k, table = b.dev("cu_q"), b.dev("cu_k"), b.dev("table")
    x = torch.zeros((b.total_q, 2, 128), device="cuda")
    out = dsa.cache_read(c, cu_k, table, b.total_k)
    ws = dsa.cache_workspace()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        dsa.cache_write(c, x, x, cu_q, cu_k, table, ws=ws)
        dsa.cache_read(c, cu_k, table, b.total_k, out=out, ws=ws)
    for seed in (1, 2):
        a = np.random.default_rng(seed).standard_normal((b.total_q, 2, 128)).astype(np.float32)
        x.copy_(dev(a))
        g.replay()
        torch.cuda.synchronize()
        st, sc = quantise(a.astype(np.float64), "mxfp8")
        rows = b.rows["k"].copy()
        for d, (t, n) in enumerate(b.lens):
            rows[b.cu_k[d] + n - t:b.cu_k[d] + n] = values(st, sc, "mxfp8")[b.cu_q[d]:b.cu_q[d] + t]
        np.testing.assert_array_equal(values(host(out[0]), host(out[1]), "mxfp8"), rows)
        assert dsa.read_status(ws) == 0
