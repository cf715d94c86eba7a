"""Host-side checks of the paged-cache entry points: nothing here reaches a GPU."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_attention_indexer_dsa_gb300 as dsa
from sparse_attention_indexer_dsa_gb300 import _abi, build_lib
from tests.paged_ref import Batch, quantise, values

P = ctypes.c_void_p
A = P(4096)
WS = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return _abi.load()


def _write(lib, **kw):
    a = dict(k=A, k_stride=0, k_scale=None, v=A, v_stride=0, v_scale=None, in_dtype=1, rule=0, cu_q=A, cu_k=A, seqs=1,
             total_q=4, table=A, max_pages=4, kp=A, kps=A, vp=A, vps=A, pages=8, page=16, kv=2, D=128, prec=1, ws=A,
             ws_bytes=WS, stream=None)
    a.update(kw)
    return lib.dsa_idx_cache_write(*a.values())


def _read(lib, **kw):
    a = dict(kp=A, kps=A, vp=A, vps=A, pages=8, page=16, kv=2, D=128, prec=1, table=A, max_pages=4, cu_k=A, seqs=1,
             total_k=4, deq=0, k=A, ks=A, v=A, vs=A, ws=A, ws_bytes=WS, stream=None)
    a.update(kw)
    return lib.dsa_idx_cache_read(*a.values())


def _attend(lib, **kw):
    a = dict(q=A, q_stride=0, kp=A, kps=A, vp=A, vps=A, pages=8, page=16, H=16, kv=2, D=128, prec=1, table=A, max_pages=4,
             cu_q=A, cu_k=A, seqs=1, total_q=4, max_q=4, max_k=4, scale=1.0, idx=None, len=None, W=0, out=A, lse=None,
             ws=A, ws_bytes=WS, stream=None)
    a.update(kw)
    return lib.dsa_idx_paged_attention(*a.values())


SHARED = [
    (dict(kp=None), 1), (dict(table=None), 1), (dict(cu_k=None), 1), (dict(prec=3), 1), (dict(D=96), 2),
    (dict(pages=0), 1), (dict(kv=0), 1), (dict(max_pages=0), 1), (dict(seqs=0), 1), (dict(page=12), 2),
    (dict(page=4), 2), (dict(page=2048), 2), (dict(pages=1 << 30), 2), (dict(kp=P(4104)), 1), (dict(kps=None), 1),
    (dict(vps=None), 1), (dict(kps=P(4097)), 1), (dict(ws=None), 4), (dict(ws_bytes=100), 4), (dict(ws=P(4112)), 1),
]


@pytest.mark.parametrize("call", [_write, _read, _attend])
@pytest.mark.parametrize("kw,code", SHARED)
def test_refusals_of_every_entry_point(lib, call, kw, code):
    assert call(lib, **kw) == code
    assert lib.dsa_idx_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), 1), (dict(cu_q=None), 1), (dict(v=None), 1), (dict(vp=None), 1), (dict(total_q=-1), 1),
    (dict(total_q=1 << 29), 2), (dict(rule=2), 1), (dict(in_dtype=3), 1), (dict(in_dtype=2), 1),
    (dict(in_dtype=2, k_scale=A), 1), (dict(k=P(4104)), 1), (dict(v=P(4104)), 1), (dict(k_stride=255), 1),
    (dict(k_stride=260), 1), (dict(v_stride=260), 1),
])
def test_write_refusals(lib, kw, code):
    assert _write(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), 1), (dict(vp=None, vps=None), 1), (dict(total_k=-1), 1), (dict(total_k=1 << 29), 2),
    (dict(ks=None), 1), (dict(vs=None), 1), (dict(k=P(4104)), 1), (dict(v=P(4104)), 1),
])
def test_read_refusals(lib, kw, code):
    assert _read(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(vp=None, vps=None), 1), (dict(cu_q=None), 1), (dict(total_q=-1), 1),
    (dict(max_q=-1), 1), (dict(max_k=-1), 1), (dict(H=0), 2), (dict(H=15), 2), (dict(H=258), 2),
    (dict(total_q=1 << 27), 2), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(idx=A, W=0), 1), (dict(W=4), 1), (dict(len=A), 1), (dict(q=P(4104)), 1), (dict(out=P(4104)), 1),
    (dict(q_stride=2047), 1), (dict(q_stride=2052), 1),
])
def test_attention_refusals(lib, kw, code):
    assert _attend(lib, **kw) == code


def test_workspace_sizes(lib):
    assert lib.dsa_idx_cache_workspace_size() == _abi.DSA_CACHE_WS_BYTES
    size = lib.dsa_idx_attention_workspace_size
    assert size(4, 1, 4, 16, 2, 128, 0) >= _abi.DSA_CACHE_WS_BYTES
    for bad in ((-1, 1, 4, 16, 2, 128, 0), (4, 0, 4, 16, 2, 128, 0), (4, 1, -1, 16, 2, 128, 0), (4, 1, 4, 0, 2, 128, 0),
                (4, 1, 4, 16, 0, 128, 0), (4, 1, 4, 15, 2, 128, 0), (4, 1, 4, 16, 2, 128, -1)):
        assert size(*bad) == 0


def test_cache_handle_checks():
    k = torch.zeros((2, 1, 16, 64), dtype=torch.uint8)
    s2, s1 = torch.zeros((2, 1, 16, 2), dtype=torch.uint8), torch.zeros((2, 1, 16, 1), dtype=torch.uint8)
    c = dsa.PagedCache(k, s2, None, None, "mxfp8")
    assert (c.num_pages, c.n_kv_heads, c.page_size, c.head_dim) == (2, 1, 16, 64)
    assert dsa.PagedCache(k, s1, k, s1, dsa.DSA_PREC_FP8).prec == "fp8"
    for bad in ((k, None, None, None, "mxfp8"), (k, s1, None, None, "mxfp8"), (k, s2, k, None, "mxfp8"),
                (k, s2, k[:1], s2, "mxfp8"), (k.transpose(0, 2), s2, None, None, "mxfp8"),
                (k.to(torch.bfloat16), s2, None, None, "bf16"), (k, None, None, None, "bf16"), (k[0], s2, None, None, "mxfp8")):
        with pytest.raises(ValueError):
            dsa.PagedCache(*bad)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):                       # not on a GPU
        dsa.cache_read(c, cu, torch.zeros((1, 2), dtype=torch.int32), 0)


def test_reference_forms_agree_with_themselves():
    """The tests' plain forms: stored rows decode to what was quantised, within the format's half step."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 2, 64))
    for prec, half in (("bf16", 2.0 ** -8), ("mxfp8", 2.0 ** -4), ("fp8", 2.0 ** -4)):
        st, sc = quantise(x, prec)
        top = np.abs(x).max(-1, keepdims=True)
        assert (np.abs(values(st, sc, prec) - x) <= half * np.abs(x) + 2.0 ** -10 * half * top * 2).all()
    b = Batch(rng, [(2, 5), (0, 3), (1, 17)], 2, 64, 8, "fp8")
    for d, (_, s) in enumerate(b.lens):
        for pos in range(s):
            pg = b.table[d, pos // 8]
            got = values(b.pages["v"][pg, :, pos % 8], b.scales["v"][pg, :, pos % 8], "fp8")
            np.testing.assert_array_equal(got, b.rows["v"][b.cu_k[d] + pos])


@pytest.mark.parametrize("kw", [dict(max_k=(1 << 30) + 1), dict(idx=A, W=(1 << 30) + 1), dict(total_q=1 << 26)])
def test_attention_counts_in_32_bits(lib, kw):
    assert _attend(lib, **kw) == 2


def test_an_empty_list_tensor_is_no_error(lib):
    """total_q = 0: a list of no rows has no address (what is left to fail here is the missing device)."""
    assert _attend(lib, total_q=0, q=None, out=None, idx=None, W=4) not in (1, 2, 4)
    assert _attend(lib, total_q=0, q=None, out=None, idx=None, W=-1) == 1
    assert _attend(lib, total_q=4, idx=None, W=4) == 1


def test_a_workspace_serves_smaller_calls(lib):
    rng = np.random.default_rng(7)
    size = lib.dsa_idx_attention_workspace_size
    for _ in range(300):
        kv, group, D = int(rng.integers(1, 9)), int(rng.integers(1, 129)), int(rng.choice([64, 128]))
        W = int(rng.choice([0, 0, 64, 2048]))
        total = [int(2 ** rng.uniform(0, 16)) for _ in range(2)]
        seqs = [int(2 ** rng.uniform(0, 9)) for _ in range(2)]
        mq = [int(2 ** rng.uniform(0, 14)) for _ in range(2)]
        n = size(max(total), max(seqs), max(mq), kv * group, kv, D, W)
        for total_q, s, q in ((total[0], seqs[0], mq[0]), (max(total), max(seqs), max(mq)), (min(total), max(seqs), 1)):
            for prec in (0, 1, 2):
                code = _attend(lib, H=kv * group, kv=kv, D=D, prec=prec, seqs=s, total_q=total_q, max_q=q, max_k=1 << 20,
                               idx=A if W else None, W=W, ws_bytes=n)
                assert code not in (1, 2, 4), (kv, group, D, W, total_q, s, q, prec)
