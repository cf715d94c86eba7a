"""Arguments that the norms with rotation and the operators of a bounded cache refuse, before anything reaches a GPU."""
import ctypes
import math

import pytest
import torch

import sparse_attention_indexer_dsa_gb300 as dsa
from sparse_attention_indexer_dsa_gb300 import _abi, build_lib, norms

A = 1 << 20          # an aligned address
BAD, UNSUP, WS = _abi.DSA_ERR_INVALID_ARG, _abi.DSA_ERR_UNSUPPORTED, _abi.DSA_ERR_WORKSPACE
REFUSED = (BAD, UNSUP, WS)


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return _abi.load()


def call(fn, base, **change):
    unknown = set(change) - set(base)
    assert not unknown, unknown
    return fn(*{**base, **change}.values())


NORM = dict(q=A, q_stride=0, k=A, k_stride=0, in_dtype=1, q_weight=A, k_weight=A, q_bias=None, k_bias=None, weight_dtype=0,
            norm=0, eps=1e-6, positions=A, total_tokens=5, n_heads=4, n_kv_heads=2, head_dim=128, rope_dim=64,
            rope_base=1e4, inv_freq=None, rope_interleaved=0, q_out=A, q_out_stride=0, k_out=A, k_out_stride=0,
            out_dtype=1, stream=None)
BACK = dict(dq_out=A, dq_out_stride=0, dk_out=A, dk_out_stride=0, grad_dtype=1, q=A, q_stride=0, k=A, k_stride=0, in_dtype=1,
            q_weight=A, k_weight=A, weight_dtype=0, norm=0, eps=1e-6, positions=A, total_tokens=5, n_heads=4, n_kv_heads=2,
            head_dim=128, rope_dim=64, rope_base=1e4, inv_freq=None, rope_interleaved=0, dq=A, dq_stride=0, dk=A, dk_stride=0,
            dq_weight=A, dk_weight=A, dq_bias=None, dk_bias=None, ws=A, ws_bytes=1 << 30, stream=None)
SHARED_NORM = [
    (BAD, dict(q=None)), (BAD, dict(k=None)), (BAD, dict(positions=None)), (BAD, dict(total_tokens=-1)), (BAD, dict(n_heads=0)),
    (BAD, dict(n_kv_heads=-1)), (UNSUP, dict(n_heads=1025)), (UNSUP, dict(n_kv_heads=2000)), (UNSUP, dict(head_dim=96)),
    (UNSUP, dict(head_dim=256)), (BAD, dict(in_dtype=2)), (BAD, dict(weight_dtype=7)), (BAD, dict(norm=2)), (BAD, dict(eps=-1e-9)),
    (BAD, dict(eps=math.nan)), (BAD, dict(eps=math.inf)), (BAD, dict(rope_dim=-8)), (BAD, dict(rope_dim=12)), (BAD, dict(rope_dim=136)),
    (BAD, dict(rope_base=0.0)), (BAD, dict(rope_base=-2.0)), (BAD, dict(rope_base=math.nan)), (BAD, dict(rope_base=math.inf)),
    (BAD, dict(q=A + 8)), (BAD, dict(k=A + 2)), (BAD, dict(q_weight=A + 4)), (BAD, dict(q_stride=511)), (BAD, dict(q_stride=516)),
    (BAD, dict(k_stride=255)), (BAD, dict(k_stride=-256)),
]


@pytest.mark.parametrize("want,change", SHARED_NORM + [
    (BAD, dict(q_out=None)), (BAD, dict(k_out=None)), (BAD, dict(q_out=A + 1)), (BAD, dict(out_dtype=2)), (BAD, dict(k_bias=A + 4)),
    (BAD, dict(q_out_stride=8)), (BAD, dict(k_out_stride=252))])
def test_norm_rope_refuses(lib, want, change):
    assert call(lib.dsa_idx_norm_rope, NORM, **change) == want, change


@pytest.mark.parametrize("want,change", SHARED_NORM + [
    (BAD, dict(dq=None)), (BAD, dict(dk=None)), (BAD, dict(dq_out=None)), (BAD, dict(dk_out=None)), (BAD, dict(grad_dtype=2)),
    (BAD, dict(dq_out=A + 8)), (BAD, dict(dk_out=A + 8)), (BAD, dict(dq_out_stride=100)), (BAD, dict(dk_out_stride=100)),
    (BAD, dict(dq_stride=100)), (BAD, dict(dq_bias=A)), (BAD, dict(dk_bias=A)), (WS, dict(ws=None)), (WS, dict(ws_bytes=100)), (BAD, dict(ws=A + 64))])
def test_norm_rope_backward_refuses(lib, want, change):
    assert call(lib.dsa_idx_norm_rope_backward, BACK, **change) == want, change


def test_frequencies_are_finite(lib):
    for f in (math.nan, math.inf):
        a = (ctypes.c_double * 32)(*([0.5] * 31 + [f]))
        assert call(lib.dsa_idx_norm_rope, NORM, inv_freq=ctypes.addressof(a)) == BAD


@pytest.mark.no_device
@pytest.mark.parametrize("change", [
    dict(), dict(n_kv_heads=0, k=None, k_out=None), dict(rope_dim=0, positions=None, rope_base=0.0), dict(q_weight=None, k_weight=None),
    dict(total_tokens=0, q=None, k=None, q_out=None, k_out=None, positions=None), dict(q_stride=520), dict(in_dtype=0, q_stride=516)])
def test_norm_rope_takes(lib, change):
    assert call(lib.dsa_idx_norm_rope, NORM, **change) not in REFUSED


WEIGH = dict(q=A, q_stride=0, lse=A, k_pages=A, k_page_scale=A, weights=A, num_pages=9, page_size=16, n_heads=8, n_kv_heads=2,
             head_dim=128, prec=1, page_table=A, max_pages=4, cu_q=A, cu_k=A, num_seqs=3, total_q=5, max_q=2, max_k=60, sm_scale=0.1,
             ws=A, ws_bytes=1 << 30, stream=None)
SELECT = dict(weights=A, num_pages=9, page_size=16, n_kv_heads=2, page_table=A, max_pages=4, cu_k=A, num_seqs=3, max_k=60, budget=20,
              sinks=2, recent=3, shared=0, kept=A, kept_len=A, ws=A, ws_bytes=8192, stream=None)
COMPACT = dict(k_pages=A, k_page_scale=A, v_pages=A, v_page_scale=A, weights=A, num_pages=9, page_size=16, n_kv_heads=2, head_dim=64,
               prec=2, page_table=A, max_pages=4, kept=A, kept_len=A, num_seqs=3, kept_heads=2, kept_width=20, ws=A, ws_bytes=8192,
               stream=None)
PAGES = [(BAD, dict(page_table=None)), (BAD, dict(num_pages=0)), (BAD, dict(max_pages=0)), (BAD, dict(num_seqs=0)), (BAD, dict(n_kv_heads=0)),
         (UNSUP, dict(page_size=24)), (UNSUP, dict(page_size=4)), (UNSUP, dict(page_size=2048)), (UNSUP, dict(num_pages=1 << 28)),
         (BAD, dict(weights=A + 4)), (WS, dict(ws=None)), (WS, dict(ws_bytes=8191)), (BAD, dict(ws=A + 16))]


@pytest.mark.parametrize("want,change", PAGES + [
    (BAD, dict(q=None)), (BAD, dict(lse=None)), (BAD, dict(k_pages=None)), (BAD, dict(k_page_scale=None)), (BAD, dict(weights=None)),
    (BAD, dict(cu_q=None)), (BAD, dict(cu_k=None)), (BAD, dict(total_q=-1)), (BAD, dict(max_q=-1)), (BAD, dict(max_k=-1)),
    (UNSUP, dict(n_heads=9)), (UNSUP, dict(n_heads=258)), (UNSUP, dict(n_heads=0)), (UNSUP, dict(total_q=1 << 28)), (UNSUP, dict(max_k=(1 << 30) + 1)),
    (UNSUP, dict(head_dim=32)), (BAD, dict(prec=3)), (BAD, dict(sm_scale=-0.1)), (BAD, dict(sm_scale=math.nan)),
    (BAD, dict(sm_scale=math.inf)), (BAD, dict(q=A + 8)), (BAD, dict(q_stride=1000)), (BAD, dict(q_stride=1028))])
def test_cache_weigh_refuses(lib, want, change):
    assert call(lib.dsa_idx_cache_weigh, WEIGH, **change) == want, change


@pytest.mark.parametrize("want,change", PAGES + [
    (BAD, dict(weights=None)), (BAD, dict(cu_k=None)), (BAD, dict(kept=None)), (BAD, dict(kept_len=None)), (BAD, dict(budget=0)),
    (BAD, dict(max_k=-1)), (BAD, dict(sinks=-1)), (BAD, dict(recent=-1)), (BAD, dict(sinks=10, recent=11)),
    (BAD, dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1)), (BAD, dict(budget=(1 << 30) + 1)), (UNSUP, dict(num_seqs=1 << 29))])
def test_evict_select_refuses(lib, want, change):
    assert call(lib.dsa_idx_evict_select, SELECT, **change) == want, change


@pytest.mark.parametrize("want,change", PAGES + [
    (BAD, dict(k_pages=None)), (BAD, dict(k_page_scale=None)), (BAD, dict(v_page_scale=None)), (BAD, dict(kept=None)),
    (BAD, dict(kept_len=None)), (BAD, dict(kept_heads=3)), (BAD, dict(kept_heads=0)), (BAD, dict(kept_width=0)), (UNSUP, dict(head_dim=100)),
    (BAD, dict(k_pages=A + 8)), (BAD, dict(prec=-1)), (UNSUP, dict(num_seqs=1 << 29))])
def test_cache_compact_refuses(lib, want, change):
    assert call(lib.dsa_idx_cache_compact, COMPACT, **change) == want, change


@pytest.mark.no_device
def test_bounded_cache_takes(lib):
    assert call(lib.dsa_idx_cache_weigh, WEIGH) not in REFUSED
    assert call(lib.dsa_idx_cache_weigh, WEIGH, total_q=0, q=None, lse=None) not in REFUSED
    assert call(lib.dsa_idx_cache_weigh, WEIGH, prec=0, k_page_scale=None, q_stride=1032) not in REFUSED
    assert call(lib.dsa_idx_evict_select, SELECT, sinks=10, recent=10, shared=1) not in REFUSED
    assert call(lib.dsa_idx_cache_compact, COMPACT, v_pages=None, v_page_scale=None, weights=None, kept_heads=1) not in REFUSED


def test_workspace_sizes(lib):
    assert lib.dsa_idx_norm_rope_workspace_size(64) < lib.dsa_idx_norm_rope_workspace_size(128)
    assert lib.dsa_idx_norm_rope_workspace_size(96) == 0
    ok = (100, 3, 50, 8, 2, 128)
    assert lib.dsa_idx_weigh_workspace_size(*ok) >= 8192
    for i, v in ((0, -1), (1, 0), (2, -1), (3, 0), (3, 9), (3, 2 * 129), (4, 0), (5, 32)):
        assert lib.dsa_idx_weigh_workspace_size(*ok[:i], v, *ok[i + 1:]) == 0, (i, v)


def test_the_binding_checks_before_the_library():
    """What the binding itself refuses; CPU tensors stand in for what is not reached."""
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.norm_rope(x, x, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="tokens"):
        dsa.norm_rope(x[0], None, None)
    w = torch.zeros(3, 2, 16)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.evict_select(w, None, None, 4, 10)
    with pytest.raises(ValueError, match="weights must be"):
        dsa.evict_select(w[0], None, None, 4, 10)
    c = dsa.PagedCache(torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16), None, None, None, "bf16")
    with pytest.raises(ValueError, match="CUDA"):
        dsa.cache_compact(c, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.cache_weigh(c, w, x, x, None, None, None, 1, 1)
    assert dsa.paged_weights(c).shape == (3, 2, 16) and dsa.paged_weights(c).dtype == torch.float32
    with pytest.raises(ValueError):
        dsa.norm_rope_workspace(96)
    with pytest.raises(ValueError):
        dsa.weigh_workspace(1, 1, 1, 3, 2, 64)
    assert set(norms._DTYPE) == {torch.float32, torch.bfloat16}


@pytest.mark.parametrize("view", [
    lambda: torch.zeros((1, 4, 64)).expand(8, 4, 64),
    lambda: torch.zeros((4, 64)).expand(2, 4, 64),
    lambda: torch.zeros(64 * 32).as_strided((8, 4, 64), (64, 64, 1)),
    lambda: torch.zeros((8, 1, 64)).expand(8, 4, 64),
    lambda: torch.zeros((8, 64, 4)).transpose(1, 2),
    lambda: torch.zeros((1, 1, 64)).expand(5, 1, 64),
])
def test_tokens_that_share_memory_are_refused(view):
    with pytest.raises(ValueError):
        norms._rows(view(), "q")


def test_token_strides():
    base = torch.zeros((8, 6, 64))
    assert norms._rows(base, "q") == (base.data_ptr(), 0)
    assert norms._rows(base[:, 2:], "q") == (base[:, 2:].data_ptr(), 6 * 64)
    assert norms._rows(base[::2, 2:], "q") == (base[:, 2:].data_ptr(), 12 * 64)
    assert norms._rows(base[:1, 2:], "q") == (base[:, 2:].data_ptr(), 0)       # one token has no next one
    assert norms._rows(base[:0, 2:], "q")[1] == 0
    one = torch.zeros((8, 1, 128))[:, :, :64]
    assert norms._rows(one, "q") == (one.data_ptr(), 128)
    for shape, dt in (((8, 6, 64), torch.bfloat16), ((8, 5, 64), torch.float32)):
        with pytest.raises(ValueError, match="k must be"):
            norms._like(base, "k", shape, dt, base.device)


def test_outputs_are_packed(monkeypatch):
    from sparse_attention_indexer_dsa_gb300 import paged
    monkeypatch.setattr(paged, "_current", lambda: 0)
    monkeypatch.setattr(paged, "_strided", lambda shape, strides, dtype: torch.empty_strided(shape, strides, dtype=dtype))
    for shape in ((5,), (0,), (3, 4), (0, 2, 64), (7, 1, 128), (2, 3, 4, 5)):
        t = paged._empty(shape, torch.bfloat16, torch.device("cuda", 0))
        assert t.shape == shape and t.stride() == torch.empty(shape).stride() and t.dtype is torch.bfloat16
    assert paged._empty((2, 3), torch.int32, torch.device("cpu")).device.type == "cpu"   # another device: torch.empty
    monkeypatch.setattr(paged, "_strided", None)
    assert paged._empty((2, 3), torch.int32, torch.device("cpu")).shape == (2, 3)


@pytest.mark.parametrize("change", [dict(q_bias=A), dict(k_bias=A), dict(q_bias=A, k_bias=A)])
def test_an_rms_norm_takes_no_biases(lib, change):
    """The backward call has no gradient for them, so the forward call refuses them."""
    assert call(lib.dsa_idx_norm_rope, NORM, **change) == BAD
    assert b"bias" in lib.dsa_idx_last_error()


@pytest.mark.no_device
def test_a_layer_norm_takes_biases(lib):
    assert call(lib.dsa_idx_norm_rope, NORM, norm=1, q_bias=A, k_bias=A) not in REFUSED
    assert call(lib.dsa_idx_norm_rope_backward, BACK, norm=1, dq_bias=A, dk_bias=A) not in REFUSED


@pytest.mark.parametrize("other", [
    lambda: torch.zeros(1),                                             # other arguments
    lambda shape, strides, dtype: None,                                 # another result
    lambda shape, strides, dtype: torch.zeros(shape, dtype=torch.float64),
    lambda shape, strides, dtype: torch.zeros((*shape, 1), dtype=dtype),
])
def test_an_allocator_of_another_kind_is_left_alone(monkeypatch, other):
    """torch's own function behind torch.empty may change from one version to the next: outputs then come from
    torch.empty, from the first call on."""
    from sparse_attention_indexer_dsa_gb300 import paged
    cpu, calls = torch.device("cpu"), []

    def strange(*args):
        calls.append(args)
        return other(*args)
    monkeypatch.setattr(paged, "_current", lambda: cpu.index)
    monkeypatch.setattr(paged, "_strided", strange)
    for _ in range(3):
        t = paged._empty((3, 4, 64), torch.bfloat16, cpu)
        assert t.shape == (3, 4, 64) and t.dtype is torch.bfloat16 and t.is_contiguous()
    assert len(calls) == 1 and paged._strided is None


def test_who_watches_allocations_sees_outputs(monkeypatch):
    from torch.utils._python_dispatch import TorchDispatchMode

    from sparse_attention_indexer_dsa_gb300 import paged
    cpu, seen = torch.device("cpu"), []
    monkeypatch.setattr(paged, "_current", lambda: cpu.index)
    monkeypatch.setattr(paged, "_strided", lambda shape, strides, dtype: torch.zeros(shape, dtype=dtype))

    class Watch(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            seen.append(str(func))
            return func(*args, **(kwargs or {}))
    with Watch():
        paged._empty((3, 4), torch.bfloat16, cpu)
    assert any("empty" in s for s in seen)
    monkeypatch.setattr(paged, "_strided", lambda *a: pytest.fail("not under deterministic algorithms"))
    torch.use_deterministic_algorithms(True)
    try:
        t = paged._empty((3, 4), torch.float32, cpu)
        assert torch.isnan(t).all()       # torch fills what it allocates
    finally:
        torch.use_deterministic_algorithms(False)


def test_frequencies_have_a_bound(lib):
    """Beyond it an angle is not what its frequency says."""
    for f in (2.0 ** 49, -2.0 ** 49, 1.7e308, -1.7e308):
        a = (ctypes.c_double * 32)(*([0.5] * 31 + [f]))
        assert call(lib.dsa_idx_norm_rope, NORM, inv_freq=ctypes.addressof(a)) == BAD
    for base in (1e-300, 5e-324, 1e-20):
        assert call(lib.dsa_idx_norm_rope, NORM, rope_base=base) == BAD
        assert call(lib.dsa_idx_norm_rope_backward, BACK, rope_base=base) == BAD
        assert call(lib.dsa_idx_norm_rope, NORM, rope_base=base) == BAD      # and again


@pytest.mark.no_device
def test_frequencies_up_to_the_bound_are_taken(lib):
    a = (ctypes.c_double * 32)(*([0.5] * 30 + [2.0 ** 48, -2.0 ** 48]))
    assert call(lib.dsa_idx_norm_rope, NORM, inv_freq=ctypes.addressof(a)) not in REFUSED
    for base in (0.5, 1.0, 1e-14, 1e300):
        assert call(lib.dsa_idx_norm_rope, NORM, rope_base=base) not in REFUSED
    assert call(lib.dsa_idx_norm_rope, NORM, rope_dim=8, rope_base=1e-18) not in REFUSED


@pytest.mark.parametrize("change", [dict(budget=(1 << 32) + 4), dict(sinks=1 << 32), dict(recent=(1 << 32) + 1), dict(max_seqlen_k=1 << 32),
                                    dict(sinks=-1), dict(max_seqlen_k=1 << 31)])
def test_sizes_beyond_32_bits_are_refused(change):
    """What ctypes hands on is 32 bits: sinks of 2^32 would be none."""
    w = torch.zeros(3, 2, 16)
    with pytest.raises(ValueError, match="2.31"):
        dsa.evict_select(w, None, None, **{**dict(budget=4, max_seqlen_k=10), **change})


def test_a_rotation_beyond_32_bits_is_refused(monkeypatch):
    class Cuda(torch.Tensor):      # a CPU tensor that passes for one on the GPU
        is_cuda = True
    q = torch.zeros(4, 2, 64).as_subclass(Cuda)
    for dim in ((1 << 32) + 64, 1 << 31, -8):
        with pytest.raises(ValueError, match="multiple of 8"):
            norms._inputs(q, None, None, (None,) * 4, "rms", dim, None)
