"""The paged-cache entry points on the arguments at their limits: refused with an
error and nothing written, or taken with the documented result."""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_dsa_gb300 as dsa
from sparse_attention_indexer_dsa_gb300 import _abi
from tests.gpu_util import dev, host
from tests.paged_ref import Batch
from tests.test_gpu_paged_attention import _queries
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
