"""The paged-cache entry points on the arguments at their limits: refused with an
error and nothing written, or taken with the documented result."""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_dsa_gb300 as dsa
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
