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
