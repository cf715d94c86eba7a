"""Arguments of the paged-cache binding that the kernels must never see, and those
that they have to take: nothing here reaches a GPU."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import sparse_attention_indexer_dsa_gb300 as dsa
from sparse_attention_indexer_dsa_gb300 import _abi, paged
from tests.test_paged_host import A as _A
from tests.test_paged_host import _attend, _read, _write, lib  # noqa: F401

CPU = torch.device("cpu")


def _tokens(t, heads=4, head_dim=64):
    return paged._tokens(t, "k", CPU, (torch.bfloat16,), heads, head_dim)


def test_token_strides():
    """The stride handed on is one that the kernel can walk without leaving the tensor: 0 (packed) only
    where the tokens are packed."""
    base = torch.zeros((8, 6, 64), dtype=torch.bfloat16)
    t = base[:, :4].contiguous()
    assert _tokens(t) == (t.data_ptr(), 0)
    assert _tokens(base[:, 2:]) == (base[:, 2:].data_ptr(), 6 * 64)
    assert _tokens(base[:1, 2:]) == (base[:1, 2:].data_ptr(), 0)          # one token has no next one
    one = torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    assert _tokens(one.expand(1, 4, 64)) == (one.data_ptr(), 0)
    assert _tokens(base[:0, 2:])[1] == 0


@pytest.mark.parametrize("view", [
    lambda: torch.zeros((1, 4, 64), dtype=torch.bfloat16).expand(8, 4, 64),
    lambda: torch.zeros((4, 64), dtype=torch.bfloat16).expand(2, 4, 64),
    lambda: torch.zeros(64 * 32, dtype=torch.bfloat16).as_strided((8, 4, 64), (64, 64, 1)),
    lambda: torch.zeros((8, 1, 64), dtype=torch.bfloat16).expand(8, 4, 64),
    lambda: torch.zeros((8, 64, 4), dtype=torch.bfloat16).transpose(1, 2),
])
def test_tokens_that_share_memory_are_refused(view):
    with pytest.raises(ValueError):
        _tokens(view())


def test_one_head_expanded_over_tokens_is_refused():
    with pytest.raises(ValueError):
        _tokens(torch.zeros((1, 1, 64), dtype=torch.bfloat16).expand(5, 1, 64), heads=1)


@pytest.mark.no_device
@pytest.mark.parametrize("prec", [0, 1, 2])
@pytest.mark.parametrize("v", [True, False])
def test_no_tokens_have_no_addresses(lib, prec, v):  # noqa: F811
    """Empty tensors have no address, of rows, codes and scales alike: no argument is missing then (what
    is left to fail here is the missing device)."""
    refused = (_abi.DSA_ERR_INVALID_ARG, _abi.DSA_ERR_UNSUPPORTED, _abi.DSA_ERR_WORKSPACE)
    pages = {} if v else dict(vp=None, vps=None)
    for src in (_abi.DSA_DTYPE_F32, _abi.DSA_DTYPE_BF16, _abi.DSA_DTYPE_OPERAND):
        assert _write(lib, total_q=0, k=None, v=None, k_scale=None, v_scale=None, in_dtype=src, prec=prec, **pages) not in refused
    for deq in (0, 1):
        assert _read(lib, total_k=0, k=None, v=None, ks=None, vs=None, deq=deq, prec=prec, **pages) not in refused
    if prec:
        assert _write(lib, total_q=1, k_scale=None, in_dtype=_abi.DSA_DTYPE_OPERAND, prec=prec) == _abi.DSA_ERR_INVALID_ARG
        assert _read(lib, total_k=1, ks=None, prec=prec) == _abi.DSA_ERR_INVALID_ARG


def test_made_up_addresses_stay_off_a_gpu(monkeypatch):
    """Where there is a GPU, the collection skips every test that would hand a kernel a made-up address."""
    from tests import conftest

    class Item:
        def __init__(self, name, *keywords):
            self.originalname, self.keywords, self.marks = name, set(keywords), []

        def add_marker(self, m):
            self.marks.append(m)

    items = [Item(n) for n in sorted(conftest.MADE_UP_ADDRESSES)] + [Item("x", "no_device"), Item("y"), Item("z", "gpu")]
    monkeypatch.setattr(conftest, "gpu_available", lambda: True)
    conftest.pytest_collection_modifyitems(None, items)
    assert [len(i.marks) for i in items] == [1] * len(conftest.MADE_UP_ADDRESSES) + [1, 0, 0]
    from tests import test_abi, test_paged_host
    for n in conftest.MADE_UP_ADDRESSES:
        assert hasattr(test_abi, n) or hasattr(test_paged_host, n)


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38, float("inf"), -1e-45, float("nan")])
def test_scales_that_no_logit_takes(lib, scale):  # noqa: F811
    """sm_scale is multiplied by log2(e) on its way: what overflows there is refused as an infinity is."""
    assert _attend(lib, scale=scale) == _abi.DSA_ERR_INVALID_ARG


def test_the_package_is_imported_without_cuda_in_torch():
    """A torch built without CUDA has no such names in torch._C; the paged cache's handle still works there."""
    code = ("import torch\n"
            "for n in [n for n in vars(torch._C) if n.startswith('_cuda_')]: delattr(torch._C, n)\n"
            "import sparse_attention_indexer_dsa_gb300 as dsa\n"
            "k = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16)\n"
            "assert dsa.PagedCache(k, None, k, None).page_size == 16\n"
            "from sparse_attention_indexer_dsa_gb300 import paged\n"
            "assert callable(paged._stream) and callable(paged._current)\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_device_0_is_device_0(monkeypatch, lib):  # noqa: F811
    """A device given by its number is that device, number 0 too; None is the current one."""
    seen = []
    for name in ("empty", "zeros"):
        make = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, device, _make=make, **k: (seen.append(device), _make(*a, device="cpu", **k))[1])
    calls = (lambda d: dsa.paged_cache(2, 16, 1, 64, device=d).k, lambda d: dsa.cache_workspace(d),
             lambda d: dsa.attention_workspace(4, 1, 4, 16, 2, 128, device=d),
             lambda d: dsa.workspace(8, 1, 8, 64, 128, 16, device=d))
    for call in calls:
        for given, want in ((0, 0), (1, 1), ("cuda:0", "cuda:0"), (None, "cuda")):
            seen.clear()
            call(given)
            assert set(seen) == {want}, (given, seen)


def test_what_a_call_needs_is_within_what_every_smaller_call_needs(lib):  # noqa: F811
    rng = np.random.default_rng(8)
    every, one = lib.dsa_idx_attention_workspace_size, lib.dsa_idx_attention_call_workspace_size
    for _ in range(2000):
        kv, group, D = int(rng.integers(1, 9)), int(rng.integers(1, 129)), int(rng.choice([64, 128]))
        W, total, seqs, mq, mk = int(rng.choice([0, 0, 64, 2048])), *(int(2 ** rng.uniform(0, n)) for n in (16, 9, 14, 17))
        page, prec = int(rng.choice([8, 16, 64, 1024])), int(rng.integers(0, 3))
        need = one(total, seqs, mq, mk, kv * group, kv, D, page, prec, W)
        assert _abi.DSA_CACHE_WS_BYTES <= need <= every(total, seqs, mq, kv * group, kv, D, W)
        sizes = dict(H=kv * group, kv=kv, D=D, prec=prec, page=page, seqs=seqs, total_q=total, max_q=mq, max_k=mk, W=W,
                     idx=_A if W else None)
        assert _attend(lib, ws_bytes=need - 1, **sizes) == _abi.DSA_ERR_WORKSPACE
    assert one(4096, 1, 4096, 32768, 64, 8, 128, 64, 0, 0) == _abi.DSA_CACHE_WS_BYTES     # undivided pairs
    for bad in ((-1, 1, 4, 9, 16, 2, 128, 16, 0, 0), (4, 0, 4, 9, 16, 2, 128, 16, 0, 0), (4, 1, 4, -1, 16, 2, 128, 16, 0, 0),
                (4, 1, 4, 9, 15, 2, 128, 16, 0, 0), (4, 1, 4, 9, 16, 2, 96, 16, 0, 0), (4, 1, 4, 9, 16, 2, 128, 0, 0, 0)):
        assert one(*bad) == 0


@pytest.mark.parametrize("current", [0, 1])
def test_the_status_is_read_on_the_workspace_s_device(monkeypatch, current):
    """As the calls run on their tensors' device, whichever is the current one, so is their status read
    behind that device's stream."""
    class Ws:
        is_cuda, device = True, torch.device("cuda", 1)
        is_contiguous = staticmethod(lambda: True)
        data_ptr = staticmethod(lambda: 4096)

    class Lib:
        @staticmethod
        def dsa_idx_read_status(address, stream, out):
            seen.append((address, stream, now[-1]))
            out._obj.value = 5
            return 0

    class On:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            now.append(self.index)

        def __exit__(self, *a):
            now.pop()

    seen, now = [], [current]
    monkeypatch.setattr(_abi, "load", lambda: Lib)
    monkeypatch.setattr(paged, "_stream", lambda index: 100 + index)
    monkeypatch.setattr(paged, "_current", lambda: now[-1])
    monkeypatch.setattr(dsa, "_stream", lambda: 100 + now[-1])
    monkeypatch.setattr(torch.cuda, "device", On)
    assert dsa.read_status(Ws) == 5
    assert seen == [(4096, 101, 1)] and now == [current]


def test_a_handle_stays_what_was_checked():
    """The calls take sizes from the keys alone: values replaced by fewer pages would be read behind their end."""
    k = torch.zeros((4, 1, 16, 64), dtype=torch.uint8)
    sc = torch.zeros((4, 1, 16, 2), dtype=torch.uint8)
    c = dsa.PagedCache(k, sc, k.clone(), sc.clone(), dsa.DSA_PREC_MXFP8)
    assert c.prec == "mxfp8"
    for name, t in (("k", k[:2]), ("v", k[:2]), ("k_scale", sc[:2]), ("v_scale", None), ("prec", "fp8")):
        with pytest.raises(AttributeError):
            setattr(c, name, t)
