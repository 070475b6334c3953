"""Arguments that the binding refuses, or passes on unchanged, without a GPU."""

import ctypes

import pytest
import torch

import long_context_sparse_cca_b200 as cca

BF, F16 = torch.bfloat16, torch.float16


class _Lib:
    """Every call succeeds; its arguments are kept."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return lambda *a: 4096
        return lambda *a: self.calls.append((name, a)) or 0


@pytest.fixture
def lib(monkeypatch):
    """CPU tensors in place of CUDA ones, and no library."""
    fake = _Lib()
    point = lambda t, *a: None if t is None else ctypes.c_void_p(t.data_ptr())  # noqa: E731
    monkeypatch.setattr(cca, "lib", lambda: fake)
    for name in ("_dev", "_lens"):
        monkeypatch.setattr(cca, name, point)
    monkeypatch.setattr(cca, "_here", lambda t, name, dev: t.data_ptr())
    monkeypatch.setattr(cca, "_device", lambda t, name: 0)
    monkeypatch.setattr(cca, "_stream", lambda s: None)
    monkeypatch.setattr(cca, "_raw_stream", lambda s, dev: 0)
    return fake


def _bf(*shape):
    return torch.zeros(shape, dtype=BF)


def _cache():
    return cca.Cache(3, 4, 2, 64, 16, 64, core_cap=8, device="cpu")


def _paged(**kw):
    a = dict(B=3, Hq=4, Hkv=2, d=64, g=16, w=64, page=16, core_pages=8, raw_pages=16, max_len=200,
             device="cpu")
    return cca.PagedCache(**{**a, **kw})


def _with_workspace():
    qt, kt = _bf(3, 4, 64), _bf(3, 2, 64)
    q, k, core = _bf(1, 4, 96, 64), _bf(1, 2, 96, 64), torch.zeros((1, 2, 6, 64), dtype=F16)
    lens, lse = torch.zeros(3, dtype=torch.int64), torch.zeros((1, 4, 96))
    i32 = torch.zeros(3, dtype=torch.int32)
    return {
        "cca_attn_backward": lambda ws: cca.cca_attn_backward(q, k, k, core, core, q, lse, q, 16, 64,
                                                              workspace=ws),
        "cca_attn_decode": lambda ws: cca.cca_attn_decode(_cache(), qt, workspace=ws),
        "cca_decode_step": lambda ws: cca.cca_decode_step(_cache(), qt, kt, kt, workspace=ws),
        "cca_attn_decode_rows": lambda ws: cca.cca_attn_decode_rows(_cache(), lens, qt,
                                                                    workspace=ws),
        "cca_attn_prefill_packed": lambda ws: cca.cca_attn_prefill_packed(
            q[0], k[0], k[0], core[0], core[0], torch.tensor([0, 96], dtype=torch.int32), 16, 64,
            workspace=ws),
        "cca_attn_decode_paged": lambda ws: cca.cca_attn_decode_paged(_paged(), qt, workspace=ws),
        "cca_paged_step": lambda ws: cca.cca_paged_step(_paged(), qt, kt, kt, workspace=ws),
        "cca_paged_fork": lambda ws: cca.cca_paged_fork(_paged(), i32, workspace=ws),
        "cca_paged_compact": lambda ws: cca.cca_paged_compact(_paged(), workspace=ws),
    }


CALLS = ["cca_attn_backward", "cca_attn_decode", "cca_decode_step", "cca_attn_decode_rows",
         "cca_attn_prefill_packed", "cca_attn_decode_paged", "cca_paged_step", "cca_paged_fork",
         "cca_paged_compact"]


@pytest.mark.parametrize("name", CALLS)
def test_workspace_without_its_bytes_is_refused(lib, name):
    """An expanded tensor says a million elements and has one."""
    call = _with_workspace()[name]
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20),
               torch.zeros(1 << 14, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            call(ws)
    with pytest.raises(ValueError, match="CUDA"):
        call(torch.zeros(1 << 14, dtype=torch.uint8))


class _Ws:
    """A contiguous CUDA tensor of 64 floats."""
    is_cuda = True

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def numel(self):
        return 64

    def element_size(self):
        return 4


def test_workspace_size_is_in_bytes():
    at, n = cca._workspace(_Ws())
    assert (at.value, n) == (4096, 256)


BIG = 1 << 32  # what ctypes would pass as 0


def _numbers():
    q, k, core = _bf(4, 96, 64), _bf(2, 96, 64), torch.zeros((2, 6, 64), dtype=F16)
    cu, rows = torch.tensor([0, 96], dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    qt, kt = _bf(3, 4, 64), _bf(3, 2, 64)
    q4, k4, c4 = q[None], k[None], core[None]
    return {
        "window of prompts": lambda x: cca.cca_attn_prefill_packed(q, k, k, core, core, cu, 16, x),
        "window of a paged cache": lambda x: _paged(w=x),
        "heads of a paged cache": lambda x: _paged(Hq=x),
        "layer of a fill": lambda x: cca.cca_paged_fill(_paged(), k, k, core, core, cu, rows,
                                                        layer=x),
        "layer of a step": lambda x: cca.cca_paged_step(_paged(), qt, kt, kt, layer=x),
        "layer of an attention": lambda x: cca.cca_attn_decode_paged(_paged(), qt, layer=x),
        "tokens": lambda x: cca.cca_paged_reserve(_paged(), x << 32),
        "window of a prompt": lambda x: cca.cca_attn_prefill(q4, k4, k4, c4, c4, 16, x),
        "window of a cache": lambda x: cca.Cache(3, 4, 2, 64, 16, x, 8, tail_cap=80, device="cpu"),
    }


@pytest.mark.parametrize("name", ["window of prompts", "window of a paged cache",
                                  "heads of a paged cache", "layer of a fill", "layer of a step",
                                  "layer of an attention", "tokens", "window of a prompt",
                                  "window of a cache"])
def test_numbers_beyond_the_librarys_are_refused(lib, monkeypatch, name):
    monkeypatch.setattr(cca, "_workspace", lambda t: (0, t.numel()))
    with pytest.raises(ValueError, match="does not fit"):
        _numbers()[name](BIG)
    assert not [c for c in lib.calls if not c[0].endswith("bytes")]


def test_int():
    assert [cca._int(x, "x") for x in (0, -1, 2**31 - 1, -2**31)] == [0, -1, 2**31 - 1, -2**31]
    assert cca._int(2**40, "x", 64) == 2**40
    for x in (2**31, -2**31 - 1, 1 << 80):
        with pytest.raises(ValueError):
            cca._int(x, "x")
