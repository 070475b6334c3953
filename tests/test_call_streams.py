"""Memory that the binding allocates for a call on ``stream``.

Outputs, hidden workspaces and the cache's own workspace come from the pool
of that stream.  From the current stream's pool, a block that the current
stream has freed, but is still working on, would be written at once; and one
freed after the call would be handed out while the call's work still runs.
"""

import contextlib
import ctypes

import numpy as np
import pytest
import torch
from torch.overrides import TorchFunctionMode

import long_context_sparse_cca_b200 as cca

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


class _Stream:
    cuda_stream = 77


class _Allocations(TorchFunctionMode):
    """The stream that is current at each allocation."""

    def __init__(self):
        super().__init__()
        self.current, self.seen = [None], []

    def __torch_function__(self, func, types, args=(), kwargs=None):
        if func.__name__ in ("empty", "zeros", "new_empty", "new_zeros", "empty_like"):
            self.seen.append(self.current[-1])
        return func(*args, **(kwargs or {}))

    @contextlib.contextmanager
    def on(self, stream):
        self.current.append(stream)
        yield
        self.current.pop()


class _Lib:
    """Every call succeeds, every workspace takes 4096 bytes."""

    def __getattr__(self, name):
        return lambda *a: 4096 if name.endswith("workspace_bytes") else 0


@pytest.fixture
def allocations(monkeypatch):
    """CPU tensors in place of CUDA ones, and no library."""
    seen = _Allocations()
    point = lambda t, *a: None if t is None else ctypes.c_void_p(t.data_ptr())  # noqa: E731
    monkeypatch.setattr(cca, "lib", _Lib)
    monkeypatch.setattr(cca, "_dev", point)
    monkeypatch.setattr(cca, "_lens", point)
    monkeypatch.setattr(cca, "_workspace", lambda t: (point(t), t.numel()))
    monkeypatch.setattr(cca, "_here", lambda t, name, dev: t.data_ptr())
    monkeypatch.setattr(cca, "_device", lambda t, name: 0)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda at, **kw: at)
    monkeypatch.setattr(torch.cuda, "stream", seen.on)
    return seen


def _bf(*shape):
    return torch.zeros(shape, dtype=BF)


def _prompt():
    q, k = _bf(1, 4, 96, 64), _bf(1, 2, 96, 64)
    core = torch.zeros((1, 2, 6, 64), dtype=F16)
    return q, k, core


def _packed():
    q, k = _bf(4, 96, 64), _bf(2, 96, 64)
    core = torch.zeros((2, 6, 64), dtype=F16)
    return q, k, core, torch.tensor([0, 90, 96], dtype=torch.int32)


def _cache():
    return cca.Cache(3, 4, 2, 64, 16, 64, core_cap=8, device="cpu")


def _paged():
    return cca.PagedCache(3, 4, 2, 64, 16, 64, 16, 8, 16, 200, device="cpu")


def _calls():
    q, k, core = _prompt()
    pq, pk, pcore, cu = _packed()
    o, lse = _bf(1, 4, 96, 64), torch.zeros((1, 4, 96))
    qt, kt = _bf(3, 4, 64), _bf(3, 2, 64)
    lens = torch.zeros(3, dtype=torch.int64)
    return {  # the call and how many tensors it allocates
        "pool": (lambda s: cca.cca_pool(q, k, k, 16, stream=s), 2),
        "prefill": (lambda s: cca.cca_attn_prefill(q, k, k, core, core, 16, 64, stream=s), 1),
        "lse": (lambda s: cca.cca_attn_prefill_lse(q, k, k, core, core, 16, 64, stream=s), 2),
        "backward": (lambda s: cca.cca_attn_backward(q, k, k, core, core, o, lse, o, 16, 64,
                                                     stream=s), 4),
        "lca": (lambda s: cca.cca_lca_pool(q, k, k, 16, 16, stream=s), 2),
        "decode": (lambda s, c=_cache(): cca.cca_attn_decode(c, qt, stream=s), 2),
        "step": (lambda s, c=_cache(): cca.cca_decode_step(c, qt, kt, kt, stream=s), 2),
        "rows": (lambda s, c=_cache(): cca.cca_attn_decode_rows(c, lens, qt, stream=s), 2),
        "noalloc": (lambda s, c=_cache(): cca.cca_attn_decode_noalloc(c, qt, stream=s), 1),
        "pool_packed": (lambda s: cca.cca_pool_packed(pq, pk, pk, cu, 16, stream=s), 1),
        "packed": (lambda s: cca.cca_attn_prefill_packed(pq, pk, pk, pcore, pcore, cu, 16, 64,
                                                         stream=s), 2),
        "packed_token_order": (lambda s: cca.cca_attn_prefill_packed(
            pq.transpose(0, 1).contiguous().transpose(0, 1), pk, pk, pcore, pcore, cu, 16, 64,
            stream=s), 2),
        "paged_decode": (lambda s, c=_paged(): cca.cca_attn_decode_paged(c, qt, stream=s), 1),
        "paged_step": (lambda s, c=_paged(): cca.cca_paged_step(c, qt, kt, kt, stream=s), 1),
        "compact": (lambda s, c=_paged(): cca.cca_paged_compact(c, stream=s), 1),
    }


@pytest.mark.parametrize("name", ["pool", "prefill", "lse", "backward", "lca", "decode", "step",
                                  "rows", "noalloc", "pool_packed", "packed",
                                  "packed_token_order", "paged_decode", "paged_step", "compact"])
def test_allocations_are_on_the_calls_stream(allocations, name):
    call, n = _calls()[name]
    with allocations:
        call(_Stream)
    assert allocations.seen == [_Stream.cuda_stream] * n


# ---- on the GPU: the current stream is behind, and still writes what it has freed


@pytest.mark.gpu
@pytest.mark.parametrize("S", [3, 70])  # without and with a workspace of the call's own
def test_freed_memory_of_a_stream_that_is_behind(S):
    """Blocks of the current stream's pool, freed while their writes are still
    queued, are not what a call on another stream takes."""
    from long_context_sparse_cca_b200 import build
    build.build()
    rng = np.random.default_rng(S)
    lens = rng.integers(1, 200, size=S)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    total = int(lens.sum())
    gen = torch.Generator(device="cuda").manual_seed(S)
    Q, K, V = (torch.randn((h, total, 64), generator=gen, device="cuda").to(BF) for h in (4, 2, 2))
    kc, vc = cca.cca_pool_packed(Q, K, V, cu, 16)
    want = cca.cca_attn_prefill_packed(Q, K, V, kc, vc, cu, 16, 64)
    side = torch.cuda.Stream()
    nbytes = [2 * 4 * total * 64, 2 * 2 * (total // 16) * 64 * 2,
              cca.cca_packed_workspace_bytes(S, total)]
    torch.cuda.synchronize()
    for _ in range(3):
        # a fresh pool for the side stream's blocks, and on the current stream
        # blocks of the sizes that the calls want, written late
        torch.cuda.empty_cache()
        torch.cuda._sleep(20_000_000)  # about 10 ms
        late = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in nbytes for _ in range(2)]
        for t in late:
            t.fill_(0x7f)
        del late, t
        core = cca.cca_pool_packed(Q, K, V, cu, 16, stream=side)
        got = cca.cca_attn_prefill_packed(Q, K, V, *core, cu, 16, 64, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(core[0], kc) and torch.equal(core[1], vc)
        assert torch.equal(got, want)
    assert cca.cca_device_status() == cca.CCA_OK


@pytest.mark.gpu
def test_core_rows_dropped_while_the_stream_reads_them():
    """The rows that only the call's arguments held go back to the side
    stream's pool: the current stream does not get them."""
    from long_context_sparse_cca_b200 import build
    build.build()
    gen = torch.Generator(device="cuda").manual_seed(1)
    Q, K, V = (torch.randn((h, 3000, 128), generator=gen, device="cuda").to(BF)
               for h in (8, 8, 8))
    cu = torch.tensor([0, 3000], dtype=torch.int32, device="cuda")
    kc, vc = cca.cca_pool_packed(Q, K, V, cu, 16)
    want = cca.cca_attn_prefill_packed(Q, K, V, kc, vc, cu, 16, 64)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = cca.cca_attn_prefill_packed(
            Q, K, V, *cca.cca_pool_packed(Q, K, V, cu, 16, stream=side), cu, 16, 64, stream=side)
        for _ in range(4):  # the current stream takes blocks of the rows' size, and writes them
            torch.empty((2, 8, 3000 // 16, 128), dtype=F16, device="cuda").fill_(9.0)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert cca.cca_device_status() == cca.CCA_OK
