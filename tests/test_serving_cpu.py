"""Packed prompts and the paged cache without a GPU: what the C ABI and the
binding refuse before any launch, the page-upkeep model's own invariants
under random calls (it is the GPU tests' oracle), and the barrier protocol
of the packed attention kernel."""

import ctypes
import os
import random
import re

import numpy as np
import pytest

import long_context_sparse_cca_b200 as cca
import protocol_models as pm
from long_context_sparse_cca_b200 import build as cca_build
from serving_model import PagedModel, window_start

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # aligned, never dereferenced: every call below fails its checks
FAR = 1 << 24   # buffers this far apart do not overlap
P = ctypes.c_void_p
BAD, NOT_HERE = cca.CCA_ERR_INVALID_ARG, cca.CCA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    cca_build.build()
    return cca.lib()


def _at(i):
    return FAKE + i * FAR


def _rows(i, total=300, d=128, row=None, head=None, data=None):
    return cca._RowsStruct(_at(i) if data is None else data, d if row is None else row,
                           total * d if head is None else head)


def _pool(L, q=None, k=None, v=None, Kc=_at(4), Vc=_at(5), S=2, Hq=4, Hkv=2, total=300, d=128,
          g=16, cu=_at(6)):
    return L.cca_pool_packed(q or _rows(1), k or _rows(2), v or _rows(3), P(cu), P(Kc), P(Vc), S,
                             Hq, Hkv, total, d, g, None)


def test_pool_packed_refusals(L):
    assert _pool(L, S=0) == BAD
    assert _pool(L, S=8193) == NOT_HERE
    assert _pool(L, cu=0) == BAD
    assert _pool(L, cu=_at(6) + 2) == BAD
    assert _pool(L, Hq=3) == BAD
    assert _pool(L, d=96) == NOT_HERE
    assert _pool(L, total=-1) == BAD
    assert _pool(L, g=257) == NOT_HERE
    assert _pool(L, q=_rows(1, data=0)) == BAD
    assert _pool(L, k=_rows(2, data=_at(2) + 2)) == BAD   # 16-byte alignment
    assert _pool(L, k=_rows(2, row=120)) == BAD           # rows that overlap
    assert _pool(L, k=_rows(2, row=130)) == BAD           # a stride of 260 bytes
    assert _pool(L, v=_rows(3, head=0)) == BAD            # a broadcast head
    assert _pool(L, v=_rows(3, head=300 * 128 + 4)) == BAD
    assert _pool(L, q=_rows(1, row=1 << 39)) == BAD       # beyond a tensor map's strides
    assert _pool(L, Kc=0) == BAD
    assert _pool(L, Kc=_at(2)) == BAD                     # output on an input
    assert _pool(L, Kc=_at(2) + 256 * 301) == BAD         # ... on its second head
    assert _pool(L, Vc=_at(4)) == BAD                     # outputs on one another
    assert _pool(L, Hq=50, Hkv=2, S=8192, g=256) == NOT_HERE  # beyond shared memory
    # nothing to pool: no complete group fits
    assert _pool(L, q=_rows(1, data=0), total=15, Kc=0, Vc=0) == cca.CCA_OK


def _attn(L, q=None, k=None, v=None, o=None, Kc=_at(4), Vc=_at(5), S=2, Hq=4, Hkv=2, total=300,
          d=128, g=16, w=64, cu=_at(6), dt=0, ws=_at(9), n=None):  # S = 2: no workspace
    n = L.cca_packed_workspace_bytes(S, total) if n is None else n
    return L.cca_attn_prefill_packed(q or _rows(1), k or _rows(2), v or _rows(3), P(Kc), P(Vc),
                                     P(cu), o or _rows(7), dt, S, Hq, Hkv, total, d, g, w, P(ws),
                                     n, None)


def test_attn_prefill_packed_refusals(L):
    assert _attn(L, S=0) == BAD
    assert _attn(L, cu=0) == BAD
    assert _attn(L, dt=2) == BAD
    assert _attn(L, w=-1) == BAD
    assert _attn(L, d=32) == NOT_HERE
    assert _attn(L, Kc=0) == BAD                          # w < total needs the core rows
    assert _attn(L, Vc=_at(5) + 8) == BAD
    assert _attn(L, q=_rows(1, row=132)) == BAD
    assert _attn(L, o=_rows(7, data=_at(7) + 16)) == BAD  # 32-byte stores
    assert _attn(L, o=_rows(7, row=136)) == BAD           # output strides: multiples of 16
    assert _attn(L, o=_rows(7, head=128)) == BAD          # heads on one another
    assert _attn(L, o=_rows(7, row=128, head=256)) == BAD
    assert _attn(L, o=_rows(1)) == BAD                    # in place of Q
    assert _attn(L, o=_rows(4)) == BAD                    # on the core rows
    assert _attn(L, S=65, ws=_at(9) + 128) == BAD
    assert _attn(L, S=65, ws=0) == BAD
    assert _attn(L, S=65, n=L.cca_packed_workspace_bytes(65, 300) - 1) == BAD
    assert _attn(L, S=65, ws=_at(7)) == BAD               # workspace on the output
    assert _attn(L, S=65, ws=_at(6)) == BAD               # ... on the offsets
    assert _attn(L, total=0, q=_rows(1, data=0), o=_rows(7, data=0), Kc=0, ws=0) == cca.CCA_OK


def test_packed_workspace_bytes(L):
    size = L.cca_packed_workspace_bytes
    assert size(0, 100) == size(8193, 100) == size(1, -1) == 0
    # none while each CTA orders the blocks by itself
    assert size(1, 0) == size(64, 192 * 256 + 255) == 0
    assert size(65, 0) > 0 and size(64, 193 * 256) > 0
    assert 0 < size(1, 100000) < size(8192, 100000)
    # then 16 bytes for every block that S sequences of `total` rows can have
    for lens in ([1] * 100, [257, 1, 0, 300] * 20, [0] * 70, [512, 511, 513] * 50, [70000, 3]):
        blocks = sum(-(-n // 256) for n in lens)
        assert size(len(lens), sum(lens)) >= 256 + 16 * blocks


def _paged(**kw):
    names = ("k_core", "v_core", "k_raw", "v_raw", "core_table", "raw_table", "core_ref",
             "raw_ref", "lens")
    a = {n: _at(20 + i) for i, n in enumerate(names)}
    a.update(layers=2, B=4, Hq=4, Hkv=2, d=128, g=16, w=64, page=16, core_cols=2, raw_cols=32,
             core_pages=8, raw_pages=40)
    a.update(kw)
    return cca._PagedStruct(*(a[n] for n, _ in cca._PagedStruct._fields_))


BAD_CACHES = [
    (dict(layers=0), BAD), (dict(B=0), BAD), (dict(B=4097), NOT_HERE), (dict(Hq=3), BAD),
    (dict(Hq=64), NOT_HERE), (dict(d=96), NOT_HERE), (dict(g=0), BAD), (dict(g=257), NOT_HERE),
    (dict(w=-1), BAD), (dict(page=24), BAD), (dict(page=0), BAD), (dict(page=8), NOT_HERE),
    (dict(page=2048), NOT_HERE), (dict(raw_cols=1 << 21, page=1024), NOT_HERE),
    (dict(raw_cols=0), BAD), (dict(raw_pages=0), BAD),
    (dict(core_cols=0), BAD), (dict(core_pages=0), BAD), (dict(core_cols=-1), BAD),
    (dict(core_cols=0, core_pages=0), BAD),  # a window that ends needs core rows
    (dict(k_raw=0), BAD), (dict(v_core=_at(21) + 8), BAD), (dict(lens=_at(28) + 4), BAD),
    (dict(raw_table=0), BAD), (dict(core_ref=_at(26) + 2), BAD)]


@pytest.mark.parametrize("change,want", BAD_CACHES, ids=[str(c[0]) for c in BAD_CACHES])
def test_paged_cache_refusals(L, change, want):
    """Every paged call refuses an invalid cache, and says 0 for its workspace."""
    c = ctypes.byref(_paged(**change))
    ws = (P(_at(40)), 1 << 20)
    assert L.cca_paged_workspace_bytes(c) == 0
    assert L.cca_paged_reserve(c, None, 1, None) == want
    assert L.cca_paged_fill(c, 0, _rows(1), _rows(2), P(_at(4)), P(_at(5)), P(_at(6)), P(_at(7)),
                            2, 300, None) == want
    assert L.cca_attn_decode_paged(c, 0, P(_at(1)), P(_at(2)), 0, *ws, None) == want
    assert L.cca_paged_step(c, 0, P(_at(1)), P(_at(2)), P(_at(3)), P(_at(4)), 0, *ws, None) == want
    assert L.cca_paged_fork(c, P(_at(1)), *ws, None) == want
    assert L.cca_paged_compact(c, P(_at(1)), *ws, None) == want


def test_paged_call_refusals(L):
    c = ctypes.byref(_paged())
    n = L.cca_paged_workspace_bytes(c)
    assert n > 0
    # a cache of plain causal attention needs no core buffers
    plain = _paged(k_core=0, v_core=0, core_table=0, core_ref=0, core_cols=0, core_pages=0, w=512)
    assert L.cca_paged_workspace_bytes(ctypes.byref(plain)) > 0
    assert L.cca_paged_reserve(c, None, -1, None) == BAD
    assert L.cca_paged_reserve(c, P(_at(1) + 4), 0, None) == BAD

    def fill(layer=0, k=None, Kc=_at(4), cu=_at(6), rows=_at(7), S=2, total=300):
        return L.cca_paged_fill(c, layer, k or _rows(1), _rows(2), P(Kc), P(_at(5)), P(cu),
                                P(rows), S, total, None)
    assert fill(layer=2) == BAD and fill(layer=-1) == BAD
    assert fill(rows=0) == BAD and fill(cu=0) == BAD and fill(Kc=0) == BAD
    assert fill(k=_rows(1, row=4)) == BAD
    assert fill(S=0) == BAD and fill(S=8193) == NOT_HERE
    assert fill(k=_rows(1, data=_at(22))) == BAD          # prompts inside the pool
    assert fill(total=0, k=_rows(1, data=0)) == cca.CCA_OK

    def step(layer=0, q=_at(1), k=_at(2), v=_at(3), o=_at(4), dt=0, ws=_at(40), n=n):
        return L.cca_paged_step(c, layer, P(q), P(k), P(v), P(o), dt, P(ws), n, None)
    assert step(layer=2) == BAD and step(layer=-1) == BAD
    assert step(q=0) == BAD and step(k=_at(2) + 8) == BAD and step(v=0) == BAD
    assert step(o=0) == BAD and step(o=_at(1)) == BAD and step(o=_at(3)) == BAD
    assert step(dt=2) == BAD and step(ws=0) == BAD and step(ws=_at(40) + 64) == BAD
    assert step(n=n - 1) == BAD and step(o=_at(40)) == BAD

    def attn(q=_at(1), o=_at(4), dt=0, ws=_at(40), n=n, layer=0):
        return L.cca_attn_decode_paged(c, layer, P(q), P(o), dt, P(ws), n, None)
    assert attn(q=0) == BAD and attn(o=_at(1)) == BAD and attn(dt=5) == BAD
    assert attn(n=n - 1) == BAD and attn(ws=_at(40) + 8) == BAD and attn(layer=7) == BAD
    assert L.cca_paged_fork(c, None, P(_at(40)), n, None) == BAD
    assert L.cca_paged_fork(c, P(_at(1)), P(_at(40)), n - 1, None) == BAD
    assert L.cca_paged_compact(c, P(_at(1) + 4), P(_at(40)), n, None) == BAD
    assert L.cca_paged_compact(c, P(_at(1)), P(0), n, None) == BAD


def test_new_statuses():
    assert cca.status_string(cca.CCA_ERR_SEQLENS) == "CCA_ERR_SEQLENS"
    assert cca.status_string(cca.CCA_ERR_PAGE) == "CCA_ERR_PAGE"


def test_binding_checks():
    """Devices, types and shapes, before the library is called."""
    import torch
    q = torch.zeros((4, 300, 64), dtype=torch.bfloat16)
    k = torch.zeros((2, 300, 64), dtype=torch.bfloat16)
    cu = torch.tensor([0, 300], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        cca.cca_pool_packed(q, k, k, cu, 16)
    with pytest.raises(ValueError, match="CUDA"):
        cca.cca_attn_prefill_packed(q, k, k, None, None, cu, 16, 1 << 30)
    with pytest.raises(ValueError, match="Q must be a torch.bfloat16"):
        cca._rows(q.float(), "Q", (4, 300, 64), torch.bfloat16, 0)
    with pytest.raises(ValueError, match="rows of Q must be contiguous"):
        cca._rows(q.transpose(1, 2).contiguous().transpose(1, 2), "Q", (4, 300, 64),
                  torch.bfloat16, 0)
    with pytest.raises(ValueError, match="device 0"):
        cca._rows(q, "Q", (4, 300, 64), torch.bfloat16, 0)
    with pytest.raises(ValueError, match="int32"):
        cca._offsets(cu.long(), 0)
    with pytest.raises(ValueError, match="K must be"):
        cca._rows(k[:, :299], "K", (2, 300, 64), torch.bfloat16, 0)
    with pytest.raises(ValueError, match="heads, total, d"):
        cca._packed_shapes(q[None], k)
    with pytest.raises(ValueError):
        cca.PagedCache(0, 4, 2, 64, 16, 64, 16, 8, 16, 200, device="cpu")
    c = cca.PagedCache(3, 4, 2, 64, 16, 64, 16, 8, 16, 200, device="cpu")
    t = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        cca.cca_paged_fork(c, t)
    with pytest.raises(ValueError, match="CUDA"):
        cca.cca_paged_reserve(c, 1)
    with pytest.raises(ValueError):
        cca.PagedCache.from_tensors(c.core_table, c.raw_table, c.core_ref[1:], c.raw_ref, c.lens,
                                    *c.pools, Hq=4, g=16, w=64)
    with pytest.raises(ValueError):
        cca.PagedCache.from_tensors(c.core_table, c.raw_table, c.core_ref, c.raw_ref,
                                    c.lens.int(), *c.pools, Hq=4, g=16, w=64)


class _Fake:
    """A CUDA tensor of another device: enough for the binding's checks."""
    is_cuda, device = True, "cuda:1"

    def get_device(self):
        return 1


def test_binding_refuses_another_device(monkeypatch):
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="not the current device"):
        cca._device(_Fake(), "Q")
    with pytest.raises(ValueError, match="device 0"):
        cca._here(_Fake(), "K", 0)


def test_paged_cache_state_round_trip():
    import torch
    c = cca.PagedCache(3, 4, 2, 64, 16, 64, page=16, core_pages=8, raw_pages=16, max_len=200,
                       layers=2, device="cpu")
    assert (c.core_cols, c.raw_cols) == (1, 13)
    assert c.core_table.eq(-1).all() and c.raw_table.eq(-1).all()
    assert c.lens.data_ptr() % 8 == 0
    for t in c.pools:
        t.copy_(torch.randn(t.shape).to(t.dtype))
    c.lens.copy_(torch.tensor([5, 0, 77]))
    c.raw_ref[3] = 1
    d = cca.PagedCache.from_state_dict(c.state_dict(), device="cpu")
    assert torch.equal(c.tables, d.tables)
    assert (d.layers, d.B, d.Hq, d.Hkv, d.d, d.g, d.w, d.page) == (2, 3, 4, 2, 64, 16, 64, 16)
    for a, b in zip(c.pools, d.pools):
        assert torch.equal(a, b) and a.data_ptr() != b.data_ptr()
    assert c.nbytes() == sum(t.numel() * 2 for t in c.pools) + c.tables.numel() * 4


def test_struct_matches_header():
    """The binding's struct fields are the header's, in its order."""
    with open(os.path.join(ROOT, "include", "cca.h")) as f:
        text = f.read()
    body = re.search(r"typedef struct \{([^}]*)\} cca_paged_cache;", text).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = re.findall(r"\b(\w+)\s*[,;]", body.replace("*", " "))
    assert names == [n for n, _ in cca._PagedStruct._fields_]


# ---- the page-upkeep model

@pytest.mark.parametrize("seed", range(6))
def test_model_invariants(seed):
    rng = random.Random(seed)
    g, w, page = rng.choice([(16, 64, 16), (8, 250, 32), (4, 0, 16), (16, 64, 64)])
    m = PagedModel(6, g, w, page, core_pages=14, raw_pages=60, core_cols=5, raw_cols=60)
    label = 0
    for _ in range(60):
        what = rng.choice("rrrffc")
        if what == "r":
            m.reserve(rng.choice([1, [rng.choice([0, 1, rng.randint(0, 300)]) for _ in range(6)]]))
            for pool in (0, 1):  # every page in use holds something of its own
                for p in range(m.pages[pool]):
                    if m.ref[pool][p] and m.content[pool][p] is None:
                        m.content[pool][p] = label = label + 1
        elif what == "f":
            m.fork([rng.randint(-1, 5) for _ in range(6)])
        else:
            live = m.compact()
            assert [int((r[:n] > 0).sum()) for r, n in zip(m.ref, live)] == live
            assert all((r[n:] == 0).all() for r, n in zip(m.ref, live))
        m.check()


def test_model_fork_keeps_contents():
    m = PagedModel(4, 16, 64, 16, 8, 32, 4, 32)
    m.reserve([100, 0, 40, 0])
    m.content = [[f"{i}:{p}" for p in range(n)] for i, n in enumerate(m.pages)]
    before = [[m.content[i][p] for p in m.table[i][0] if p >= 0] for i in (0, 1)]
    m.fork([-1, 0, 2, 0])
    for b in (1, 3):
        assert [[m.content[i][p] for p in m.table[i][b] if p >= 0] for i in (0, 1)] == before
    assert m.lens.tolist() == [0, 100, 40, 100]
    assert window_start(99, 16, 64) == 32


# ---- the barrier protocol of the packed attention kernel

def _packed_items(lens, g, w, Hq, cta, grid, zigzag=True):
    """Blocks with the most key tiles first, as the kernel deals them:
    (local tiles, core tiles, [tiles that reach behind the sequence])."""
    blocks = sorted(((-(blk + 1), s, n, blk) for s, n in enumerate(lens)
                     for blk in range(-(-n // 256))))
    out = []
    for item in range(cta, len(blocks) * Hq, grid):
        k = item // grid
        if zigzag and k % 2 and (k + 1) * grid <= len(blocks) * Hq:
            item = (2 * k + 1) * grid - 1 - item
        _, _, n, blk = blocks[item // Hq]
        t0, tlast = blk * 256, min(blk * 256 + 255, n - 1)
        nl = (tlast - pm.ws_of(t0, g, w) + 128) // 128
        nc = (pm.ws_of(tlast, g, w) // g + 127) // 128
        lo = pm.ws_of(t0, g, w)
        behind = [lo + 128 * j + 127 > n - 1 for j in range(nl)]
        behind += [128 * j + 127 > n // g - 1 for j in range(nc)]
        out.append((nl, nc, behind))
    return out


def _producer(sim, items, KST=3, VST=2):
    """The packed kernel's TMA producer: a value tile that reaches behind its
    sequence lands on a barrier of the producer's own, and v_full completes
    with the zeros that are copied over it."""
    qc = kc = vc = raw = 0
    for nl, nc, behind in items:
        if qc > 0:
            yield from sim.wait("q_empty", qc - 1)
        sim.arrive("q_full")
        qc += 1
        for j in range(nl + nc):
            if kc >= KST:
                yield from sim.wait(f"k_empty{kc % KST}", kc // KST - 1)
            sim.arrive(f"k_full{kc % KST}")
            kc += 1
            if vc >= VST:
                yield from sim.wait(f"v_empty{vc % VST}", vc // VST - 1)
            if behind[j]:
                sim.arrive("raw")
                yield from sim.wait("raw", raw)
                raw += 1
                yield
            sim.arrive(f"v_full{vc % VST}")
            vc += 1


@pytest.mark.parametrize("case", [
    ([5, 1, 128, 77], 16, 64, 2), ([300, 0, 513, 2], 8, 40, 2), ([1], 16, 64, 1),
    ([2049, 100], 16, 1024, 4), ([257, 255, 256], 4, 0, 1), ([700], 1, 10, 3)], ids=str)
def test_packed_prefill_protocol(case):
    lens, g, w, Hq = case
    n_items = sum(-(-n // 256) for n in lens) * Hq
    for grid in sorted({1, 2, 3, min(n_items, 148)}):
        for cta in sorted({0, grid - 1, grid // 2}):
            items = _packed_items(lens, g, w, Hq, cta, grid, zigzag=grid != 2)
            for seed in range(2):
                sim = pm.Sim()
                roles = pm.prefill_roles(sim, [(nl, nc) for nl, nc, _ in items])
                sim.bar("raw")
                roles[0] = _producer(sim, items)
                sim.run(roles, seed)


def test_packed_blocks_places():
    """The attention kernel's list: every (sequence, block) pair finds a slot
    cu[s] // 256 + s + blk of its own within total // 256 + S."""
    rng = np.random.default_rng(5)
    for _ in range(200):
        S = int(rng.integers(1, 12))
        lens = rng.integers(0, rng.choice([2, 300, 2000]), size=S)
        lead, trail = rng.integers(0, 600, size=2)
        cu = lead + np.concatenate([[0], np.cumsum(lens)])
        slots = [int(cu[s]) // 256 + s + blk
                 for s in range(S) for blk in range(-(-int(lens[s]) // 256))]
        assert len(set(slots)) == len(slots)
        assert not slots or max(slots) < (int(cu[-1]) + int(trail)) // 256 + S
