"""A row that cca_paged_reserve refuses keeps not only its length and pages
but its tokens: the steps behind the refusal leave it as it is, and when
there is room again it goes on where it was."""

import ctypes

import numpy as np
import pytest

import long_context_sparse_cca_b200 as cca
import oracle
from gpu_util import assert_close, to_cuda
from long_context_sparse_cca_b200 import build as cca_build
from long_context_sparse_cca_b200 import synth
from serving_model import packed_inputs
from test_serving_cpu import BAD_CACHES, _at, _paged

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def built():
    cca_build.build()


@pytest.mark.parametrize("change,want", BAD_CACHES, ids=[str(c[0]) for c in BAD_CACHES])
def test_refuses_an_invalid_cache(built, change, want):
    assert cca.lib().cca_paged_reserve_held(ctypes.byref(_paged(**change)), None, 1, P(_at(40)),
                                            1 << 20, None) == want


def test_refusals(built):
    c, L = ctypes.byref(_paged()), cca.lib()
    n = L.cca_paged_workspace_bytes(c)
    for args in ((None, -1, P(_at(40)), n), (P(_at(1) + 4), 0, P(_at(40)), n),
                 (None, 1, P(0), n), (None, 1, P(_at(40) + 64), n), (None, 1, P(_at(40)), n - 1)):
        assert L.cca_paged_reserve_held(c, *args, None) == cca.CCA_ERR_INVALID_ARG


# ---- on the GPU

HQ, HKV, D, G, W, PAGE = 4, 2, 64, 16, 32, 16


class Loop:
    """Rows that take steps as long as there is room; each row's history is
    what it was granted."""

    def __init__(self, B, lens, core_pages, raw_pages, layers=2, max_len=400):
        import torch
        self.torch, self.layers = torch, layers
        self.c = cca.PagedCache(B, HQ, HKV, D, G, W, PAGE, core_pages, raw_pages, max_len=max_len,
                                layers=layers)
        n = torch.tensor(lens, dtype=torch.int64, device="cuda")
        cca.cca_paged_reserve(self.c, n)
        self.hist = []
        rows = torch.arange(B, dtype=torch.int32, device="cuda")
        for layer in range(layers):
            q, k, v, cu = packed_inputs(lens, HQ, HKV, D, 100 + layer)
            Q, K, V = (to_cuda(x) for x in (q, k, v))
            cu_d = torch.from_numpy(cu).cuda()
            Kc, Vc = cca.cca_pool_packed(Q, K, V, cu_d, G)
            cca.cca_paged_fill(self.c, K, V, Kc, Vc, cu_d, rows, layer=layer)
            self.hist.append([[x[:, cu[b]:cu[b + 1]] for x in (q, k, v)] for b in range(B)])
        assert cca.cca_device_status() == cca.CCA_OK
        self.inputs = [[torch.zeros((B, h, D), dtype=torch.bfloat16, device="cuda")
                        for h in (HQ, HKV, HKV)] for _ in range(layers)]
        self.seed = 1000

    def calls(self):
        cca.cca_paged_reserve(self.c, 1)
        return [cca.cca_paged_step(self.c, *x, layer=i, out_dtype=self.torch.float32)
                for i, x in enumerate(self.inputs)]

    def step(self, run=None):
        """One turn; returns which rows were granted a token."""
        torch, c = self.torch, self.c
        before = c.lens.tolist()
        new = []
        for x in self.inputs:
            self.seed += 10
            new.append([synth.random_bf16(tuple(t.shape), self.seed + i)
                        for i, t in enumerate(x)])
            for t, y in zip(x, new[-1]):
                t.copy_(to_cuda(y))
        tables = c.tables.clone()
        outs = run() if run else self.calls()
        status = cca.cca_device_status()
        granted = [a > b for a, b in zip(c.lens.tolist(), before)]
        refused = [n > 0 and not y for n, y in zip(before, granted)]
        assert status == (cca.CCA_ERR_CAPACITY if any(refused) else cca.CCA_OK)
        for layer, o in enumerate(outs):
            for b in range(c.B):
                if not granted[b]:
                    assert bool((o[b] == 0).all()), "a held or free row's output"
                    continue
                h = self.hist[layer][b] = [np.concatenate([x, y[b][:, None]], 1)
                                           for x, y in zip(self.hist[layer][b], new[layer])]
                self.check(layer, b, o[b], h)
        if not any(granted):
            assert torch.equal(c.tables, tables)
        return granted

    def check(self, layer, b, o, h):
        x = [synth.bf16_bits_to_f64(np.ascontiguousarray(y[None])) for y in h]
        n = x[0].shape[2]
        ref = oracle.prefill(*x, G, min(W, n), rows=[n - 1])[0, :, 0]
        assert_close(o, ref, None, f"layer {layer} row {b} of {n} tokens")

    def fork(self, parent):
        cca.cca_paged_fork(self.c, self.torch.tensor(parent, dtype=self.torch.int32,
                                                     device="cuda"))
        self.hist = [[h[p] if p >= 0 else None for p in parent] for h in self.hist]


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["eager", "graph"])
@pytest.mark.parametrize("short", ["raw", "core"])
def test_refused_rows_go_on_where_they_were(built, how, short):
    """Three rows, pages for fewer: those that reach a page's end are refused,
    turn after turn, until another row is freed."""
    import torch
    lens = [47, 40, 37] if short == "raw" else [265, 262, 240]
    need = [sum(-(-n // PAGE) - (max(n - 1 - W, 0) // G * G) // PAGE for n in lens),
            sum(-(-(n // G) // PAGE) for n in lens)]
    # none more than they hold of the one pool, enough of the other
    r = Loop(3, lens, need[1] + (20 if short == "raw" else 0),
             need[0] + (0 if short == "raw" else 40))
    run = None
    if how == "graph":
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = r.calls()

        def run():
            graph.replay()
            return outs
    granted = [r.step(run) for _ in range(24)]
    assert not all(granted[-1]) and any(not all(g) for g in granted[:-4])
    held = [b for b in range(3) if not granted[-1][b]]
    kept = [n for b, n in enumerate(r.c.lens.tolist()) if b in held]
    r.fork([b if b in held else -1 for b in range(3)] if len(held) < 3 else [0, 1, -1])
    left = [b for b in held if r.hist[0][b] is not None]
    more = [r.step(run) for _ in range(3)]
    assert any(more[0][b] for b in left), (held, kept)


@pytest.mark.gpu
def test_held_row_is_handed_on_and_freed(built):
    """A fork between the refusal and a step: the copy is held too, a freed
    and refilled row is not."""
    import torch
    r = Loop(3, [32, 20, 5], 12, 2 + 2 + 1, layers=1)  # all pages in use
    keep = [t.clone() for t in r.c.pools]
    cca.cca_paged_reserve(r.c, 1)
    assert cca.cca_device_status() == cca.CCA_ERR_CAPACITY
    assert r.c.lens.tolist() == [32, 21, 6]
    # row 0 is held; its two full pages are shared by row 2
    r.fork([0, 1, 0])
    q, k, v = (to_cuda(synth.random_bf16((3, h, D), 9 + h)) for h in (HQ, HKV, HKV))
    o = cca.cca_paged_step(r.c, q, k, v, out_dtype=torch.float32)
    assert cca.cca_device_status() == cca.CCA_OK
    assert bool((o[[0, 2]] == 0).all()) and not bool((o[1] == 0).all())
    pages = r.c.raw_table[0][r.c.raw_table[0] >= 0].long()
    for a, b in zip(keep[2:], r.c.pools[2:]):
        assert torch.equal(a[:, pages], b[:, pages])
    # the attention reads held rows as ever
    assert not bool((cca.cca_attn_decode_paged(r.c, q)[[0, 2]] == 0).any(-1).all())
    # row 2 ends and is used again, at the length at which it was held
    r.fork([0, -1, -1])
    cca.cca_paged_reserve(r.c, torch.tensor([0, 0, 32], device="cuda"))
    assert cca.cca_device_status() == cca.CCA_OK and r.c.lens.tolist() == [32, 0, 32]
    o = cca.cca_paged_step(r.c, q, k, v, out_dtype=torch.float32)
    assert bool((o[:2] == 0).all()) and not bool((o[2] == 0).all())
    # and with room, row 0 takes its step
    r.fork([0, -1, -1])
    cca.cca_paged_reserve(r.c, 1)
    o = cca.cca_paged_step(r.c, q, k, v, out_dtype=torch.float32)
    assert cca.cca_device_status() == cca.CCA_OK
    h = [np.concatenate([x, synth_row[0][:, None]], 1) for x, synth_row in zip(
        r.hist[0][0], (synth.random_bf16((3, n, D), 9 + n) for n in (HQ, HKV, HKV)))]
    r.check(0, 0, o[0], h)


@pytest.mark.gpu
@pytest.mark.parametrize("more", [2, 16, 75])
def test_further_prompt_fills_the_whole_row_again(built, more):
    """A row given several tokens at once is the whole sequence, filled again;
    the tokens between are not left as the pages' former rows had them."""
    import torch
    r = Loop(2, [50, 33], 12, 30, layers=1)
    for t in r.c.pools[2:]:  # what free pages and rows without a token hold
        t[:, r.c.raw_ref == 0] = float("nan")
    for _ in range(3):
        r.step()
    cca.cca_paged_reserve(r.c, torch.tensor([more, 0], device="cuda"))
    assert cca.cca_device_status() == cca.CCA_OK
    new = packed_inputs([more], HQ, HKV, D, 77)[:3]
    h = r.hist[0][0] = [np.concatenate([x, y], 1) for x, y in zip(r.hist[0][0], new)]
    n = h[0].shape[1]
    assert r.c.lens.tolist() == [n, 36]
    Q, K, V = (to_cuda(x) for x in h)
    cu, row = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [0]))
    # not the new tokens alone: they are not as long as the row
    part = torch.tensor([0, more], dtype=torch.int32, device="cuda")
    x = [t[:, :more] for t in (Q, K, V)]
    cca.cca_paged_fill(r.c, *x[1:], *cca.cca_pool_packed(*x, part, G), part, row)
    assert cca.cca_device_status() == cca.CCA_ERR_PAGE
    cca.cca_paged_fill(r.c, K, V, *cca.cca_pool_packed(Q, K, V, cu, G), cu, row)
    assert cca.cca_device_status() == cca.CCA_OK
    q = Q[:, -1].expand(2, HQ, D).contiguous()
    o = cca.cca_attn_decode_paged(r.c, q, out_dtype=torch.float32)
    r.check(0, 0, o[0], h)
    for _ in range(2):
        r.step()


@pytest.mark.gpu
def test_rows_that_ask_for_nothing_stay_what_they_were(built):
    """n = 0 neither holds a row nor lets it go."""
    import torch
    r = Loop(2, [32, 20], 12, 2 + 2, layers=1)
    i64 = lambda *x: torch.tensor(x, dtype=torch.int64, device="cuda")  # noqa: E731
    q, k, v = (to_cuda(synth.random_bf16((2, h, D), 20 + h)) for h in (HQ, HKV, HKV))

    def step():
        return [bool((x == 0).all()) for x in cca.cca_paged_step(r.c, q, k, v)]
    cca.cca_paged_reserve(r.c, i64(0, 0))
    assert step() == [False, False]
    cca.cca_paged_reserve(r.c, i64(1, 1))  # row 0 has no page for token 32
    assert cca.cca_device_status() == cca.CCA_ERR_CAPACITY
    assert step() == [True, False]
    cca.cca_paged_reserve(r.c, i64(0, 0))
    assert step() == [True, False]
    cca.cca_paged_reserve(r.c, i64(-1, -1))  # refused: held
    assert cca.cca_device_status() == cca.CCA_ERR_CAPACITY
    assert step() == [True, True]
    cca.cca_paged_reserve(r.c, i64(0, 1))
    assert step() == [True, False]
    # the C call without a workspace leaves no note, and takes none away
    n = i64(0, 1)
    assert cca.lib().cca_paged_reserve(r.c.struct, P(n.data_ptr()), 0, None) == cca.CCA_OK
    assert step() == [True, False]
    assert cca.cca_device_status() == cca.CCA_OK


@pytest.mark.gpu
def test_histories_under_random_calls(built):
    """Prompts, steps, forks and compaction in small pools, in any order:
    every row's keys are those that it was granted."""
    assert sum(_random_calls(seed) for seed in range(8)) > 20


def _random_calls(seed):
    """Returns how many steps were refused."""
    import random

    import torch
    rng = random.Random(seed)
    B, g, w, page = rng.choice([3, 8]), 4, rng.choice([0, 10, 40]), 16
    c = cca.PagedCache(B, 2, 1, D, g, w, page, rng.choice([4, 9]), rng.choice([8, 14]), max_len=160)
    hist = [[] for _ in range(B)]
    refused = 0

    def check(what):
        table, n = c.raw_table.cpu().numpy(), c.lens.tolist()
        k = c.k_raw[0, :, 0].float().cpu().numpy()
        for b in range(B):
            assert n[b] == len(hist[b]), (what, b)
            lo = max(n[b] - 1 - w, 0) // g * g
            got = np.array([k[table[b, t // page], t % page] for t in range(lo, n[b])])
            assert got.size == 0 or (got == np.array(hist[b][lo:])[:, None]).all(), (what, b)

    for turn in range(120):
        what = rng.choice("ssssspfc")
        before = c.lens.tolist()
        if what == "s":
            cca.cca_paged_reserve(c, 1)
            x = [rng.randrange(256) for _ in range(B)]
            k = torch.tensor(x, device="cuda")[:, None, None].expand(B, 1, D).bfloat16()
            q = torch.ones((B, 2, D), dtype=torch.bfloat16, device="cuda")
            o = cca.cca_paged_step(c, q, k.contiguous(), k.contiguous())
            for b, (a, z) in enumerate(zip(before, c.lens.tolist())):
                if z > a:
                    hist[b].append(x[b])
                else:
                    refused += a > 0
                    assert bool((o[b] == 0).all())
        elif what == "p":
            n = [0 if a or rng.random() < 0.5 else rng.randint(1, 60) for a in before]
            cca.cca_paged_reserve(c, torch.tensor(n, device="cuda"))
            rows = [b for b, z in enumerate(c.lens.tolist()) if z and not before[b]]
            if rows:
                x = [[rng.randrange(256) for _ in range(n[b])] for b in rows]
                flat = torch.tensor(sum(x, []), device="cuda")
                K = flat[None, :, None].expand(1, -1, D).bfloat16().contiguous()
                cu = torch.tensor([0, *np.cumsum([len(y) for y in x])], dtype=torch.int32,
                                  device="cuda")
                core = cca.cca_pool_packed(K.expand(2, -1, -1).contiguous(), K, K, cu, g)
                cca.cca_paged_fill(c, K, K, *core, cu,
                                   torch.tensor(rows, dtype=torch.int32, device="cuda"))
                for b, y in zip(rows, x):
                    hist[b] = y
        elif what == "f":
            parent = [rng.choice([b, b, b, rng.randint(-1, B - 1)]) for b in range(B)]
            cca.cca_paged_fork(c, torch.tensor(parent, dtype=torch.int32, device="cuda"))
            hist = [list(hist[p]) if p >= 0 and z else [] for p, z in zip(parent, c.lens.tolist())]
        else:
            cca.cca_paged_compact(c)
        assert cca.cca_device_status() in (cca.CCA_OK, cca.CCA_ERR_CAPACITY), (turn, what)
        check((turn, what))
    return refused


@pytest.mark.gpu
def test_notes_are_in_the_workspace_of_the_call(built):
    """A refusal noted in one workspace holds the row for steps with that one."""
    import torch
    r = Loop(2, [32, 20], 12, 2 + 2, layers=1)
    ws = torch.zeros_like(r.c.workspace)
    q, k, v = (to_cuda(synth.random_bf16((2, h, D), 20 + h)) for h in (HQ, HKV, HKV))
    cca.cca_paged_reserve(r.c, 1, workspace=ws)  # row 0 has no page for token 32
    assert cca.cca_device_status() == cca.CCA_ERR_CAPACITY
    keep = r.c.k_raw.clone()
    o = cca.cca_paged_step(r.c, q, k, v, workspace=ws)
    assert bool((o[0] == 0).all()) and not bool((o[1] == 0).all())
    row = r.c.raw_table[0][r.c.raw_table[0] >= 0].long()
    assert torch.equal(r.c.k_raw[:, row], keep[:, row])
    assert not bool((cca.cca_paged_step(r.c, q, k, v)[0] == 0).all())
    assert cca.cca_device_status() == cca.CCA_OK
