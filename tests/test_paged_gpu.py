"""The paged decode cache through the C ABI: page upkeep against the CPU
model (exactly), attention against the fp64 oracle on each row's own history
(the suite's tolerances, gpu_util), and prompts, steps, forks, frees and
compaction together, as a server uses them."""

import random

import numpy as np
import pytest

import oracle
from gpu_util import assert_close, to_cuda
from long_context_sparse_cca_b200 import synth
from serving_model import PagedModel, packed_inputs, window_start

pytestmark = pytest.mark.gpu
ALL = 1 << 30


@pytest.fixture(scope="module")
def cca():
    from long_context_sparse_cca_b200 import build
    build.build()
    import long_context_sparse_cca_b200 as m
    return m


def _i64(x):
    import torch
    return torch.tensor(x, dtype=torch.int64, device="cuda")


def _i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _same_tables(c, m, what=""):
    assert c.lens.tolist() == m.lens.tolist(), what
    for name, a, b in (("core_table", c.core_table, m.table[0]), ("raw_table", c.raw_table, m.table[1]),
                       ("core_ref", c.core_ref, m.ref[0]), ("raw_ref", c.raw_ref, m.ref[1])):
        assert np.array_equal(a.cpu().numpy(), b), (what, name)


def _label(c):
    """Every page of every layer holds its own number, and a tag of its pool,
    layer and tensor."""
    import torch
    for i, t in enumerate(c.pools):
        layers, pages = t.shape[:2]
        x = torch.arange(layers * pages, device="cuda").view(layers, pages, 1, 1, 1)
        t.copy_((x % 251 + i * 256).to(t.dtype).expand(t.shape))


def _content(c):
    """Labels of the pages (checked to be whole pages)."""
    out = []
    for t in c.pools:
        assert bool((t == t[:, :, :1, :1, :1]).all())
        out.append(t[:, :, 0, 0, 0].float().cpu().numpy())
    return out


# ---------------------------------------------------------------- page upkeep

@pytest.mark.parametrize("seed", range(8))
def test_upkeep_matches_model(cca, seed):
    """Random calls; tables, counts, lengths and the pages' contents are the
    model's after each."""
    rng = random.Random(seed)
    B = rng.choice([1, 5, 40])
    g, w, page = rng.choice([(16, 64, 16), (8, 250, 32), (4, 0, 16), (16, 64, 64), (16, ALL, 16)])
    plain = w == ALL
    core_pages, raw_pages = (0 if plain else rng.choice([9, 60])), rng.choice([30, 1500])
    c = cca.PagedCache(B, 2, 1, 64, g, w, page, core_pages, raw_pages, max_len=60 * page,
                       layers=rng.choice([1, 3]))
    m = PagedModel(B, g, w, page, core_pages, raw_pages, c.core_cols, c.raw_cols)
    _label(c)
    m.content = [[p for p in range(n)] for n in m.pages]
    start = _content(c)
    statuses = set()
    for step in range(40):
        what = rng.choice("rrrrffc")
        want = cca.CCA_OK
        if what == "r" and rng.random() < 0.5:
            if m.reserve(1):
                want = cca.CCA_ERR_CAPACITY
            cca.cca_paged_reserve(c, 1)
        elif what == "r":
            n = [rng.choice([0, 0, 1, -3, rng.randint(1, 40 * page)]) for _ in range(B)]
            if m.reserve(n):
                want = cca.CCA_ERR_CAPACITY
            cca.cca_paged_reserve(c, _i64(n))
        elif what == "f":
            parent = [rng.randint(-1, B - 1) if rng.random() < 0.5 else b for b in range(B)]
            if rng.random() < 0.2:
                parent[0] = rng.choice([-2, B, 1 << 30])
            failed, wrong = m.fork(parent)
            want = (cca.CCA_ERR_CAPACITY if failed else cca.CCA_ERR_PAGE if wrong else cca.CCA_OK)
            cca.cca_paged_fork(c, _i32(parent))
        else:
            live = m.compact()
            assert cca.cca_paged_compact(c).tolist() == live
        got = cca.cca_device_status()
        statuses.add(got)
        assert got == want, (step, what)
        _same_tables(c, m, (step, what))
        for i, (now, then) in enumerate(zip(_content(c), start)):
            pool = i // 2
            used = [p for p in range(m.pages[pool]) if m.ref[pool][p]]
            labels = [m.content[pool][p] for p in used]
            assert np.array_equal(now[:, used], then[:, labels]), (step, what, i)
    assert cca.CCA_OK in statuses


def test_large_pools(cca):
    """Thousands of rows and pages: more than one pass of every scan."""
    rng = random.Random(3)
    B, g, w, page = 4096, 16, 64, 16
    c = cca.PagedCache(B, 1, 1, 64, g, w, page, 6000, 40000, max_len=1024)
    m = PagedModel(B, g, w, page, 6000, 40000, c.core_cols, c.raw_cols)
    n = [rng.choice([0, 1, 15, 16, 17, rng.randint(1, 600)]) for _ in range(B)]
    m.reserve(n)
    cca.cca_paged_reserve(c, _i64(n))
    _same_tables(c, m, "reserve")
    parent = [rng.randint(-1, B - 1) for _ in range(B)]
    m.fork(parent)
    cca.cca_paged_fork(c, _i32(parent))
    _same_tables(c, m, "fork")
    m.reserve(1)
    cca.cca_paged_reserve(c, 1)
    _same_tables(c, m, "step")
    assert cca.cca_paged_compact(c).tolist() == m.compact()
    _same_tables(c, m, "compact")
    cca.cca_device_status()


def test_upkeep_replayed_in_a_graph(cca):
    import torch
    args = (3, 2, 1, 64, 16, 64, 16, 12, 60)
    a, b = (cca.PagedCache(*args, max_len=500) for _ in range(2))
    m = PagedModel(3, 16, 64, 16, 12, 60, a.core_cols, a.raw_cols)
    for c in (a, b):
        _label(c)
        cca.cca_paged_reserve(c, _i64([100, 37, 0]))
    m.reserve([100, 37, 0])
    parent = _i32([0, 1, 0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cca.cca_paged_fork(a, parent)
        cca.cca_paged_reserve(a, 1)
        live = cca.cca_paged_compact(a)
    for p in ([0, 1, 0], [1, 1, 2], [0, -1, 2], [2, 0, 0]):
        parent.copy_(_i32(p))
        graph.replay()
        m.fork(p)
        m.reserve(1)
        want = m.compact()
        assert live.tolist() == want
        _same_tables(a, m, p)
        cca.cca_paged_fork(b, _i32(p))
        cca.cca_paged_reserve(b, 1)
        cca.cca_paged_compact(b)
        for x, y in zip(a.pools, b.pools):
            assert torch.equal(x, y)
    assert cca.cca_device_status() == cca.CCA_OK


# ---------------------------------------------------------------- attention

class Rows:
    """Rows of a cache with the history each has seen (bit patterns)."""

    def __init__(self, cca, B, Hq, Hkv, d, g, w, page, max_len, layers=1, core=True, slack=3):
        import torch
        self.cca, self.torch = cca, torch
        self.shape = (Hq, Hkv, d)
        self.g, self.w, self.layers = g, w, layers
        raw = B * (min(max_len, w + g) // page + slack)
        self.c = cca.PagedCache(B, Hq, Hkv, d, g, w, page, B * (max_len // g // page + 2) if core else 0,
                                raw, max_len=max_len, layers=layers)
        # pages hold NaN until something is written to them
        for t in self.c.pools:
            t.fill_(float("nan"))
        self.hist = [[None] * B for _ in range(layers)]
        self.seed = 1000

    def prompts(self, rows, lens, order="head"):
        Hq, Hkv, d = self.shape
        torch, cca = self.torch, self.cca
        n = [0] * self.c.B
        for b, x in zip(rows, lens):
            n[b] = x
        cca.cca_paged_reserve(self.c, _i64(n))
        for layer in range(self.layers):
            self.seed += 10
            q, k, v, cu = packed_inputs(lens, Hq, Hkv, d, self.seed)
            Q, K, V = (to_cuda(x) for x in (q, k, v))
            if order == "token":
                Q, K, V = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (Q, K, V))
            cu_d = _i32(cu.tolist())
            Kc = Vc = None
            if self.c.core_cols:
                Kc, Vc = cca.cca_pool_packed(Q, K, V, cu_d, self.g)
            cca.cca_paged_fill(self.c, K, V, Kc, Vc, cu_d, _i32(rows), layer=layer)
            for s, b in enumerate(rows):
                self.hist[layer][b] = [x[:, cu[s]:cu[s + 1]] for x in (q, k, v)]

    def step(self, call="step", dtype=None, check=True):
        """One token for every row in use, all layers, checked."""
        Hq, Hkv, d = self.shape
        torch, cca, c = self.torch, self.cca, self.c
        cca.cca_paged_reserve(c, 1)
        outs = []
        for layer in range(self.layers):
            self.seed += 10
            q = synth.random_bf16((c.B, Hq, d), self.seed)
            k = synth.random_bf16((c.B, Hkv, d), self.seed + 1, scale=1.5)
            v = synth.random_bf16((c.B, Hkv, d), self.seed + 2)
            o = cca.cca_paged_step(c, to_cuda(q), to_cuda(k), to_cuda(v), layer=layer,
                                   out_dtype=dtype or torch.float32)
            if check:
                again = cca.cca_attn_decode_paged(c, to_cuda(q), layer=layer,
                                                  out_dtype=dtype or torch.float32)
                assert torch.equal(o, again), "the step's output is the attention over its result"
            for b in range(c.B):
                h = self.hist[layer][b]
                if h is None:
                    assert not check or bool((o[b] == 0).all())
                    continue
                self.hist[layer][b] = [np.concatenate([x, y[b][:, None]], 1)
                                       for x, y in zip(h, (q, k, v))]
            outs.append(o)
            if check:
                self.check(layer, o)
        return outs

    def check(self, layer, o):
        for b in range(self.c.B):
            h = self.hist[layer][b]
            if h is None:
                continue
            x = [synth.bf16_bits_to_f64(np.ascontiguousarray(y[None])) for y in h]
            n = x[0].shape[2]
            ref = oracle.prefill(*x, self.g, min(self.w, n), rows=[n - 1])[0, :, 0]
            assert_close(o[b], ref, None, f"layer {layer} row {b} of {n} tokens")

    def fork(self, parent):
        self.cca.cca_paged_fork(self.c, _i32(parent))
        for layer in range(self.layers):
            self.hist[layer] = [self.hist[layer][p] if p >= 0 else None for p in parent]


CASES = [  # Hq, Hkv, d, g, w, page, prompts, core pages?
    (4, 2, 128, 16, 64, 16, [200, 257, 1, 79], True),
    (1, 1, 64, 16, 64, 64, [15, 16, 17, 31], True),
    (8, 8, 64, 8, 250, 32, [1000, 3, 250, 258], True),
    (16, 1, 128, 24, 100, 16, [500, 23, 24, 124], True),
    (6, 2, 64, 32, 0, 128, [63, 64, 5000, 32], True),
    (12, 4, 128, 1, 10, 16, [300, 1, 2, 9], True),
    (10, 2, 64, 16, 1024, 1024, [2100, 1039, 4, 1040], True),
    (32, 2, 128, 256, 300, 64, [2500, 255, 256, 511], True),
    (4, 1, 64, 16, ALL, 16, [300, 16, 1, 700], False),
    (4, 4, 128, 16, ALL, 32, [33, 32, 31, 2000], True),
    (32, 2, 64, 256, 300, 16, [2500, 255, 256, 511], True),
    (12, 1, 128, 16, 64, 16, [200, 257, 1, 79], True),
    (9, 1, 64, 32, 40, 16, [500, 31, 1, 64], True),
    (8, 1, 128, 16, 64, 32, [1500, 257, 2, 80], True),
    (14, 2, 128, 17, 50, 16, [333, 17, 34, 800], True),
]


@pytest.mark.parametrize("case", CASES, ids=[str(c) for c in CASES])
def test_steps_match_oracle(cca, case):
    """Prompts, then steps over group, window and page borders; every row
    against its own history; one row is free."""
    Hq, Hkv, d, g, w, page, lens, core = case
    r = Rows(cca, 5, Hq, Hkv, d, g, w, page, max(lens) + 40, core=core)
    r.prompts([0, 3, 2, 4], lens, order="token" if d == 64 else "head")
    assert cca.cca_device_status() == cca.CCA_OK
    for i in range(2 * min(g, 16) + 2):
        r.step(check=i < 2 or i % 5 == 0)
    assert cca.cca_device_status() == cca.CCA_OK


@pytest.mark.parametrize("B,Hq,Hkv,d", [(4096, 2, 2, 64), (3000, 8, 1, 128), (700, 16, 1, 128),
                                        (1000, 3, 1, 64)])
def test_many_rows(cca, B, Hq, Hkv, d):
    """Batches whose list takes the room of a ring's stage or of warps; rows
    of 0 to 60 tokens, every one against its own attention in fp64 (w = 0 and
    g = 4: core rows of all groups but the last)."""
    import torch
    g, w, page = 4, 0, 16
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 61, size=B)
    total = int(lens.sum())
    q, k, v, cu = packed_inputs(lens.tolist(), Hq, Hkv, d, B)
    Q, K, V = (to_cuda(x) for x in (q, k, v))
    c = cca.PagedCache(B, Hq, Hkv, d, g, w, page, 2 * B, 2 * B, max_len=64)
    cca.cca_paged_reserve(c, _i64(lens.tolist()))
    half = B // 2  # (a call takes up to 8192 sequences; two calls here)
    for a, b in ((0, half), (half, B)):
        lo, hi = int(cu[a]), int(cu[b])
        x = [t[:, lo:hi] for t in (Q, K, V)]
        cu_d = _i32((cu[a:b + 1] - lo).tolist())
        Kc, Vc = cca.cca_pool_packed(*x, cu_d, g)
        cca.cca_paged_fill(c, x[1], x[2], Kc, Vc, cu_d, _i32(list(range(a, b))))
    qt = to_cuda(synth.random_bf16((B, Hq, d), 3 * B))
    o = cca.cca_attn_decode_paged(c, qt, out_dtype=torch.float32)
    assert cca.cca_device_status() == cca.CCA_OK
    # the definition, all rows at once: groups before the window's, then it
    f = torch.float64
    n = torch.from_numpy(lens).cuda()
    ws = (n - 1).clamp(min=0) // g * g
    p = torch.arange(64, device="cuda")
    first = torch.from_numpy(cu[:-1].astype(np.int64)).cuda()
    at = (first[:, None] + p).clamp(max=max(total - 1, 0))
    Kr, Vr = (t[:, at].to(f) for t in (K, V))                       # [Hkv, B, 64, d]
    qg = Q[:, at[:, g - 1::g]].to(f).view(Hkv, Hq // Hkv, B, 16, d)  # the groups' last queries
    kg, vg = (t.view(Hkv, B, 16, g, d) for t in (Kr, Vr))
    a = torch.softmax(torch.einsum("hrbjd,hbjgd->hrbjg", qg, kg) / d ** 0.5, -1).mean(1)
    Kc, Vc = (torch.einsum("hbjg,hbjgd->hbjd", a, t) for t in (kg, vg))
    keys, vals = torch.cat([Kc, Kr], 2), torch.cat([Vc, Vr], 2)
    seen = torch.cat([p[:16] < (ws // g)[:, None],
                      (p >= ws[:, None]) & (p < n[:, None])], 1)
    s = torch.einsum("bhrd,hbkd->bhrk", qt.to(f).view(B, Hkv, -1, d), keys) / d ** 0.5
    s = s.masked_fill(~seen[:, None, None], -float("inf"))
    ref = torch.einsum("bhrk,hbkd->bhrd", torch.nan_to_num(torch.softmax(s, -1)), vals)
    assert_close(o, ref.reshape(B, Hq, d).cpu().numpy(), None, "o")


def test_steps_from_an_empty_prompt(cca):
    """A conversation that begins with its first step."""
    r = Rows(cca, 2, 4, 2, 64, 4, 8, 16, 200)
    cca.cca_paged_reserve(r.c, _i64([1, 0]))
    q, k, v = (synth.random_bf16((2, h, 64), 5 + h) for h in (4, 2, 2))
    o = cca.cca_paged_step(r.c, to_cuda(q), to_cuda(k), to_cuda(v), out_dtype=r.torch.float32)
    r.hist[0][0] = [x[0][:, None] for x in (q, k, v)]
    r.check(0, o)
    assert bool((o[1] == 0).all())
    for _ in range(20):
        r.step()
    assert cca.cca_device_status() == cca.CCA_OK


def test_bf16_output_is_the_rounded_f32_one(cca):
    r = Rows(cca, 3, 8, 2, 128, 16, 64, 16, 400)
    r.prompts([0, 1, 2], [300, 64, 7])
    cca.cca_paged_reserve(r.c, 1)
    q, k, v = (to_cuda(synth.random_bf16((3, h, 128), 50 + h)) for h in (8, 2, 2))
    a = cca.cca_paged_step(r.c, q, k, v, out_dtype=r.torch.float32)
    assert r.torch.equal(cca.cca_paged_step(r.c, q, k, v), a.bfloat16())


def test_serving_run(cca):
    """Prompts, samples forked from them, beams that change places, rows that
    end and are used again, compaction in between: every row's output is the
    oracle's on its own history, in two layers."""
    r = Rows(cca, 6, 4, 2, 64, 16, 64, 16, 600, layers=2, slack=6)
    r.prompts([1, 4], [203, 70])
    assert cca.cca_device_status() == cca.CCA_OK
    r.fork([1, 1, 1, 4, 4, 4])
    for _ in range(3):
        r.step(check=False)
    r.step()
    r.fork([1, 0, 0, -1, 5, 5])
    cca.cca_paged_compact(r.c)
    for _ in range(18):
        r.step(check=False)
    r.step()
    r.prompts([3], [129])
    r.step()
    r.fork([-1, 1, 3, 3, -1, 5])
    live = cca.cca_paged_compact(r.c)
    r.step()
    r.prompts([0, 4], [16, 300], order="token")
    for _ in range(17):
        r.step(check=False)
    r.step()
    assert cca.cca_device_status() == cca.CCA_OK
    assert live.tolist()[1] <= r.c.raw_pages
    # a saved session goes on where it was
    saved = r.c.state_dict()
    r.c = type(r.c).from_state_dict(saved)
    r.step()
    assert cca.cca_device_status() == cca.CCA_OK


def test_steps_replayed_in_a_graph(cca):
    """A captured step replayed over group, window and page borders equals
    eager steps bit for bit."""
    import torch
    runs = []
    for how in ("eager", "graph"):
        r = Rows(cca, 3, 4, 2, 128, 16, 64, 16, 400, layers=2)
        r.prompts([0, 2], [150, 60])
        q, k, v = (torch.zeros((3, h, 128), dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2))

        def once():
            cca.cca_paged_reserve(r.c, 1)
            return [cca.cca_paged_step(r.c, q, k, v, layer=i) for i in range(2)]
        outs = []
        graph = None
        for i in range(40):
            for j, t in enumerate((q, k, v)):
                t.copy_(to_cuda(synth.random_bf16(tuple(t.shape), 7000 + 3 * i + j)))
            if how == "eager":
                o = once()
            else:
                if graph is None:
                    torch.cuda.synchronize()
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph):
                        o = once()
                graph.replay()
            outs += [x.clone() for x in o]
        runs.append((outs, r.c))
    assert cca.cca_device_status() == cca.CCA_OK
    for x, y in zip(runs[0][0], runs[1][0]):
        assert torch.equal(x, y)
    assert torch.equal(runs[0][1].tables, runs[1][1].tables)


def test_pages_scattered_over_a_large_pool(cca):
    """Pool offsets beyond 2^31 elements; the same result as with the pages
    in order."""
    import torch
    Hq, Hkv, d, g, w, page = 2, 2, 128, 16, 64, 64
    far = (1 << 31) // (Hkv * page * d) + 5  # pages: the last ones lie behind 2^31 elements
    c = cca.PagedCache(1, Hq, Hkv, d, g, w, page, 4, far, max_len=2000)
    r = Rows(cca, 1, Hq, Hkv, d, g, w, page, 2000)
    c.raw_ref[:far - 4] = 1
    n, m = 300, 300 // g
    q, k, v, cu = packed_inputs([n], Hq, Hkv, d, 31)
    Q, K, V = (to_cuda(x) for x in (q, k, v))
    qt = to_cuda(synth.random_bf16((1, Hq, d), 99))
    outs = []
    for cache in (c, r.c):
        Kc, Vc = cca.cca_pool_packed(Q, K, V, _i32([0, n]), g)
        cca.cca_paged_reserve(cache, _i64([n]))
        cca.cca_paged_fill(cache, K, V, Kc, Vc, _i32([0, n]), _i32([0]))
        outs.append(cca.cca_attn_decode_paged(cache, qt))
    assert cca.cca_device_status() == cca.CCA_OK
    assert int(c.raw_table.max()) >= far - 4 and m > 0
    assert torch.equal(*outs)


def test_two_attentions_at_once(cca):
    """Two streams read one cache, each with a workspace of its own."""
    import torch
    r = Rows(cca, 3, 8, 2, 128, 16, 64, 16, 3000)
    r.prompts([0, 1, 2], [2900, 1500, 64])
    qs = [to_cuda(synth.random_bf16((3, 8, 128), 700 + i)) for i in range(2)]
    want = [cca.cca_attn_decode_paged(r.c, q) for q in qs]
    ws = [torch.zeros_like(r.c.workspace) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [cca.cca_attn_decode_paged(r.c, q, workspace=x, stream=s)
               for q, x, s in zip(qs, ws, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert cca.cca_device_status() == cca.CCA_OK


def test_same_call_same_bits(cca):
    """Over and over, whatever the order in which CTAs arrive at a pair."""
    import torch
    r = Rows(cca, 4, 4, 1, 128, 16, 1024, 16, 9000)
    r.prompts([0, 1, 2, 3], [8800, 1, 5000, 300])
    q = to_cuda(synth.random_bf16((4, 4, 128), 71))
    want = cca.cca_attn_decode_paged(r.c, q, out_dtype=torch.float32)
    for _ in range(50):
        assert torch.equal(want, cca.cca_attn_decode_paged(r.c, q, out_dtype=torch.float32))
    assert cca.cca_device_status() == cca.CCA_OK


# ---------------------------------------------------------------- refusals on the device

def test_fill_leaves_out_what_does_not_fit(cca):
    import torch
    Hq, Hkv, d, g, w, page = 2, 2, 64, 16, 64, 16
    q, k, v, cu = packed_inputs([40, 50], Hq, Hkv, d, 8)
    Q, K, V = (to_cuda(x) for x in (q, k, v))
    cu_d = _i32(cu.tolist())
    Kc, Vc = cca.cca_pool_packed(Q, K, V, cu_d, g)

    def fill(rows, lens=(40, 50), break_page=False, fork=None):
        c = cca.PagedCache(2, Hq, Hkv, d, g, w, page, 4, 20, max_len=200)
        cca.cca_paged_reserve(c, _i64(lens))
        if fork:
            cca.cca_paged_fork(c, _i32(fork))
        if break_page:
            c.raw_table[0, 1] = -1
        for t in c.pools:
            t.fill_(5.0)
        cca.cca_paged_fill(c, K, V, Kc, Vc, cu_d, _i32(rows))
        return c, cca.cca_device_status()

    whole, st = fill([0, 1])
    assert st == cca.CCA_OK
    for rows, lens in (([0, 2], (40, 50)), ([0, -1], (40, 50)), ([0, 1], (40, 51))):
        c, st = fill(rows, lens)
        assert st == cca.CCA_ERR_PAGE
        pages = whole.raw_table[0][whole.raw_table[0] >= 0]
        assert torch.equal(c.k_raw[:, pages], whole.k_raw[:, pages])  # the other one is there
        others = [p for p in range(20) if p not in pages.tolist()]
        assert bool((c.k_raw[:, others] == 5).all()) and bool((c.v_raw[:, others] == 5).all())
    c, st = fill([1, 1], (40, 50))  # named twice: the later sequence
    assert st == cca.CCA_ERR_PAGE
    p1 = whole.raw_table[1][whole.raw_table[1] >= 0]
    assert torch.equal(c.k_raw[:, p1], whole.k_raw[:, p1])
    p0 = whole.raw_table[0][whole.raw_table[0] >= 0]
    assert bool((c.k_raw[:, p0] == 5).all())
    c, st = fill([0, 1], break_page=True)
    assert st == cca.CCA_ERR_PAGE
    # pages of two rows are not written
    c, st = fill([0, 1], lens=(40, 50), fork=[0, 0])
    assert st == cca.CCA_ERR_PAGE
    shared = c.raw_table[0, :2]
    assert bool((c.k_raw[:, shared] == 5).all())
    # offsets out of order: nothing is written
    c = cca.PagedCache(2, Hq, Hkv, d, g, w, page, 4, 20, max_len=200)
    cca.cca_paged_reserve(c, _i64([40, 50]))
    cca.cca_paged_fill(c, K, V, Kc, Vc, _i32([0, 91, 90]), _i32([0, 1]))
    assert cca.cca_device_status() == cca.CCA_ERR_SEQLENS
    assert bool((c.k_raw == 0).all())


def test_step_does_not_write_shared_or_missing_pages(cca):
    import torch
    r = Rows(cca, 2, 2, 2, 64, 16, 64, 16, 200)
    r.prompts([0], [32])
    cca.cca_paged_fork(r.c, _i32([0, 0]))  # two full pages, shared
    before = [t.clone() for t in r.c.pools]
    q, k, v = (to_cuda(synth.random_bf16((2, 2, 64), 60 + i)) for i in range(3))
    cca.cca_paged_step(r.c, q, k, v)       # without cca_paged_reserve
    assert cca.cca_device_status() == cca.CCA_ERR_PAGE
    for a, b in zip(before, r.c.pools):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    cca.cca_paged_reserve(r.c, 1)
    r.c.raw_table[1, 2] = -1
    r.c.raw_table[0, 1] = 10 ** 6
    o = cca.cca_paged_step(r.c, q, k, v, out_dtype=torch.float32)
    assert cca.cca_device_status() == cca.CCA_ERR_PAGE
    assert bool(torch.isfinite(o).all())


def test_garbage_lengths_and_tables(cca):
    """Whatever the tables hold, nothing outside the cache is touched."""
    import torch
    c = cca.PagedCache(4, 2, 1, 64, 16, 64, 16, 4, 12, max_len=150)
    gen = torch.Generator().manual_seed(4)
    for trial in range(6):
        guard = [t.clone() for t in c.pools]
        c.lens.copy_(torch.tensor([-5, 1 << 62, 140, -(1 << 62)]))
        for t in (c.core_table, c.raw_table):
            t.copy_(torch.randint(-(1 << 31), 1 << 31, t.shape, generator=gen).int())
        c.core_ref.fill_(1)
        c.raw_ref.fill_(1)
        q, k, v = (torch.ones((4, h, 64), dtype=torch.bfloat16, device="cuda") for h in (2, 1, 1))
        if trial < 2:
            c.lens.copy_(torch.tensor([-5, 148, 140, 1 << 62]))
            cca.cca_paged_step(c, q, k, v)
            assert bool((cca.cca_attn_decode_paged(c, q)[[0, 3]] == 0).all())
        elif trial == 2:
            cca.cca_paged_reserve(c, 1)
        elif trial == 3:
            cca.cca_paged_fork(c, _i32([2, 1, 1, 0]))
        elif trial == 4:
            cca.cca_paged_compact(c)
        else:
            cu = _i32([0, 140])
            x = torch.ones((1, 140, 64), dtype=torch.bfloat16, device="cuda")
            kc = torch.ones((1, 8, 64), dtype=torch.float16, device="cuda")
            cca.cca_paged_fill(c, x, x, kc, kc, cu, _i32([2]))
        assert cca.cca_device_status() in (cca.CCA_ERR_PAGE, cca.CCA_ERR_CAPACITY)
        if trial in (0, 1, 2, 5):
            for a, b in zip(guard, c.pools):
                assert torch.equal(a, b)


def test_window_start_of_the_model():
    assert [window_start(t, 16, 64) for t in (0, 63, 64, 79, 80, 96)] == [0, 0, 0, 0, 16, 32]
