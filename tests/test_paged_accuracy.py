"""How near the paged decode's outputs are to fp64, beyond the suite's
tolerance: a weight is held in two 16-bit numbers, and that has to show.

The bound.  With q in {-1, 0, 1} and keys that are multiples of 1/4 all scores
are exact, so that against fp64 on the cache's own rows an output is off by
at most e * sum_j w_j |v_j| + 2^-40 * sum_core |v_j|, w the softmax, e the
sum of
  2^-16 + 2^-20  the weights' two numbers (8 bits each at least; for more
                 than 8 query heads the second one has 2^-20 added),
  2^-21          ex2.approx, 2^-22 for the weights and for their sum,
  s * 2^-22      scaling the scores, at most s (log2 units), and subtracting
                 the maximum, for the weights and for their sum,
  n * 2^-22      n additions each of P V (2^-23: the tensor cores may cut
                 off) and of the weights' sum (2^-24), and the joins;
2^-40 is half of fp16's smallest number over the 2^15 that core weights are
relative to.  One 16-bit number alone is off by 2^-9 (bf16) or 2^-12 (fp16) of
a weight: the emulations below show that the bound tells.
"""

import math

import pytest
import torch

import long_context_sparse_cca_b200 as cca
from long_context_sparse_cca_b200 import build as cca_build

BF, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64


def _rows_of(table, pool, b, lo, hi, page):
    """Rows lo .. hi - 1 of a row of the batch, [Hkv, n, d]."""
    x = torch.arange(lo, hi, device=pool.device)
    return pool[0][table[b, x // page].long(), :, x % page].transpose(0, 1)


def _seen(c, b):
    """Core and raw (keys, values) that the newest token of row b sees."""
    n = int(c.lens[b])
    ws = max(n - 1 - c.w, 0) // c.g * c.g
    core = [_rows_of(c.core_table, t, b, 0, ws // c.g, c.page) for t in (c.k_core, c.v_core)]
    raw = [_rows_of(c.raw_table, t, b, ws, n, c.page) for t in (c.k_raw, c.v_raw)]
    return core, raw


def _reference(c, q, b):
    """Row b in fp64: output, sum of w |v|, sum of |v| over core rows, scores'
    size in log2 units, keys."""
    (kc, vc), (kr, vr) = _seen(c, b)
    k, v = torch.cat([kc.to(F64), kr.to(F64)], 1), torch.cat([vc.to(F64), vr.to(F64)], 1)
    x = q[b].to(F64).view(c.Hkv, -1, c.d) @ k.transpose(1, 2) / math.sqrt(c.d)
    w = torch.softmax(x, -1)
    r = c.Hq // c.Hkv
    core = vc.to(F64).abs().sum(1, keepdim=True).expand(-1, r, -1)
    return ((w @ v).reshape(c.Hq, c.d), (w @ v.abs()).reshape(c.Hq, c.d),
            core.reshape(c.Hq, c.d), float(x.abs().max()) / math.log(2), k.shape[1])


def _off(got, ref):
    """How many times the bound an output is off."""
    o, size, core, s, n = ref
    e = 2.0 ** -16 + 2.0 ** -20 + 2.0 ** -21 + s * 2.0 ** -22 + n * 2.0 ** -22
    return float(((got.to(F64) - o).abs() / (e * size + 2.0 ** -40 * core + 1e-300)).max())


def _filled(lens, Hq, Hkv, d, g, w, page, device, seed=0):
    """A cache with rows of these lengths, keys of multiples of 1/4, and
    queries of -1, 0 and 1."""
    gen = torch.Generator().manual_seed(seed)
    B = len(lens)
    cols = max(-(-n // page) for n in lens), max(max(-(-(n // g) // page) for n in lens), 1)
    raw, core = torch.full((B, cols[0]), -1), torch.full((B, cols[1]), -1)
    at = [0, 0]
    for b, n in enumerate(lens):
        lo = max(n - 1 - w, 0) // g * g // page
        for t, i, a, z in ((raw, 0, lo, -(-n // page)), (core, 1, 0, -(-(n // g) // page))):
            t[b, a:z] = torch.arange(at[i], at[i] + z - a)
            at[i] += z - a
    pages = max(at[0], 1), max(at[1], 1)

    def pool(n, dtype, key):
        shape = (1, n, Hkv, page, d)
        x = torch.randint(-8, 9, shape, generator=gen) / 4 if key else \
            torch.randn(shape, generator=gen)
        return x.to(dtype).to(device)

    def ref(t, n):
        t = t[t >= 0]
        return torch.bincount(t, minlength=n).int()
    c = cca.PagedCache.from_tensors(
        core.int().to(device), raw.int().to(device), ref(core, pages[1]).to(device),
        ref(raw, pages[0]).to(device), torch.tensor(lens).to(device), pool(pages[1], F16, True),
        pool(pages[1], F16, False), pool(pages[0], BF, True), pool(pages[0], BF, False),
        Hq=Hq, g=g, w=w)
    q = torch.randint(-1, 2, (B, Hq, d), generator=gen).to(BF).to(device)
    return c, q


CASES = [  # lens, Hq, Hkv, d, g, w: raw rows alone, core rows and one raw one, both
    ([2, 3, 5, 9, 17, 40], 4, 2, 128, 16, 64), ([2, 3, 5, 9, 17, 40], 12, 1, 64, 16, 64),
    ([65, 129, 321, 641], 8, 2, 64, 16, 0), ([65, 129, 321, 641], 16, 1, 128, 16, 0),
    ([97, 200, 333], 3, 1, 128, 8, 20), ([97, 200, 333], 10, 1, 64, 8, 20),
]


def _emulated(c, q, b, split, up):
    """Row b with the weights in one or two numbers of their tiles' types,
    core ones relative to 2^-up of the largest."""
    (kc, vc), (kr, vr) = _seen(c, b)
    x = [q[b].to(F64).view(c.Hkv, -1, c.d) @ k.to(F64).transpose(1, 2) /
         (math.sqrt(c.d) * math.log(2)) for k in (kc, kr)]
    top = torch.cat(x, -1).amax(-1, keepdim=True)
    num, den = 0.0, 0.0
    for s, v, dtype, u in ((x[0], vc, F16, up), (x[1], vr, BF, 0)):
        p = torch.exp2(s - top + u)
        held = p.to(F32).to(dtype).to(F64)
        if split:
            held = held + (p - held).to(F32).to(dtype).to(F64)
        num, den = num + held @ v.to(F64) * 2.0 ** -u, den + p.sum(-1, keepdim=True) * 2.0 ** -u
    return (num / den).reshape(c.Hq, c.d)


@pytest.fixture(scope="module")
def built():
    cca_build.build()


@pytest.mark.parametrize("case", CASES, ids=str)
def test_the_bound_tells_one_number_from_two(built, case):
    c, q = _filled(*case, 16, "cpu")
    refs = [_reference(c, q, b) for b in range(c.B)]
    assert max(_off(_emulated(c, q, b, True, 15), r) for b, r in enumerate(refs)) <= 0.6
    assert max(_off(_emulated(c, q, b, False, 15), r) for b, r in enumerate(refs)) > 1.5


def _heavy(device, B, Hkv, N=3000):
    """One core key with nearly all the weight and a value of zero, N - 1 of
    2^-25.97 of it with values of 1000."""
    c, q = _filled([16 * N + 1] * B, Hkv, Hkv, 64, 16, 0, 64, device)
    for t in (*c.pools, q):
        t.zero_()
    q[:, :, 0] = 16
    c.v_core.fill_(1000)
    first = c.core_table[:, 0].long()
    c.k_core[0, first, :, 5, 0] = 9
    c.v_core[0, first, :, 5] = 0
    return c, q


def test_the_bound_tells_weights_that_fp16_loses(built):
    c, q = _heavy("cpu", 1, 1)
    ref = _reference(c, q, 0)
    assert 0.04 < float(ref[0].min()) and float(ref[0].max()) < 0.05
    assert _off(_emulated(c, q, 0, True, 15), ref) <= 0.6
    assert _off(_emulated(c, q, 0, True, 0), ref) > 100


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_outputs_within_the_bound(built, case):
    c, q = _filled(*case, 16, "cuda")
    o = cca.cca_attn_decode_paged(c, q, out_dtype=F32)
    assert cca.cca_device_status() == cca.CCA_OK
    for b in range(c.B):
        assert _off(o[b], _reference(c, q, b)) <= 1, b


def _infinite(c, at):
    """Values of raw rows: at[i] = (row, token, head, dim, value)."""
    for b, t, h, dim, x in at:
        page = int(c.raw_table[b, t // c.page])
        assert page >= 0
        c.v_raw[0, page, h, t % c.page, dim] = x


INF = float("inf")


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 128), (8, 1, 64), (12, 1, 128), (32, 2, 64)])
@pytest.mark.parametrize("lens,g,w", [([5, 33, 64], 16, 64), ([200, 90], 8, 40),
                                      ([9000, 7000, 1], 16, 1 << 30), ([20000], 16, 8000)])
def test_infinite_values(built, Hq, Hkv, d, lens, g, w):
    """An infinite value makes the outputs that see it infinite, as in the
    formula; infinities of both signs and NaN make them NaN; all others are
    what they were.  In one warp's tiles, and in many CTAs'."""
    c, q = _filled(lens, Hq, Hkv, d, g, w, 64, "cuda", seed=d)
    last, mid = lens[0] - 1, lens[0] - min(lens[0], w) // 2 - 1
    _infinite(c, [(0, last, 0, 3, INF), (0, mid, 0, 40, -INF), (0, last, Hkv - 1, d - 1, INF),
                  (0, mid, Hkv - 1, d - 1, -INF), (0, mid, 0, 17, float("nan")),
                  (len(lens) - 1, lens[-1] - 1, 0, 0, -INF)])
    o = cca.cca_attn_decode_paged(c, q, out_dtype=F32)
    assert cca.cca_device_status() == cca.CCA_OK
    seen = torch.zeros(3, dtype=torch.int64)
    for b in range(c.B):
        ref = _reference(c, q, b)
        for i, kind in enumerate((torch.isnan, torch.isposinf, torch.isneginf)):
            assert torch.equal(kind(o[b]), kind(ref[0])), (b, kind)
            seen[i] += int(kind(ref[0]).sum())
        fine = torch.isfinite(ref[0])
        zeros = [torch.where(fine, x, 0.0) for x in (o[b], *ref[:3])]
        assert _off(zeros[0], (*zeros[1:], *ref[3:])) <= 1, b
    r = Hq // Hkv
    assert seen.tolist() == [2 * r, r, 2 * r]


@pytest.mark.gpu
@pytest.mark.parametrize("Hq", [2, 24])
def test_infinite_value_of_the_newest_token(built, Hq):
    c, q = _filled([30, 100], Hq, 2, 64, 16, 1 << 30, 16, "cuda")
    k, v = (torch.zeros((2, 2, 64), dtype=BF, device="cuda") for _ in range(2))
    v[1, 0, 9], v[0, 1, 50] = INF, -INF
    o = cca.cca_paged_step(c, q, k, v, out_dtype=F32)
    assert cca.cca_device_status() == cca.CCA_OK
    for b in range(2):
        ref = _reference(c, q, b)[0]
        assert torch.equal(torch.isinf(o[b]), torch.isinf(ref))
        assert torch.equal(o[b].sign()[torch.isinf(ref)], ref.float().sign()[torch.isinf(ref)])
        assert not bool(torch.isnan(o[b]).any())


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hkv", [(1, 1), (8, 16)])  # a tile for each warp, and many
def test_light_core_rows_behind_a_heavy_one(built, B, Hkv):
    c, q = _heavy("cuda", B, Hkv)
    o = cca.cca_attn_decode_paged(c, q, out_dtype=F32)
    assert cca.cca_device_status() == cca.CCA_OK
    for b in range(B):
        assert _off(o[b], _reference(c, q, b)) <= 1, b
