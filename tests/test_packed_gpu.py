"""Packed prompts (cca_pool_packed, cca_attn_prefill_packed) through the
C ABI against the fp64 oracle, each sequence by itself.

Tolerances are the suite's (gpu_util): the tensor cores take P rounded to
bf16, at most 2^-9 of each weight, so an output is off by at most
2^-9 max |v| <= 2^-9 * 4.6 < 1e-2 for the normal values used here (4.6: the
largest of a million); the pooled rows are fp32 sums rounded to fp16.  A
packed call and the call on one sequence alone run the same arithmetic in
the same order, so those agree bit for bit.
"""

import numpy as np
import pytest

import oracle
from gpu_util import assert_close, to_cuda, to_f64
from long_context_sparse_cca_b200 import synth
from serving_model import packed_inputs

pytestmark = pytest.mark.gpu
ALL = 1 << 30


@pytest.fixture(scope="module")
def cca():
    from long_context_sparse_cca_b200 import build
    build.build()
    import long_context_sparse_cca_b200 as m
    return m


def _i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _layout(x, layout):
    """[H, total, d] in one of the memory orders that occur."""
    import torch
    if layout == "head":
        return x
    if layout == "token":
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    H, n, d = x.shape  # heads of a wider projection, rows with a gap
    wide = torch.full((n, H + 3, d), float("nan"), dtype=x.dtype, device=x.device)
    wide[:, 1:H + 1] = x.transpose(0, 1)
    return wide[:, 1:H + 1].transpose(0, 1)


CASES = [
    ([5, 1, 128, 77], 2, 2, 64, 16, 64, "head", 0, 0),
    ([1], 1, 1, 128, 16, 64, "head", 0, 0),
    ([300, 0, 0, 513, 2, 0], 4, 2, 128, 8, 40, "token", 7, 70),
    ([257, 255, 256, 1], 6, 2, 64, 32, 100, "wide", 3, 0),
    ([700, 31], 3, 1, 128, 1, 10, "token", 0, 1),
    ([129, 2000], 2, 1, 128, 24, 100, "head", 11, 300),
    ([900, 33, 1024, 1], 4, 4, 64, 16, ALL, "wide", 2, 3),
    ([15, 15, 15, 16, 17], 2, 2, 128, 16, 0, "token", 0, 0),
    ([2500], 16, 1, 64, 256, 300, "head", 5, 5),
]


@pytest.mark.parametrize("case", CASES, ids=[str(c) for c in CASES])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_packed_matches_oracle(cca, case, out):
    import torch
    lens, Hq, Hkv, d, g, w, layout, lead, trail = case
    q, k, v, cu = packed_inputs(lens, Hq, Hkv, d, 100 + len(lens), lead, trail)
    total = q.shape[1]
    nobody = np.ones(total, bool)
    nobody[cu[0]:cu[-1]] = False
    Q, K, V = (to_cuda(x) for x in (q, k, v))
    for x in (Q, K, V):  # rows that no sequence owns hold anything
        x[:, torch.from_numpy(nobody).cuda()] = float("nan")
    Q, K, V = (_layout(x, layout) for x in (Q, K, V))
    cu_d = torch.from_numpy(cu).cuda()
    core = w < total
    Kc = Vc = None
    if core:
        Kc, Vc = (torch.full((Hkv, total // g, d), 7.0, dtype=torch.float16, device="cuda")
                  for _ in range(2))
        cca.cca_pool_packed(Q, K, V, cu_d, g, Kc, Vc)
    dt = torch.float32 if out == "f32" else torch.bfloat16
    O = _layout(torch.full((Hq, total, d), 3.0, dtype=dt, device="cuda"),
                "head" if layout == "head" else "token")
    cca.cca_attn_prefill_packed(Q, K, V, Kc, Vc, cu_d, g, w, O=O)
    assert cca.cca_device_status() == cca.CCA_OK
    assert bool((O[:, torch.from_numpy(nobody).cuda()] == 3.0).all()), "rows of no sequence"
    seen = np.zeros(total // g, bool)
    for s, n in enumerate(lens):
        a, b = int(cu[s]), int(cu[s + 1])
        if n == 0:
            continue
        qs, ks, vs = (synth.bf16_bits_to_f64(np.ascontiguousarray(x[None, :, a:b])) for x in (q, k, v))
        c = slice(a // g, a // g + n // g)
        seen[c] = True
        if core and n >= g:
            Kr, Vr = oracle.pool(qs, ks, vs, g)
            assert_close(Kc[:, c], Kr[0], None, f"Kc of sequence {s}")
            assert_close(Vc[:, c], Vr[0], None, f"Vc of sequence {s}")
        ref = oracle.prefill(qs, ks, vs, g, min(w, total))[0]
        assert_close(O[:, a:b].contiguous(), ref, None, f"O of sequence {s}")
    if core:
        empty = torch.from_numpy(~seen).cuda()
        assert bool((Kc[:, empty] == 0).all()) and bool((Vc[:, empty] == 0).all())


@pytest.mark.parametrize("d,g,w", [(128, 16, 64), (64, 32, 250)])
def test_packed_equals_one_sequence_at_a_time(cca, d, g, w):
    """Bit for bit, also with a sequence of NaN and infinities next to it."""
    import torch
    lens, Hq, Hkv = [333, 200, 1, 700], 4, 2
    q, k, v, cu = packed_inputs(lens, Hq, Hkv, d, 900)
    Q, K, V = (to_cuda(x) for x in (q, k, v))
    for x, bad in ((Q, float("nan")), (K, float("inf")), (V, float("nan"))):
        x[:, cu[1]:cu[2]] = bad
    cu_d = torch.from_numpy(cu).cuda()
    Kc, Vc = cca.cca_pool_packed(Q, K, V, cu_d, g)
    O = cca.cca_attn_prefill_packed(Q, K, V, Kc, Vc, cu_d, g, w)
    assert cca.cca_device_status() in (cca.CCA_OK, cca.CCA_ERR_RANGE)  # the sequence of NaN
    for s in (0, 2, 3):
        a, b = int(cu[s]), int(cu[s + 1])
        x = [t[None, :, a:b].contiguous() for t in (Q, K, V)]
        kc, vc = cca.cca_pool(*x, g)
        o = cca.cca_attn_prefill(*x, kc, vc, g, w)
        c = slice(a // g, a // g + lens[s] // g)
        assert torch.equal(Kc[:, c], kc[0]) and torch.equal(Vc[:, c], vc[0]), s
        assert torch.equal(O[:, a:b], o[0]), s
    assert cca.cca_device_status() == cca.CCA_OK


def test_many_sequences(cca):
    """As many sequences as a call takes, most of one token: each token is
    its own output (softmax over itself)."""
    import torch
    S, d = 8192, 64
    lens = [1] * S
    lens[100], lens[5000] = 300, 0
    q, k, v, cu = packed_inputs(lens, 2, 1, d, 77)
    Q, K, V = (to_cuda(x) for x in (q, k, v))
    cu_d = torch.from_numpy(cu).cuda()
    Kc, Vc = cca.cca_pool_packed(Q, K, V, cu_d, 16)
    O = cca.cca_attn_prefill_packed(Q, K, V, Kc, Vc, cu_d, 16, 64)
    assert cca.cca_device_status() == cca.CCA_OK
    one = torch.ones(q.shape[1], dtype=torch.bool)
    one[100:400] = False
    one = one.cuda()
    assert torch.equal(O[:, one], V.expand(2, -1, -1)[:, one])
    qs, ks, vs = (synth.bf16_bits_to_f64(np.ascontiguousarray(x[None, :, 100:400])) for x in (q, k, v))
    assert_close(O[:, 100:400].contiguous(), oracle.prefill(qs, ks, vs, 16, 64)[0], None, "O")


@pytest.mark.parametrize("cu", [[-1, 5, 20], [0, 9, 5], [0, 10, 21], [5, 2, 20]], ids=str)
def test_bad_offsets_write_nothing(cca, cu):
    import torch
    q, k, v, _ = packed_inputs([20], 2, 2, 64, 5)
    Q, K, V = (to_cuda(x) for x in (q, k, v))
    cu_d = torch.tensor(cu, dtype=torch.int32, device="cuda")
    Kc, Vc = (torch.full((2, 5, 64), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    O = torch.full((2, 20, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    cca.cca_pool_packed(Q, K, V, cu_d, 4, Kc, Vc)
    assert cca.cca_device_status() == cca.CCA_ERR_SEQLENS
    cca.cca_attn_prefill_packed(Q, K, V, Kc, Vc, cu_d, 4, 8, O=O)
    assert cca.cca_device_status() == cca.CCA_ERR_SEQLENS
    assert bool((Kc == 7).all()) and bool((Vc == 7).all()) and bool((O == 3).all())
    assert cca.cca_device_status() == cca.CCA_OK


def test_packed_replayed_graph_follows_new_offsets(cca):
    """A captured call reads the offsets on the device: the same graph, other
    lengths; and a call on a side stream."""
    import torch
    d, g, w = 64, 16, 64
    q, k, v, cu = packed_inputs([400, 300], 2, 2, d, 40)
    Q, K, V = (to_cuda(x) for x in (q, k, v))
    cu_d = torch.from_numpy(cu).cuda()
    O = torch.zeros_like(Q)
    run = lambda: cca.cca_attn_prefill_packed(  # noqa: E731
        Q, K, V, *cca.cca_pool_packed(Q, K, V, cu_d, g), cu_d, g, w, O=O)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for other in ([0, 400, 700], [0, 1, 700], [200, 200, 650]):
        cu_d.copy_(torch.tensor(other, dtype=torch.int32))
        O.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        got = O.clone()
        O.fill_(3.0)
        run()
        assert torch.equal(got, O), other
    assert cca.cca_device_status() == cca.CCA_OK


def test_packed_stream_argument(cca):
    import torch
    q, k, v, cu = packed_inputs([500, 200], 2, 2, 128, 41)
    Q, K, V = (to_cuda(x) for x in (q, k, v))
    cu_d = torch.from_numpy(cu).cuda()
    Kc, Vc = cca.cca_pool_packed(Q, K, V, cu_d, 16)
    O = cca.cca_attn_prefill_packed(Q, K, V, Kc, Vc, cu_d, 16, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Kc2, Vc2 = cca.cca_pool_packed(Q, K, V, cu_d, 16, stream=side)
    O2 = cca.cca_attn_prefill_packed(Q, K, V, Kc2, Vc2, cu_d, 16, 64, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(O, O2) and torch.equal(Kc, Kc2)
    assert to_f64(O).shape == (2, 700, 128)


def test_nothing_to_do(cca):
    """No rows at all, and rows that no sequence owns: outputs stay as they
    were."""
    import torch
    Q, K = (torch.zeros((h, 0, 64), dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    none = _i32([0, 0])
    Kc, Vc = cca.cca_pool_packed(Q, K, K, none, 16)
    assert Kc.shape == Vc.shape == (2, 0, 64)
    assert cca.cca_attn_prefill_packed(Q, K, K, Kc, Vc, none, 16, 64).shape == (4, 0, 64)
    Q, K = (torch.full((h, 300, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
            for h in (4, 2))
    for cu in ([0, 0, 0], [300, 300], [17, 17, 17, 17]):
        Kc, Vc = cca.cca_pool_packed(Q, K, K, _i32(cu), 16)
        assert bool((Kc == 0).all()) and bool((Vc == 0).all())
        O = torch.full_like(Q, 3.0)
        cca.cca_attn_prefill_packed(Q, K, K, Kc, Vc, _i32(cu), 16, 64, O=O)
        assert bool((O == 3).all())
    assert cca.cca_device_status() == cca.CCA_OK


@pytest.mark.parametrize("S", [64, 65])
def test_block_order_by_every_cta_or_by_a_kernel(cca, S):
    """On both sides of the border the same result, bit for bit, as one
    sequence after the other."""
    import torch
    rng = np.random.default_rng(S)
    lens = rng.integers(1, 700, size=S)
    lens[0] = 900
    q, k, v, cu = packed_inputs(lens.tolist(), 2, 1, 64, S)
    assert (cca.cca_packed_workspace_bytes(S, q.shape[1]) > 0) == (S > 64)
    Q, K, V = (to_cuda(x) for x in (q, k, v))
    Kc, Vc = cca.cca_pool_packed(Q, K, V, _i32(cu.tolist()), 16)
    O = cca.cca_attn_prefill_packed(Q, K, V, Kc, Vc, _i32(cu.tolist()), 16, 64)
    for s in range(0, S, 7):
        a, b = int(cu[s]), int(cu[s + 1])
        x = [t[None, :, a:b].contiguous() for t in (Q, K, V)]
        assert torch.equal(O[:, a:b], cca.cca_attn_prefill(*x, *cca.cca_pool(*x, 16), 16, 64)[0])
    assert cca.cca_device_status() == cca.CCA_OK
