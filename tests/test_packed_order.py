"""Packed prompts in the orders in which the attention kernel takes its
blocks: head by head where what a query looks back into exceeds half the L2,
and every other round of the CTAs backwards where there are few rounds.  Each
case is large enough to reach its order; the outputs are, bit for bit, those
of one sequence after the other, which are tested against the oracle."""

import numpy as np
import pytest
import torch

import long_context_sparse_cca_b200 as cca
from long_context_sparse_cca_b200 import build as cca_build

pytestmark = pytest.mark.gpu
ALL = 1 << 30


@pytest.fixture(scope="module")
def built():
    cca_build.build()


def _check(lens, Hq, Hkv, d, g, w, every=1):
    total = sum(lens)
    gen = torch.Generator(device="cuda").manual_seed(total)
    Q, K, V = (torch.randn((h, total, d), generator=gen, device="cuda").to(torch.bfloat16)
               for h in (Hq, Hkv, Hkv))
    at = np.concatenate([[0], np.cumsum(lens)])
    cu = torch.tensor(at, dtype=torch.int32, device="cuda")
    kc, vc = cca.cca_pool_packed(Q, K, V, cu, g)
    O = torch.full_like(Q, float("nan"))
    cca.cca_attn_prefill_packed(Q, K, V, kc, vc, cu, g, w, O=O)
    assert cca.cca_device_status() == cca.CCA_OK
    assert bool(torch.isfinite(O).all())  # every block was taken
    for s in range(0, len(lens), every):
        a, b = int(at[s]), int(at[s + 1])
        x = [t[None, :, a:b].contiguous() for t in (Q, K, V)]
        assert torch.equal(O[:, a:b], cca.cca_attn_prefill(*x, *cca.cca_pool(*x, g), g, w)[0]), s


def _many(n, most, seed):
    """n lengths of 1 to `most`, short ones among them."""
    rng = np.random.default_rng(seed)
    return [int(x) for x in np.exp(rng.uniform(0, np.log(most), size=n))]


@pytest.mark.parametrize("lens,g,w", [
    ([1500, 2500, 1, 400], 16, ALL),                  # each CTA orders the blocks
    (_many(70, 250, 1) + [1800, 700, 513], 16, ALL),  # a kernel does
    ([5000, 257, 3500, 43], 2, 10),                   # core rows of all heads
    (_many(80, 300, 2) + [5600], 2, 10),
], ids=["causal", "causal-list", "core", "core-list"])
def test_head_by_head(built, lens, g, w):
    Hkv, d = 32, 128
    if w == ALL:
        lens = lens + [max(1, 4200 - sum(lens))]
    else:
        lens = lens + [max(1, 8600 - sum(lens))]
    far = sum(lens) if w == ALL else sum(lens) // g
    assert 4 * Hkv * far * d > torch.cuda.get_device_properties(0).L2_cache_size / 2
    _check(lens, Hkv, Hkv, d, g, w, every=1 if len(lens) < 20 else 9)


@pytest.mark.parametrize("lens,Hq,Hkv,d,g,w", [
    ([2000, 1777, 900, 33, 1400, 1024, 1, 1057], 16, 4, 64, 16, ALL),
    ([3000, 200, 1], 24, 8, 128, 16, 64),
    ([256 * 11 + 1], 31, 1, 64, 32, 300),
    (_many(66, 500, 3), 6, 2, 64, 8, 40),  # the order of a kernel
    ([1100] * 20, 9, 3, 128, 16, ALL),
], ids=str)
def test_rounds_backwards(built, lens, Hq, Hkv, d, g, w):
    """At least two rounds and at most eight, the last one not full."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    items = sum(-(-n // 256) for n in lens) * Hq
    assert 2 * sms <= items and items % sms != 0
    assert (sum(lens) // 256 + len(lens)) * Hq <= 8 * sms
    _check(lens, Hq, Hkv, d, g, w, every=1 if len(lens) < 20 else 9)


def test_list_in_a_workspace_of_the_callers(built):
    """More than 64 sequences, in a captured graph with a workspace of the
    caller's: each replay makes the list anew, from the offsets it finds."""
    S, d, g, w = 70, 64, 8, 40
    gen = torch.Generator(device="cuda").manual_seed(7)
    total = 9000
    Q, K, V = (torch.randn((h, total, d), generator=gen, device="cuda").to(torch.bfloat16)
               for h in (4, 2, 2))
    cu = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    n = cca.cca_packed_workspace_bytes(S, total)
    assert n > 0
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
    core = [torch.zeros((2, total // g, d), dtype=torch.float16, device="cuda") for _ in range(2)]
    O = torch.zeros_like(Q)

    def run(**kw):
        cca.cca_pool_packed(Q, K, V, cu, g, *core)
        return cca.cca_attn_prefill_packed(Q, K, V, *core, cu, g, w, **kw)
    run(O=O, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(O=O, workspace=ws)
    for seed in range(4):
        lens = _many(S, 900, 20 + seed)
        at = np.minimum(np.concatenate([[0], np.cumsum(lens)]) + 5 * seed, total)
        cu.copy_(torch.tensor(at, dtype=torch.int32))
        O.zero_()
        graph.replay()
        got = O.clone()
        want = torch.zeros_like(Q)
        run(O=want)
        assert torch.equal(got, want), seed
        assert bool((got[:, at[0]:at[-1]] != 0).any(-1).all())
    with pytest.raises(cca.CCAError):
        run(O=O, workspace=ws[:n - 1])
    assert cca.cca_device_status() == cca.CCA_OK
