"""Calls of several host threads.  A kernel's allowance of shared memory is
the process's: a call that sets it to its own size may lower it between
another thread's setting and that thread's launch, which then fails."""

import glob
import os
import re
import threading

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_allowances_do_not_depend_on_the_call():
    """Each is the same value whatever the call's sizes are."""
    values = []
    for path in glob.glob(os.path.join(ROOT, "long_context_sparse_cca_b200", "csrc", "*")):
        with open(path) as f:
            text = f.read()
        values += re.findall(r"cudaFuncAttributeMaxDynamicSharedMemorySize,\s*([^;]*);", text)
    assert len(values) >= 4
    for v in values:  # the kernels' own constants, or all that an SM has beside them
        assert re.match(r"(C|LQ|LK)::SMEM(_PK)?\)|static_cast<int>\(kSmemMost - own\)\)", v), v


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["step", "pool", "mixed"])
def test_two_threads_with_other_sizes(what):
    """Two host threads launch the same kernels with other amounts of shared
    memory, each on a stream of its own."""
    import torch
    import long_context_sparse_cca_b200 as cca
    from long_context_sparse_cca_b200 import build
    build.build()
    BF, N = torch.bfloat16, 4000

    def steps(B):  # free rows: nothing but zero outputs
        c = cca.PagedCache(B, 1, 1, 64, 16, 64, 16, 8, 16, 64)
        q, o = torch.zeros((B, 1, 64), dtype=BF, device="cuda"), []

        def run(stream):
            o.append(torch.full_like(q, 1.0))
            for _ in range(N):
                cca.cca_paged_step(c, q, q, q, o_t=o[0], stream=stream)
        return run, lambda: bool((o[0] == 0).all())

    def pools(S):
        q, k = (torch.ones((h, 512, 64), dtype=BF, device="cuda") for h in (4, 1))
        cu = torch.full((S + 1,), 512, dtype=torch.int32, device="cuda")
        cu[0] = 0
        out = [torch.zeros((1, 2, 64), dtype=torch.float16, device="cuda") for _ in range(2)]

        def run(stream):
            for _ in range(N):
                cca.cca_pool_packed(q, k, k, cu, 256, *out, stream=stream)
        return run, lambda: all(bool((x == 1).all()) for x in out)

    jobs = {"step": [steps(2), steps(2900)], "pool": [pools(2500), pools(8000)],
            "mixed": [steps(5), steps(2500), pools(2600), pools(7000)]}[what]
    streams, failed = [torch.cuda.Stream() for _ in jobs], []
    torch.cuda.synchronize()

    def work(run, stream):
        try:
            run(stream)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(run, s)) for (run, _), s in zip(jobs, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    assert all(check() for _, check in jobs)
    assert cca.cca_device_status() == cca.CCA_OK
