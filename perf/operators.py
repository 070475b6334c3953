"""The serving operators of this library, measured: attention of packed prompts, one decode step
over a paged cache, and the upkeep of that cache's pages.

The method is CCA-Attention's: a query t of a sequence sees the core keys of the groups j < ws(t)/g
and the raw keys ws(t) .. t under one softmax, ws(t) = g * floor(max(t - w, 0) / g); the core row of
group j is the mean of its g key and value rows weighted by softmax(q . k / sqrt(d)) of the query of
its last token (mean over the query heads that share a key/value head).  A window w that covers the
whole sequence is plain causal attention.

Packed prompts: Q [Hq, total, d], K and V [Hkv, total, d], sequence s in rows cu[s] .. cu[s + 1] - 1;
its core rows start at row cu[s] // g of Kc, Vc [Hkv, total // g, d], other rows of them are zero.

Paged cache: pools of pages of `page` rows for every key/value head, core rows (fp16) in one pool,
raw rows (bf16) in the other: [layers, pages, Hkv, page, d].  Row b of a batch holds lens[b] tokens;
core row j of it is row j % page of page core_table[b, j // page], token p is row p % page of page
raw_table[b, p // page]; an entry without a page is -1.  A reference count per page says how many
table entries name it; a page with count 0 is free.  New pages are the free ones of lowest number,
in the order of the batch's rows.
"""

import math
import random

import numpy as np
import torch

own = False

LAYOUTS = ("head", "token")  # memory order of Q, K, V and O: [H, total, d] or [total, H, d]
ALL = 1 << 30                # a window over everything: plain causal attention


def listed():
    return [
        # the smallest prompts: a few short ones at a small model's heads; latency counts
        dict(name="prompt small", kind="prompt", Hq=2, Hkv=2, d=64, g=16, w=64, lens="5,1,128,77",
             layout="head", page=0),
        # an ordinary batch of prompts of very different lengths, grouped heads, as the projections
        # leave them in memory, and the filling of their cache pages
        dict(name="prompt ragged", kind="prompt", Hq=32, Hkv=8, d=128, g=32, w=2048,
             lens="7001,3,4096,1500,2783,1001", layout="token", page=64),
        # one long prompt and a single token: the long end of the range
        dict(name="prompt long", kind="prompt", Hq=32, Hkv=32, d=128, g=16, w=1024,
             lens="32768,1", layout="head", page=0),
        # layers that keep full causal attention, beside the ones that do not
        dict(name="prompt causal", kind="prompt", Hq=16, Hkv=4, d=64, g=16, w=ALL,
             lens="2000,1777,900,33,1400,1024,1,1057", layout="token", page=0),
        # one conversation, short: latency; its token completes a group
        dict(name="step one", kind="step", Hq=32, Hkv=8, d=128, g=16, w=1024, lens="784",
             page=64),
        # a batch at 64K tokens of context: the bandwidth case
        dict(name="step batch", kind="step", Hq=32, Hkv=32, d=128, g=16, w=1024,
             lens="65537,65552,65570,65600,65700,65777,65791,65792", page=64),
        # continuous batching: rows of every length, grouped heads
        dict(name="step ragged", kind="step", Hq=32, Hkv=8, d=128, g=32, w=2048, page=32,
             lens=",".join(str(int(16384 ** (i / 63.0))) for i in range(64))),
        # full causal attention of one token over long pages of small heads
        dict(name="step causal", kind="step", Hq=16, Hkv=2, d=64, g=16, w=ALL, page=16,
             lens="32768,32001,30000,25555,20000,16384,12000,9999,8192,5000,3000,2047,1000,100,17,1"),
        # eight beams of one conversation take over the best one's pages
        dict(name="fork beams", kind="fork", Hkv=8, d=128, g=16, w=1024, page=64, layers=2,
             lens="1500", copies=8, core_pages=64, raw_pages=256),
        # sixteen prompts, four samples of each, at a model's four layers
        dict(name="fork samples", kind="fork", Hkv=8, d=128, g=16, w=1024, page=64, layers=4,
             lens="1037,2049,3000,4111,5008,6600,7777,8191,9001,10100,11111,12345,13579,14444,15001,16001",
             copies=4, core_pages=512, raw_pages=1024),
        # a small pool with holes after a few conversations ended
        dict(name="compact small", kind="compact", Hkv=2, d=64, g=16, w=64, page=16, layers=2,
             B=8, core_pages=64, raw_pages=128, live=0.4, longest=900),
        # a large pool that shrinks after a burst of load
        dict(name="compact large", kind="compact", Hkv=8, d=128, g=16, w=1024, page=64, layers=4,
             B=24, core_pages=512, raw_pages=1024, live=0.4, longest=16000),
    ]


def _between(rng, lo, hi):
    """A whole number, spread over the range's logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("prompt", "prompt", "step", "step", "fork", "compact"))
    d = rng.choice((64, 128))
    if kind == "prompt":
        Hq, Hkv = rng.choice(((2, 2), (6, 2), (8, 1), (12, 12), (16, 4), (32, 8)))
        g, w = rng.choice(((16, 64), (16, 1024), (32, 2048), (8, 250), (24, 100), (16, ALL)))
        lens = [_between(rng, 1, 8000 if w != ALL else 2000) for _ in range(rng.randint(1, 10))]
        page = rng.choice((0, 0, 16, 64)) if w != ALL else 0
        return dict(kind=kind, Hq=Hq, Hkv=Hkv, d=d, g=g, w=w, lens=",".join(map(str, lens)),
                    layout=rng.choice(LAYOUTS), page=page)
    page = rng.choice((16, 32, 64, 128))
    if kind == "step":
        Hq, Hkv = rng.choice(((1, 1), (6, 2), (16, 1), (16, 2), (32, 8), (32, 32)))
        g, w = rng.choice(((16, 64), (16, 1024), (32, 2048), (8, 250), (24, 100), (16, ALL)))
        most = 65536 if w != ALL else 16384
        lens = [_between(rng, 1, most) for _ in range(_between(rng, 1, 32 if Hkv < 32 else 4))]
        return dict(kind=kind, Hq=Hq, Hkv=Hkv, d=d, g=g, w=w, lens=",".join(map(str, lens)),
                    page=page)
    Hkv, layers = rng.choice((1, 2, 5, 8)), rng.randint(1, 4)
    g, w = rng.choice(((16, 64), (16, 1024), (8, 250)))
    if kind == "fork":
        lens = [_between(rng, 1, 16000) for _ in range(_between(rng, 1, 12))]
        return dict(kind=kind, Hkv=Hkv, d=d, g=g, w=w, page=page, layers=layers,
                    lens=",".join(map(str, lens)), copies=rng.randint(2, 8),
                    core_pages=sum(n // g // page + 1 for n in lens) + 8 * len(lens) * 3,
                    raw_pages=(len(lens) * (w + g)) // page + 8 * len(lens) * 4)
    B = _between(rng, 1, 24)
    return dict(kind=kind, Hkv=Hkv, d=d, g=g, w=w, page=page, layers=layers, B=B,
                core_pages=_between(rng, 24, 512), raw_pages=_between(rng, 48, 1024),
                live=round(rng.uniform(0.1, 0.9), 3), longest=_between(rng, 40, 16000))


# ---------------------------------------------------------------- inputs

def _ints(text):
    return [int(x) for x in text.split(",")]


def _window_start(t, g, w):
    return max(t - w, 0) // g * g


def _pooled(case, total):
    """Whether a pass over prompts pools: some window ends before the first token, or a cache is filled."""
    return case["w"] < total or case["page"] > 0


def _rows(lens, g, w, page):
    """Host view of a batch: per row the range of raw columns and the number of core columns."""
    raw = [(_window_start(n - 1, g, w) // page, -(-n // page)) if n else (0, 0) for n in lens]
    core = [-(-(n // g) // page) for n in lens]
    return raw, core


def _compact_lens(case):
    """Rows of as many tokens as the share of the pools in use allows."""
    rng = random.Random(case["B"] * 1000 + case["core_pages"])
    lens = [_between(rng, 1, case["longest"]) for _ in range(case["B"])]
    fit = lambda n: (sum(n[1]) <= case["live"] * case["core_pages"]  # noqa: E731
                     and sum(hi - lo for lo, hi in n[0]) <= case["live"] * case["raw_pages"])
    while not fit(_rows(lens, case["g"], case["w"], case["page"])):
        lens = [n * 7 // 8 if n > case["page"] else 0 for n in lens]
    return lens


def _tables(lens, g, w, page, rng, spread=1.0):
    """Tables of a batch whose pages lie scattered over the pools, as they do after hours of use."""
    raw, core = _rows(lens, g, w, page)
    raw_table = np.full((len(lens), max([hi for _, hi in raw] + [1]) + 1), -1, np.int32)
    core_table = np.full((len(lens), max(core + [1]) + 1), -1, np.int32)
    n_raw, n_core = sum(hi - lo for lo, hi in raw), sum(core)
    raw_pages, core_pages = int(n_raw * spread) + 1, int(n_core * spread) + 1
    ids, at = rng.permutation(raw_pages), 0
    for b, (lo, hi) in enumerate(raw):
        raw_table[b, lo:hi] = ids[at:at + hi - lo]
        at += hi - lo
    ids, at = rng.permutation(core_pages), 0
    for b, n in enumerate(core):
        core_table[b, :n] = ids[at:at + n]
        at += n
    return core_table, raw_table, core_pages, raw_pages


def _counts(table, pages):
    return np.bincount(table[table >= 0], minlength=pages).astype(np.int32)


def _gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _normal(gen, shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _pools(gen, case, layers, core_pages, raw_pages):
    shape = lambda n: (layers, n, case["Hkv"], case["page"], case["d"])  # noqa: E731
    return (torch.empty(shape(core_pages), dtype=torch.float16, device="cuda").normal_(0, 0.5, generator=gen),
            torch.empty(shape(core_pages), dtype=torch.float16, device="cuda").normal_(0, 0.5, generator=gen),
            torch.empty(shape(raw_pages), dtype=torch.bfloat16, device="cuda").normal_(generator=gen),
            torch.empty(shape(raw_pages), dtype=torch.bfloat16, device="cuda").normal_(generator=gen))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    s = dict(case)
    if case["kind"] == "prompt":
        s["lens"] = lens = _ints(case["lens"])
        Hq, Hkv, d, g, total = case["Hq"], case["Hkv"], case["d"], case["g"], sum(_ints(case["lens"]))
        s["cu"] = _gpu(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
        for name, H in (("Q", Hq), ("K", Hkv), ("V", Hkv)):
            x = _normal(gen, (H, total, d) if case["layout"] == "head" else (total, H, d))
            if name == "K":  # one key row in a hundred stands out, as in trained models
                heavy = torch.rand(x.shape[:2] + (1,), generator=gen, device="cuda") < 0.01
                x = torch.where(heavy, x * 4, x)
            s[name] = x if case["layout"] == "head" else x.transpose(0, 1)
        if case["page"]:
            ct, rt, core_pages, raw_pages = _tables(lens, g, case["w"], case["page"], rng)
            s["tables"] = (_gpu(ct), _gpu(rt), _gpu(_counts(ct, core_pages)),
                           _gpu(_counts(rt, raw_pages)), _gpu(np.array(lens, np.int64)))
            s["pools"] = _pools(gen, case, 1, core_pages, raw_pages)
            s["rows"] = _gpu(np.arange(len(lens), dtype=np.int32))
            at = [(i, j, sum(lens[:i]) // g + j) for i, n in enumerate(lens) for j in range(n // g)]
            s["core_at"] = _gpu(np.array(at, np.int64).reshape(-1, 3).T)
    elif case["kind"] == "step":
        s["lens"] = lens = _ints(case["lens"])
        B, Hq, Hkv, d = len(lens), case["Hq"], case["Hkv"], case["d"]
        ct, rt, core_pages, raw_pages = _tables(lens, case["g"], case["w"], case["page"], rng)
        s["tables"] = (_gpu(ct), _gpu(rt), _gpu(_counts(ct, core_pages)),
                       _gpu(_counts(rt, raw_pages)), _gpu(np.array(lens, np.int64)))
        s["pools"] = _pools(gen, case, 1, core_pages, raw_pages)
        s["q_t"] = _normal(gen, (B, Hq, d))
        s["k_t"], s["v_t"] = _normal(gen, (B, Hkv, d)), _normal(gen, (B, Hkv, d))
        s["done"] = _gpu(np.array([b for b, n in enumerate(lens) if n % case["g"] == 0], np.int64))
    elif case["kind"] == "fork":
        # row i * copies holds a sequence, the other copies - 1 rows behind it hold what an earlier
        # fork of it left there: sequences of their own, of the same length
        parents, copies = _ints(case["lens"]), case["copies"]
        s["lens"] = lens = [n for n in parents for _ in range(copies)]
        raw, core = _rows(lens, case["g"], case["w"], case["page"])
        core_pages, raw_pages, cols = case["core_pages"], case["raw_pages"], case["page"]
        ct = np.full((len(lens), max(lens) // case["g"] // cols + 3), -1, np.int32)
        rt = np.full((len(lens), max(lens) // cols + 3), -1, np.int32)
        for table, pages, of in ((ct, core_pages, [(0, n) for n in core]), (rt, raw_pages, raw)):
            free = list(rng.permutation(pages))
            for b, (lo, hi) in enumerate(of):
                table[b, lo:hi] = table[b - 1, lo:hi] if b % copies else [free.pop() for _ in range(hi - lo)]
                if b % copies and hi > lo:  # its last page is its own
                    table[b, hi - 1] = free.pop()
        s["tables"] = (_gpu(ct), _gpu(rt), _gpu(_counts(ct, core_pages)),
                       _gpu(_counts(rt, raw_pages)), _gpu(np.array(lens, np.int64)))
        s["parent"] = _gpu(np.array([b // copies * copies for b in range(len(lens))], np.int32))
        copied = [[b for b, n in enumerate(lens) if b % copies and m(n) % cols]
                  for m in (lambda n: n // case["g"], lambda n: n)]
        s["copied"] = [_gpu(np.array(x, np.int64)) for x in copied]
        s["pools"] = _pools(gen, case, case["layers"], core_pages, raw_pages)
    else:
        B, g, w, page = case["B"], case["g"], case["w"], case["page"]
        s["lens"] = lens = _compact_lens(case)
        ct = np.full((B, case["longest"] // g // page + 2), -1, np.int32)
        rt = np.full((B, case["longest"] // page + 2), -1, np.int32)
        raw, core = _rows(lens, g, w, page)
        s["moved"] = []
        for table, pages, of in ((ct, case["core_pages"], [(0, n) for n in core]),
                                 (rt, case["raw_pages"], raw)):
            ids, at = rng.permutation(pages), 0
            for b, (lo, hi) in enumerate(of):
                table[b, lo:hi] = ids[at:at + hi - lo]
                at += hi - lo
            s["moved"].append(int((ids[:at] >= at).sum()))
        s["tables"] = (_gpu(ct), _gpu(rt), _gpu(_counts(ct, case["core_pages"])),
                       _gpu(_counts(rt, case["raw_pages"])), _gpu(np.array(lens, np.int64)))
        s["pools"] = _pools(gen, case, case["layers"], case["core_pages"], case["raw_pages"])
    if own and "tables" in s:
        import long_context_sparse_cca_b200 as cca
        s["cache"] = cca.PagedCache.from_tensors(*s["tables"], *s["pools"], Hq=case.get("Hq", case["Hkv"]),
                                                 g=case["g"], w=case["w"])
        s["saved"] = s["cache"].tables.clone()
    return s


# ---------------------------------------------------------------- the plain forms

def _softmax(x, keep):
    """Softmax over the last axis of the entries that `keep` names; zeros where it names none."""
    x = x.masked_fill(~keep, -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    return x / x.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_pool(q, k, v, scale):
    """q [..., r, d] scores k, v [..., g, d] of a group: its core key and value, in fp32."""
    a = torch.softmax(q @ k.transpose(-1, -2) * scale, -1).mean(-2, keepdim=True)
    return (a @ k).squeeze(-2), (a @ v).squeeze(-2)


def _plain_prompt(s):
    Q, K, V = s["Q"].float(), s["K"].float(), s["V"].float()
    Hq, total, d = Q.shape
    Hkv, r, g, w, lens, cu = K.shape[0], Hq // K.shape[0], s["g"], s["w"], s["lens"], s["cu"].long()
    scale, dev, longest = 1.0 / math.sqrt(d), Q.device, max(s["lens"])
    start, length, S = cu[:-1], cu[1:] - cu[:-1], len(s["lens"])
    out = {}
    core = _pooled(s, total)
    if core:  # the groups' core rows
        c = torch.arange(total // g, device=dev)
        sid = (torch.searchsorted(start // g, c, right=True) - 1).clamp(min=0)
        j = c - start[sid] // g
        held = (j < length[sid] // g)[None, :, None]
        at = (start[sid] + j * g)[:, None] + torch.arange(g, device=dev)
        at = at.clamp(max=total - 1)
        q = Q[:, at[:, -1]].view(Hkv, r, -1, d).transpose(1, 2)
        Kc, Vc = _plain_pool(q, K[:, at], V[:, at], scale)
        out["Kc"], out["Vc"] = (torch.where(held, x, 0.0).half() for x in (Kc, Vc))
        Kc, Vc = out["Kc"].float(), out["Vc"].float()
    # attention, in blocks of queries: a block's local keys lie in one stretch
    n = 256
    nb = (length + n - 1) // n
    many = sum(-(-x // n) for x in lens)
    sid = torch.repeat_interleave(torch.arange(S, device=dev), nb, output_size=many)
    first = torch.cumsum(nb, 0) - nb
    t0 = (torch.arange(many, device=dev) - first[sid]) * n
    t = t0[:, None] + torch.arange(n, device=dev)
    ws = (t - w).clamp(min=0) // g * g
    p = ws[:, :1] + torch.arange(min(longest, w + g + n), device=dev)
    keep = (p[:, None] >= ws[:, :, None]) & (p[:, None] <= t[:, :, None])
    row = lambda x: (start[sid][:, None] + x).clamp(max=total - 1)  # noqa: E731
    q = Q[:, row(t)].view(Hkv, r, many, n, d).transpose(1, 2).reshape(Hkv, many, r * n, d)
    keys, vals = K[:, row(p)], V[:, row(p)]
    if core and longest > w:
        c = torch.arange(max(1, _window_start(longest - 1, g, w) // g), device=dev)
        at = ((start // g)[sid][:, None] + c).clamp(max=total // g - 1)
        keys, vals = torch.cat([Kc[:, at], keys], 2), torch.cat([Vc[:, at], vals], 2)
        keep = torch.cat([c < (ws // g)[:, :, None], keep], -1)
    a = _softmax(q @ keys.transpose(-1, -2) * scale, keep.repeat(1, r, 1))
    o = (a @ vals).view(Hkv, many, r, n, d).transpose(1, 2).reshape(Hq, many * n, d)
    tok = torch.arange(total, device=dev)
    sid = torch.searchsorted(cu, tok, right=True) - 1
    out["O"] = o[:, first[sid] * n + tok - start[sid]].to(torch.bfloat16)
    if s["page"]:  # the cache's pages: raw rows of the last token's window, core rows of all groups
        page, (ct, rt, _, _, _), (kc, vc, kr, vr) = s["page"], s["tables"], s["pools"]
        i, j, c = s["core_at"]
        kc[0][ct[i, j // page].long(), :, j % page] = out["Kc"][:, c].transpose(0, 1)
        vc[0][ct[i, j // page].long(), :, j % page] = out["Vc"][:, c].transpose(0, 1)
        i = torch.arange(S, device=dev)[:, None]
        last = length[:, None] - 1
        p = torch.minimum((last - w).clamp(min=0) // g * g + torch.arange(min(longest, w + g), device=dev), last)
        kr[0][rt[i, p // page].long(), :, p % page] = s["K"][:, start[:, None] + p].permute(1, 2, 0, 3)
        vr[0][rt[i, p // page].long(), :, p % page] = s["V"][:, start[:, None] + p].permute(1, 2, 0, 3)
        out["pools"] = s["pools"]
    return out


def _plain_step(s):
    (ct, rt, _, _, lens), (kc, vc, kr, vr) = s["tables"], [x[0] for x in s["pools"]]
    (B, Hq, d), Hkv, g, w, page = s["q_t"].shape, s["Hkv"], s["g"], s["w"], s["page"]
    scale, dev = 1.0 / math.sqrt(d), lens.device
    row = torch.arange(B, device=dev)
    t = lens - 1
    slot = rt[row, t // page].long()
    kr[slot, :, t % page], vr[slot, :, t % page] = s["k_t"], s["v_t"]
    q = s["q_t"].float().view(B, Hkv, Hq // Hkv, d)
    done = s["done"]
    p = t[done, None] - g + 1 + torch.arange(g, device=dev)
    at = rt[done[:, None], p // page].long()
    k, v = (x[at, :, p % page].float().transpose(1, 2) for x in (kr, vr))
    k, v = _plain_pool(q[done], k, v, scale)
    j = t[done] // g
    at = ct[done, j // page].long()
    kc[at, :, j % page], vc[at, :, j % page] = k.half(), v.half()
    ws = (t - w).clamp(min=0) // g * g
    longest = max(s["lens"])
    p = ws[:, None] + torch.arange(min(longest, w + g), device=dev)
    keep = p <= t[:, None]
    p = torch.minimum(p, t[:, None])
    at = rt[row[:, None], p // page].long()
    k, v = (x[at, :, p % page].float() for x in (kr, vr))
    if longest > w:
        c = torch.arange(max(1, _window_start(longest - 1, g, w) // g), device=dev).expand(B, -1)
        at = ct[row[:, None], c // page].long().clamp(min=0)
        k = torch.cat([kc[at, :, c % page].float(), k], 1)
        v = torch.cat([vc[at, :, c % page].float(), v], 1)
        keep = torch.cat([c < (ws // g)[:, None], keep], 1)
        k, v = (torch.where(keep[:, :, None, None], x, 0.0) for x in (k, v))
    a = _softmax(q @ k.permute(0, 2, 3, 1) * scale, keep[:, None, None])
    o = (a @ v.transpose(1, 2)).view(B, Hq, d).to(torch.bfloat16)
    return {"o": o, "pools": s["pools"]}


def _lowest_free(ref):
    """The pages by number, the free ones (count 0) before the others."""
    ids = torch.arange(ref.numel(), device=ref.device)
    return torch.sort(torch.where(ref == 0, ids, ids + ref.numel()))[0] % ref.numel()


def _references(table, pages):
    table = table.long().flatten()
    return torch.zeros(pages + 1, dtype=torch.int32, device=table.device).scatter_add_(
        0, torch.where(table < 0, pages, table), torch.ones_like(table, dtype=torch.int32))[:pages]


def _plain_fork_pool(s, table, ref, pools, has, copied):
    """Rows take over their parents' pages; a parent's last, partly filled page is copied."""
    src, dev = s["parent"].long(), table.device
    new = table[src].clone()
    col = has[src] - 1  # the last page's column
    hole = new.clone()
    hole[copied, col[copied]] = -1
    count = _references(hole, ref.numel())
    fresh = _lowest_free(count)[:copied.numel()]
    old = table[src[copied], col[copied]].long()
    new[copied, col[copied]] = fresh.int()
    k, v = pools
    k[:, fresh], v[:, fresh] = k[:, old], v[:, old]
    count[fresh] = 1
    return new, count


def _plain_room_pool(table, ref, lo, had, need):
    """Columns had .. need - 1 get new pages, and columns before lo go."""
    cols = torch.arange(table.shape[1], device=table.device)
    want = (cols >= had[:, None]) & (cols < need[:, None])
    order = (torch.cumsum(want.flatten(), 0) - 1).view_as(want).clamp(min=0)
    new = torch.where(want, _lowest_free(ref)[order].int(), table)
    new = torch.where(cols < lo[:, None], -1, new)
    return new, _references(new, ref.numel())


def _plain_fork(s):
    ct, rt, cref, rref, lens = s["tables"]
    kc, vc, kr, vr = s["pools"]
    g, w, page, n = s["g"], s["w"], s["page"], lens[s["parent"].long()]
    up = lambda x: (x + page - 1) // page  # noqa: E731
    ct, cref = _plain_fork_pool(s, ct, cref, (kc, vc), up(lens // g), s["copied"][0])
    rt, rref = _plain_fork_pool(s, rt, rref, (kr, vr), up(lens), s["copied"][1])
    # room for the next token
    ct, cref = _plain_room_pool(ct, cref, torch.zeros_like(n), up(n // g), up((n + 1) // g))
    rt, rref = _plain_room_pool(rt, rref, (n - w).clamp(min=0) // g * g // page, up(n), up(n + 1))
    return {"tables": (ct, rt, cref, rref, n + 1), "pools": s["pools"]}


def _plain_compact_pool(table, ref, pools, moved):
    """The used pages of the highest numbers move to the free ones of the lowest."""
    pages = ref.numel()
    ids = torch.arange(pages, device=ref.device)
    used = ref > 0
    live = used.sum()
    src = torch.sort(torch.where(used & (ids >= live), ids, ids + pages))[0][:moved]
    dst = torch.sort(torch.where(~used & (ids < live), ids, ids + pages))[0][:moved]
    to = ids.clone()
    to[src] = dst
    table = torch.where(table >= 0, to[table.long().clamp(min=0)].int(), -1)
    ref = ref.clone()
    ref[dst] = ref[src]
    ref[src] = 0
    k, v = pools
    k[:, dst], v[:, dst] = k[:, src], v[:, src]
    return table, ref, live


def _plain_compact(s):
    ct, rt, cref, rref, lens = s["tables"]
    kc, vc, kr, vr = s["pools"]
    ct, cref, core = _plain_compact_pool(ct, cref, (kc, vc), s["moved"][0])
    rt, rref, raw = _plain_compact_pool(rt, rref, (kr, vr), s["moved"][1])
    return {"tables": (ct, rt, cref, rref, lens), "live": torch.stack([core, raw]), "pools": s["pools"]}


def run(state):
    s, kind = state, state["kind"]
    if own:
        import long_context_sparse_cca_b200 as cca
        if kind == "prompt":
            Kc = Vc = None
            out = {}
            if _pooled(s, s["Q"].shape[1]):
                out["Kc"], out["Vc"] = Kc, Vc = cca.cca_pool_packed(s["Q"], s["K"], s["V"], s["cu"], s["g"])
            out["O"] = cca.cca_attn_prefill_packed(s["Q"], s["K"], s["V"], Kc, Vc, s["cu"], s["g"], s["w"])
            if s["page"]:
                cca.cca_paged_fill(s["cache"], s["K"], s["V"], Kc, Vc, s["cu"], s["rows"])
                out["pools"] = s["cache"].pools
            return out
        c = s["cache"]
        if kind == "step":
            return {"o": cca.cca_paged_step(c, s["q_t"], s["k_t"], s["v_t"]), "pools": c.pools}
        c.tables.copy_(s["saved"])  # the tables of a moment ago, all in one tensor
        if kind == "fork":
            cca.cca_paged_fork(c, s["parent"])
            cca.cca_paged_reserve(c, 1)
            return {"tables": (c.core_table, c.raw_table, c.core_ref, c.raw_ref, c.lens), "pools": c.pools}
        live = cca.cca_paged_compact(c)
        return {"tables": (c.core_table, c.raw_table, c.core_ref, c.raw_ref, c.lens), "live": live,
                "pools": c.pools}
    return {"prompt": _plain_prompt, "step": _plain_step, "fork": _plain_fork,
            "compact": _plain_compact}[kind](s)


# ---------------------------------------------------------------- what it costs, and 64 bits

def work(case):
    d, g, w, kind = case["d"], case["g"], case.get("w"), case["kind"]
    if kind in ("prompt", "step"):
        lens, Hq, Hkv = _ints(case["lens"]), case["Hq"], case["Hkv"]
        if kind == "prompt":
            t = np.concatenate([np.arange(n) for n in lens])
            total = len(t)
        else:
            t = np.array(lens) - 1
        ws = np.maximum(t - w, 0) // g * g
        pairs = float((ws // g + t - ws + 1).sum())
        flops = 4.0 * d * Hq * pairs
        if kind == "step":  # the rows of the attended keys, the new token's rows, q and o
            held = sum(n % g == 0 for n in lens)
            return {"bytes": 4.0 * d * Hkv * (pairs + len(lens) + held) + 4.0 * d * Hq * len(lens), "flops": flops}
        bytes_ = 2.0 * d * total * (2 * Hq + 2 * Hkv)
        groups = sum(n // g for n in lens)
        if _pooled(case, total):  # the core rows, and the pooling's products
            bytes_ += 4.0 * d * Hkv * (total // g)
            flops += 2.0 * d * g * groups * (Hq + 2 * Hkv)
        if case["page"]:
            held = sum(n - _window_start(n - 1, g, w) for n in lens)
            bytes_ += 4.0 * d * Hkv * (groups + held)
        return {"bytes": bytes_, "flops": flops}
    size = 4.0 * case["layers"] * case["Hkv"] * case["page"] * d  # a page of K and of V, all layers
    if kind == "fork":
        lens = _ints(case["lens"])
        many = sum((n % case["page"] > 0) + (n // g % case["page"] > 0) for n in lens) * (case["copies"] - 1)
        raw, core = _rows(lens, g, w, case["page"])
        entries = case["copies"] * (sum(core) + sum(hi - lo for lo, hi in raw))
    else:  # of the used pages, those above the used pages' number move: a share of 1 - used / pages
        raw, core = _rows(_compact_lens(case), g, w, case["page"])
        used = (sum(core), sum(hi - lo for lo, hi in raw))
        entries = sum(used)
        many = sum(n * (1 - n / p) for n, p in zip(used, (case["core_pages"], case["raw_pages"])))
    pages = case["core_pages"] + case["raw_pages"]
    return {"bytes": 2 * size * many + 8.0 * entries + 8.0 * pages, "flops": 0.0}


def _exact_rows(q, K, V, scale):
    """Softmax attention of q [r, d] over K, V [n, d], in 64 bits."""
    a = q @ K.T * scale
    a = torch.exp(a - a.max(1, keepdim=True).values)
    return a @ V / a.sum(1, keepdim=True)


def exact(case, seed):
    if case["kind"] not in ("prompt", "step"):
        return None  # whole numbers, and rows that are moved as they are
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    f, g, w, d = torch.float64, case["g"], case["w"], case["d"]
    Hq, Hkv, lens, scale = case["Hq"], case["Hkv"], _ints(case["lens"]), 1.0 / math.sqrt(case["d"])
    r = Hq // Hkv
    kc, vc = (x.to(f) for x in s["pools"][:2]) if "pools" in s else (None, None)
    ct = s["tables"][0].cpu().numpy() if "tables" in s else None

    def put(b, j, k, v):
        at = int(ct[b, j // case["page"]])
        kc[0, at, :, j % case["page"]], vc[0, at, :, j % case["page"]] = k, v

    if case["kind"] == "prompt":
        Q, K, V = (s[n].to(f) for n in "QKV")
        total = Q.shape[1]
        O = torch.empty(Hq, total, d, dtype=f, device="cuda")
        Kc = torch.zeros(Hkv, total // g, d, dtype=f, device="cuda")
        Vc = torch.zeros_like(Kc)
        a0 = 0
        for b, n in enumerate(lens):
            q, k, v, m = Q[:, a0:a0 + n], K[:, a0:a0 + n], V[:, a0:a0 + n], n // g
            c = slice(a0 // g, a0 // g + m)
            if _pooled(case, total) and m:
                ql = q[:, g - 1:m * g:g].reshape(Hkv, r, m, d)
                kg, vg = (x[:, :m * g].reshape(Hkv, m, g, d) for x in (k, v))
                a = torch.softmax(torch.einsum("hrmd,hmgd->hrmg", ql, kg) * scale, -1).mean(1)
                Kc[:, c], Vc[:, c] = torch.einsum("hmg,hmgd->hmd", a, kg), torch.einsum("hmg,hmgd->hmd", a, vg)
            for h in range(Hkv):
                keys = torch.cat([Kc[h, c].half().to(f), k[h]])
                vals = torch.cat([Vc[h, c].half().to(f), v[h]])
                nc = len(keys) - n
                place = torch.cat([torch.arange(nc, device="cuda"), torch.arange(n, device="cuda")])
                raw = torch.arange(nc + n, device="cuda") >= nc
                for t0 in range(0, n, 2048):
                    t = torch.arange(t0, min(n, t0 + 2048), device="cuda")[:, None]
                    ws = (t - w).clamp(min=0) // g * g
                    seen = torch.where(raw, (place >= ws) & (place <= t), place < ws // g)
                    for i in range(h * r, h * r + r):
                        x = (q[i, t0:t0 + 2048] @ keys.T * scale).masked_fill(~seen, -math.inf)
                        O[i, a0 + t0:a0 + t0 + len(t)] = torch.softmax(x, 1) @ vals
            if case["page"]:
                for j in range(m):
                    put(b, j, Kc[:, c][:, j], Vc[:, c][:, j])
            a0 += n
        out = {"O": O}
        if _pooled(case, total):
            out |= {"Kc": Kc, "Vc": Vc}
        return out | ({"pools": (kc, vc, None, None)} if case["page"] else {})
    o = torch.empty(len(lens), Hq, d, dtype=f, device="cuda")
    rt, page = s["tables"][1].cpu().numpy(), case["page"]
    kr, vr = s["pools"][2:]
    for b, n in enumerate(lens):
        ws = _window_start(n - 1, g, w)
        cols = _gpu(rt[b, ws // page:-(-n // page)]).long()
        off = ws // page * page
        q = s["q_t"][b].to(f).view(Hkv, r, d)
        for h in range(Hkv):
            # (the pages' rows up to the one before the last token, then the last token's)
            k, v = (torch.cat([x[0, cols, h].reshape(-1, d)[ws - off:n - 1 - off], y[b, h:h + 1]]).to(f)
                    for x, y in ((kr, s["k_t"]), (vr, s["v_t"])))
            if n % g == 0:
                first = n - g - ws
                a = torch.softmax(q[h] @ k[first:].T * scale, 1).mean(0)
                at, j = int(ct[b, (n - 1) // g // page]), (n - 1) // g % page
                kc[0, at, h, j], vc[0, at, h, j] = a @ k[first:], a @ v[first:]
            nc = ws // g
            cc = _gpu(ct[b, :-(-nc // page)]).long()
            k, v = (torch.cat([x[0, cc, h].reshape(-1, d)[:nc], y]) for x, y in ((kc, k), (vc, v)))
            o[b, h * r:h * r + r] = _exact_rows(q[h], k, v, scale)
    return {"o": o, "pools": (kc, vc, None, None)}
