"""The operators of a step that verifies trees of drafted tokens over a paged latent cache, as cases to measure:

* heads    - root-mean-square norms of every head's query and of the latents, turned by their positions; queries leave
             in bf16, latents as FP4 or E4M3 rows of the cache
* tree     - positions and ancestor masks of the requests' trees, and the attention of their nodes over the cached
             entries and their own ancestors
* logprobs - log-sum-exp, entropy, log probabilities of given tokens and the top alternatives of rows of logits
* commit   - the path of accepted nodes: its rows moved together, lengths, and pages given back

run() computes an operator from elementary torch operations, or through the library where `own` is true.
"""
import math

import torch

own = False

D = 512         # latent width
THETA = 10000.0
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the queries and latents of 16 decoding requests, 64 heads: latency
        {"name": "heads decode 16", "op": "heads", "tokens": 16, "heads": 64, "fmt": "fp4", "norm": "both", "rotate": True,
         "fused": False},
        # an odd chunk of a window layer: E4M3 latents, nothing turned, both out of one projection's rows
        {"name": "heads window 333", "op": "heads", "tokens": 333, "heads": 16, "fmt": "fp8", "norm": "both", "rotate": False,
         "fused": True},
        # prompts' chunks, 4096 tokens in all
        {"name": "heads chunk 4096", "op": "heads", "tokens": 4096, "heads": 64, "fmt": "fp4", "norm": "both", "rotate": True,
         "fused": False},
        # one request verifies a small tree: latency
        {"name": "tree 16 on 2k", "op": "tree", "requests": 1, "heads": 64, "nodes": 16, "shape": "random", "cached": 2048,
         "page": 64, "fmt": "fp4", "window": 0, "mixed": False},
        # a batch that drafts a few tokens each
        {"name": "tree 16x8 on 8k", "op": "tree", "requests": 16, "heads": 64, "nodes": 8, "shape": "beam", "cached": 8192,
         "page": 64, "fmt": "fp4", "window": 0, "mixed": False},
        # odd trees beside single tokens in a window layer, a quarter of the heads
        {"name": "tree window mixed", "op": "tree", "requests": 24, "heads": 16, "nodes": 45, "shape": "random", "cached": 3001,
         "page": 16, "fmt": "fp8", "window": 128, "mixed": True},
        # wide trees over long contexts
        {"name": "tree 8x64 on 16k", "op": "tree", "requests": 8, "heads": 64, "nodes": 64, "shape": "random", "cached": 16384,
         "page": 128, "fmt": "fp4", "window": 0, "mixed": False},
        # the next token of one request, with a few alternatives: latency
        {"name": "logprobs 1 of 32000", "op": "logprobs", "rows": 1, "vocab": 32000, "dtype": "f32", "given": 1, "top": 5,
         "scale": 1.0, "masked": False, "pad": 0},
        # every node of a batch's trees, grammar masks on some rows, an odd vocabulary in longer rows
        {"name": "logprobs 121 masked", "op": "logprobs", "rows": 121, "vocab": 100003, "dtype": "f32", "given": 4, "top": 20,
         "scale": 1.25, "masked": True, "pad": 13},
        # log probabilities of a prompt's tokens
        {"name": "logprobs 2048 of 131072", "op": "logprobs", "rows": 2048, "vocab": 131072, "dtype": "bf16", "given": 1, "top": 20,
         "scale": 1.0, "masked": False, "pad": 0},
        # a batch's accepted paths, small trees
        {"name": "commit 16x8", "op": "commit", "requests": 16, "nodes": 8, "shape": "beam", "cached": 2000, "page": 64, "fmt": "fp4"},
        # many requests with wide trees
        {"name": "commit 192x61", "op": "commit", "requests": 192, "nodes": 61, "shape": "random", "cached": 700, "page": 16,
         "fmt": "fp8"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("heads", "heads", "tree", "tree", "logprobs", "logprobs", "commit"))
    if op == "heads":
        heads = rng.choice((1, 5, 8, 16, 24, 32, 64, 64, 128))
        rotate = rng.random() < 0.8
        return {"op": op, "tokens": min(_log(rng, 1, 4096), 4096 * 64 // heads), "heads": heads, "fmt": rng.choice(("fp4", "fp4", "fp8")),
                "norm": rng.choice(("both", "both", "queries", "none")) if rotate else "both", "rotate": rotate,
                "fused": rng.random() < 0.4}
    if op == "tree":
        heads = rng.choice((5, 8, 16, 24, 32, 64, 64, 128))
        requests, nodes, cached = _log(rng, 1, 32), _log(rng, 1, 200), _log(rng, 16, 16384)
        # a drawn case stays below the largest listed one, padded to its longest request
        while requests * nodes * heads * (cached + nodes) > 8 * 64 * 64 * 16384:
            if requests > 1 and nodes > 1:
                requests = max(1, requests // 2)
            elif nodes > 1:
                nodes = max(1, nodes // 2)
            else:
                cached //= 2
        return {"op": op, "requests": requests, "heads": heads, "nodes": nodes, "shape": rng.choice(("random", "beam", "chain")),
                "cached": cached, "page": rng.choice((8, 16, 64, 128, 200)), "fmt": rng.choice(("fp4", "fp4", "fp8")),
                "window": rng.choice((0, 0, 0, 3, 100, 128, 1000)), "mixed": rng.random() < 0.5}
    if op == "logprobs":
        vocab = _log(rng, 1000, 200000)
        return {"op": op, "rows": min(_log(rng, 1, 2048), 2048 * 65536 // vocab), "vocab": vocab, "dtype": rng.choice(("bf16", "f32")),
                "given": rng.choice((0, 1, 1, 4, 9)), "top": rng.choice((0, 1, 5, 20, 64)), "scale": rng.choice((1.0, 1.25, 0.5)),
                "masked": rng.random() < 0.5, "pad": rng.choice((0, 0, 5, 96))}
    return {"op": op, "requests": _log(rng, 1, 192), "nodes": _log(rng, 1, 61), "shape": rng.choice(("random", "beam", "chain")),
            "cached": _log(rng, 1, 700), "page": rng.choice((8, 16, 64, 200)), "fmt": rng.choice(("fp4", "fp8"))}


# ----------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ceil(a, b):
    return (a + b - 1) // b


def _lengths(case, g):
    """Per request (cached, nodes): spread evenly from about a quarter of the case's sizes to all of them and, where the
    case is mixed, every other request brings one token; which request has which goes by the seed."""
    n = case["requests"]
    part = 0.25 + 0.75 * torch.arange(1, n + 1, device="cuda", dtype=torch.float64) / n
    cached = (case["cached"] * part).round().to(torch.int32)
    nodes = (case["nodes"] * part).round().to(torch.int32).clamp(min=1)
    if case.get("mixed"):
        nodes[(n - 1 - torch.arange(n, device="cuda")) % 2 == 1] = 1
    return cached[torch.randperm(n, device="cuda", generator=g)], nodes[torch.randperm(n, device="cuda", generator=g)]


def _quantize_fp4(x):
    """E2M1 codes [rows][k/2] and E4M3 scales [rows][k/16] of fp32 rows: scale amax/6, nearest code."""
    rows, k = x.shape
    xg = x.view(rows, k // 16, 16)
    s = (xg.abs().amax(2) / 6.0).to(torch.float8_e4m3fn)
    r = xg / s.float().clamp(min=2.0 ** -9).unsqueeze(2)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    c = torch.bucketize(r.abs(), mids).to(torch.uint8) | ((r < 0).to(torch.uint8) << 3)
    c = c.view(rows, k // 2, 2)
    return (c[..., 0] | (c[..., 1] << 4)).contiguous(), s.view(torch.uint8)


def _pages(case, s, cached, nodes, g, spare):
    """Block tables, and the latents' planes, of requests that hold cached + nodes entries."""
    P, dev = case["page"], "cuda"
    pages = _ceil(cached + nodes, P)
    s["held"] = int(pages.sum())
    s["n_pages"] = n_pages = int(_ceil(cached, P).sum() + _ceil(nodes, P).sum()) + spare  # (the same for every seed)
    s["max_pages"] = _ceil(case["cached"] + case["nodes"], P)
    ids = torch.randperm(n_pages, device=dev, generator=g).to(torch.int32)
    base = torch.cumsum(pages, 0) - pages
    j = torch.arange(s["max_pages"], device=dev)
    s["table"] = torch.where(j[None, :] < pages[:, None], ids[(base[:, None] + j).clamp(max=n_pages - 1)],
                             torch.full((), -1, dtype=torch.int32, device=dev))
    s["n_rows"] = n_rows = n_pages * P
    lat = torch.randn(n_rows, D, device=dev, generator=g)
    if case["fmt"] == "fp4":
        s["codes"], s["scales"] = _quantize_fp4(lat)
    else:
        s["codes"], s["scales"] = lat.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), None
    s["kv_len"] = cached + nodes
    s["q_start"] = torch.zeros(case["requests"] + 1, dtype=torch.int32, device=dev)
    s["q_start"][1:] = torch.cumsum(nodes, 0)
    s["tokens"], s["max_q"], s["max_kv"] = int(nodes.sum()), int(nodes.max()), int(s["kv_len"].max())
    return ids


def _trees(case, s, g):
    """The parent of every node within its request: -1 for the first one, then by the case's shape."""
    req = torch.searchsorted(s["q_start"][1:], torch.arange(s["tokens"], device="cuda", dtype=torch.int32), right=True)
    i = torch.arange(s["tokens"], device="cuda") - s["q_start"][req]
    if case["shape"] == "chain":
        up = i - 1
    elif case["shape"] == "beam":  # levels of four
        up = torch.where(i <= 4, 0, i - 4)
    else:
        up = (torch.rand(s["tokens"], device="cuda", generator=g, dtype=torch.float64) * i).long()
        up = torch.minimum(up, i - 1)
    s["req"], s["parent"] = req, torch.where(i == 0, -1, up).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op, dev = case["op"], "cuda"
    s = {"case": dict(case)}
    if op == "heads":
        T, H = case["tokens"], case["heads"]
        amp = torch.exp(0.5 * torch.randn(T, 1, 1, device=dev, generator=g))
        rows = (amp * torch.randn(T, H + 1, D, device=dev, generator=g)).to(torch.bfloat16)
        s["q"], s["latents"] = (rows[:, :H], rows[:, H]) if case["fused"] else (rows[:, :H].contiguous(), rows[:, H].contiguous())
        weight = lambda: (1 + 0.2 * torch.randn(D, device=dev, generator=g)).to(torch.bfloat16)  # noqa: E731
        s["q_weight"], s["l_weight"] = weight(), weight()
        if case["norm"] != "both":
            s["l_weight"] = None
        if case["norm"] == "none":
            s["q_weight"] = None
        s["max_pos"] = 131072
        s["pos"] = torch.randint(0, s["max_pos"], (T,), device=dev, generator=g)
        s["n_rows"] = 8 * _ceil(T, 8)
        s["dst"] = torch.randperm(s["n_rows"], device=dev, generator=g)[:T]
        pad = T // 16  # rows behind the step's tokens
        if pad:
            s["pos"][T - pad:] = -1
            s["dst"][T - pad:] = -1
        s["out"] = torch.zeros(T, H, D, dtype=torch.bfloat16, device=dev)
        if case["fmt"] == "fp4":
            s["codes"] = torch.zeros(s["n_rows"], D // 2, dtype=torch.uint8, device=dev)
            s["scales"] = torch.zeros(s["n_rows"], D // 16, dtype=torch.uint8, device=dev)
        else:
            s["codes"], s["scales"] = torch.zeros(s["n_rows"], D, dtype=torch.uint8, device=dev), None
    elif op == "tree":
        cached, nodes = _lengths(case, g)
        _pages(case, s, cached, nodes, g, 3)
        _trees(case, s, g)
        s["words"] = _ceil(s["max_q"], 32)
        s["q"] = torch.randn(s["tokens"], case["heads"], D, device=dev, generator=g).to(torch.bfloat16)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(s["tokens"], case["heads"], device=dev)
        s["pos"] = torch.zeros(s["tokens"], dtype=torch.int64, device=dev)
        s["mask"] = torch.zeros(s["tokens"], s["words"], dtype=torch.int32, device=dev)
    elif op == "logprobs":
        n, V = case["rows"], case["vocab"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        x = torch.empty(n, V + case["pad"], dtype=dt, device=dev)
        for i in range(0, n, 256):
            part = torch.randn(min(256, n - i), V + case["pad"], device=dev, generator=g)
            part = 2.0 * part + 0.5 * part * part.abs()  # a few tokens stand out
            if case["masked"]:  # by -inf in one of three rows, by the type's lowest value in another, few to many are left
                r = torch.arange(i, i + part.shape[0], device=dev)
                share = torch.exp(torch.empty(part.shape[0], 1, device=dev).uniform_(-10.0, 0.0, generator=g))
                off = torch.rand(part.shape, device=dev, generator=g) > share
                off[:, V // 3] = False
                part = torch.where(off & (r % 3 == 1)[:, None], -math.inf, part)
                part = torch.where(off & (r % 3 == 2)[:, None], torch.finfo(dt).min, part)
            x[i:i + part.shape[0]] = part.to(dt)
        s["logits"] = x[:, :V]
        s["tokens"] = torch.randint(0, V, (n, case["given"]), device=dev, generator=g)
        if case["given"]:
            s["tokens"][::7, 0] = -1  # a row without a token
        s["logprobs"] = torch.zeros(n, case["given"], device=dev)
        s["lse"], s["entropy"] = torch.zeros(n, device=dev), torch.zeros(n, device=dev)
        s["ids"] = torch.zeros(n, case["top"], dtype=torch.int32, device=dev)
        s["best"] = torch.zeros(n, case["top"], device=dev)
    else:
        cached, nodes = _lengths(case, g)
        ids = _pages(case, s, cached, nodes, g, 37)
        _trees(case, s, g)
        n, R = s["tokens"], case["requests"]
        s["free"] = torch.zeros(s["n_pages"], dtype=torch.int32, device=dev)
        s["free"][:37] = ids[s["held"]:s["held"] + 37]
        s["n_free"] = torch.tensor([37], dtype=torch.int32, device=dev)
        s["n_free_out"] = torch.zeros(1, dtype=torch.int32, device=dev)
        s["token"] = torch.randint(0, 50, (n,), device=dev, generator=g)
        # the model goes on with one of a node's children four times in five or so
        up = s["q_start"][s["req"]].long() + s["parent"].clamp(min=0)
        taken = torch.where((s["parent"] >= 0) & (torch.rand(n, device=dev, generator=g) < 0.8), s["token"], -1)
        s["choice"] = torch.full((n,), -1, dtype=torch.int64, device=dev).scatter_reduce(0, up, taken, "amax")
        s["choice"] = torch.where(s["choice"] < 0, torch.randint(0, 50, (n,), device=dev, generator=g), s["choice"])
        s["path"] = torch.zeros(n, dtype=torch.int32, device=dev)
        s["accepted"] = torch.zeros(R, dtype=torch.int32, device=dev)
        s["next"] = torch.zeros(R, dtype=torch.int64, device=dev)
        s["cached"] = torch.zeros(R, dtype=torch.int32, device=dev)
    return s


# ------------------------------------------------------------- plain forms
def _values(codes, scales):
    """fp32 values [rows][2 * bytes] of FP4 rows, or of E4M3 rows where scales is None."""
    if scales is None:
        return codes.view(torch.float8_e4m3fn).float()
    mags = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = torch.stack((mags[(codes & 15).long()], mags[(codes >> 4).long()]), -1).view(codes.shape[0], -1)
    return (v.view(codes.shape[0], -1, 16) * scales.view(torch.float8_e4m3fn).float().unsqueeze(2)).view(codes.shape[0], -1)


def _heads_plain(s):
    c, pos = s["case"], s["pos"]
    live = pos >= 0

    def normed(x, w):
        return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.to(x.dtype)

    def turned(x, cos, sin):
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)

    q = normed(s["q"].float(), s["q_weight"])
    z = normed(s["latents"].double(), s["l_weight"])  # codes next to a border between two values
    if c["rotate"]:
        rate = torch.pow(THETA, -torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
        angle = pos.clamp(min=0).double()[:, None] * rate
        cos, sin = torch.cos(angle), torch.sin(angle)
        q, z = turned(q, cos.float()[:, None], sin.float()[:, None]), turned(z, cos, sin)
    q = torch.where(live[:, None, None], q.to(torch.bfloat16), s["out"])
    row = torch.where(live, s["dst"], s["n_rows"])  # a row behind the cache takes what is stored nowhere
    place = lambda v: torch.zeros(s["n_rows"] + 1, v.shape[1], device="cuda", dtype=v.dtype).index_copy_(0, row, v)[:-1]  # noqa: E731
    if c["fmt"] == "fp8":
        return {"q": q, "latents": place(z.clamp(-448, 448).float()).to(torch.float8_e4m3fn)}
    zg = z.view(-1, D // 16, 16)
    scale = (zg.abs().amax(2) / 6.0).float().to(torch.float8_e4m3fn).float()
    r = (zg / torch.where(scale == 0, 1.0, scale).double().unsqueeze(2))
    a = r.abs()
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)) * (scale != 0).unsqueeze(2)
    value = torch.tensor(E2M1, device="cuda")[code.long()] * torch.where(r < 0, -1.0, 1.0).float()
    return {"q": q, "latents": place(value.view(-1, D)).to(torch.bfloat16), "scales": place(scale).to(torch.float8_e4m3fn)}


def _by_request(s, v, fill):
    """A value per node as [requests][max_q], `fill` behind a request's nodes."""
    at = s["q_start"][:-1, None] + torch.arange(s["max_q"], device="cuda")
    return torch.where(at < s["q_start"][1:, None], v[at.clamp(max=s["tokens"] - 1)], fill)


def _lineage(s):
    """[requests][max_q][max_q]: column node is the row node or an ancestor of it."""
    parent, n = _by_request(s, s["parent"], -1), s["max_q"]
    j = torch.arange(n, device="cuda")
    up = ((parent[:, :, None] == j) | (j[:, None] == j)).float()
    for _ in range(max(1, math.ceil(math.log2(n))) if n > 1 else 0):  # twice as many generations each time
        up = (torch.matmul(up, up) > 0).float()
    return up > 0


def _tree_plain(s):
    c = s["case"]
    P, H, R, W, n = c["page"], c["heads"], c["requests"], c["window"], s["max_q"]
    nodes = s["q_start"][1:] - s["q_start"][:-1]
    up = _lineage(s)
    depth = up.sum(2) - 1
    if W:
        up = up & (depth[:, None, :] > depth[:, :, None] - W)
    live = torch.arange(n, device="cuda")[None, :] < nodes[:, None]
    first = s["kv_len"] - nodes
    t = first[:, None] + depth
    bits = torch.nn.functional.pad(up, (0, 32 * s["words"] - n)).view(R, n, s["words"], 32)
    mask = (bits.long() << torch.arange(32, device="cuda")).sum(3)
    mask = torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32)
    p = torch.arange(s["max_kv"], device="cuda")
    rows = s["table"][:, p // P].clamp(min=0).long() * P + p % P
    k = _values(s["codes"][rows.view(-1)], None if s["scales"] is None else s["scales"][rows.view(-1)]).view(R, -1, D)
    q = s["q"][(s["q_start"][:-1, None] + torch.arange(n, device="cuda")).clamp(max=s["tokens"] - 1)].float().view(R, -1, D)
    old = p[None, :] < first[:, None]
    seen = old[:, None, :].expand(R, n, -1)
    if W:
        seen = seen & (p[None, None, :] > t[:, :, None] - W)
    own_node = (p[None, :] - first[:, None]).clamp(0, n - 1)
    fresh = ~old & (p[None, :] < s["kv_len"][:, None])
    seen = seen | (fresh[:, None, :] & torch.gather(up, 2, own_node[:, None, :].expand(R, n, -1)))
    x = torch.matmul(q, k.transpose(1, 2)).mul_(1.0 / math.sqrt(D)).view(R, n, H, -1)
    x.masked_fill_(~seen[:, :, None, :], -math.inf)
    top = x.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x.sub_(top).exp_()
    total = x.sum(3, keepdim=True)
    o = torch.matmul(x.view(R, -1, s["max_kv"]), k).view(R, n, H, D) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).squeeze(3)
    return {"pos": t[live].long(), "mask": mask[live], "out": o[live].to(torch.bfloat16), "lse": lse[live]}


def _logprobs_plain(s):
    c, x = s["case"], s["logits"].float()
    top = x.amax(1, keepdim=True)
    y = (x - torch.where(top == -math.inf, 0.0, top)) * c["scale"]
    e = torch.exp(y)
    total = e.sum(1)
    log_total = torch.log(total)
    spread = torch.where(e == 0, 0.0, e * y).sum(1)
    got = {"lse": top[:, 0] * c["scale"] + log_total, "entropy": log_total - spread / total}
    tok = s["tokens"]
    if c["given"]:
        got["logprobs"] = torch.where(tok >= 0, torch.gather(y, 1, tok.clamp(min=0)) - log_total[:, None], -math.inf)
    if c["top"]:
        # one whole number per value: larger values first, then the lower index
        bits = (x + 0.0).view(torch.int32)
        key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() << 32
        key = key | ((1 << 31) - 1 - torch.arange(c["vocab"], device="cuda"))
        key = torch.topk(key, c["top"], dim=1).values
        ids = (1 << 31) - 1 - (key & 0xFFFFFFFF)
        best = torch.gather(x, 1, ids)
        some = best > -math.inf
        got["ids"] = torch.where(some, ids, -1).to(torch.int32)
        got["best"] = torch.where(some, torch.gather(y, 1, ids) - log_total[:, None], -math.inf)
    return got


def _commit_plain(s):
    c = s["case"]
    P, R, n = c["page"], c["requests"], s["max_q"]
    nodes = s["q_start"][1:] - s["q_start"][:-1]
    first = s["kv_len"] - nodes
    j = torch.arange(n, device="cuda")
    live = j[None, :] < nodes[:, None]
    parent = _by_request(s, s["parent"], -1).long()
    token, choice = _by_request(s, s["token"], -1), _by_request(s, s["choice"], -2)
    match = live & (parent >= 0) & (token == torch.gather(choice, 1, parent.clamp(min=0)))
    best = torch.full((R, n), n, device="cuda").scatter_reduce(1, parent.clamp(min=0), torch.where(match, j, n), "amin")
    kept = (match & (torch.gather(best, 1, parent.clamp(min=0)) == j)) | (j == 0)
    on = live & ((_lineage(s) & ~kept[:, None, :]).sum(2) == 0)
    accepted = on.sum(1)
    place = torch.where(on, torch.cumsum(on, 1) - 1, n)
    path = torch.full((R, n + 1), -1, device="cuda").scatter(1, place, j.expand(R, n))[:, :n]
    moved = j[None, :] < accepted[:, None]
    src = first[:, None] + torch.where(moved, path, 0)
    dst = first[:, None] + torch.where(moved, j, 0)  # (behind the path: the first node's row onto itself)
    row = lambda p: (torch.gather(s["table"], 1, p // P).long() * P + p % P).view(-1)  # noqa: E731
    src, dst = row(src), row(dst)
    for plane in (s["codes"], s["scales"]):
        if plane is not None:
            plane.index_copy_(0, dst, plane[src])
    cached = first + accepted
    pj = torch.arange(s["max_pages"], device="cuda")
    back = (pj >= _ceil(cached, P)[:, None]) & (pj < _ceil(s["kv_len"], P)[:, None])
    order = torch.cumsum(back.view(-1), 0).view(R, -1)
    at = torch.where(back, s["n_free"] + order[-1, -1] - order, s["n_pages"])
    free = torch.cat((s["free"], s["free"][:1])).scatter(0, at.view(-1), s["table"].view(-1))[:-1]
    last = torch.gather(path, 1, (accepted - 1)[:, None].long())
    return {"path": path[live].to(torch.int32), "accepted": accepted.to(torch.int32),
            "next": torch.gather(choice, 1, last)[:, 0], "cached": cached.to(torch.int32), "free": free,
            "n_free": (s["n_free"] + order[-1, -1]).to(torch.int32), "codes": s["codes"],
            **({} if s["scales"] is None else {"scales": s["scales"]})}


# ------------------------------------------------------------ the library
def _kept(s, name, make):
    if name not in s:  # kept by a program for all its steps
        s[name] = make()
    return s[name]


def _bytes(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def _run_own(s):
    from csa2_sparse_attention_gb300 import abi
    c, st = s["case"], torch.cuda.current_stream()
    fmt = abi.FMT_FP4 if c.get("fmt") == "fp4" else abi.FMT_FP8
    if c["op"] == "heads":
        ws = _kept(s, "ws", lambda: _bytes(abi.STATUS_BYTES))
        table = None
        if c["rotate"]:
            def make():
                t = _bytes(abi.csa2_rope_table_bytes(D, s["max_pos"]))
                abi.csa2_rope_table_init(THETA, D, s["max_pos"], t, st)
                return t
            table = _kept(s, "rope", make)
        abi.csa2_head_norm_rope(s["q"], s["q"].stride(0), c["heads"], s["q_weight"], s["out"], s["latents"], s["latents"].stride(0),
                                s["l_weight"], c["tokens"], EPS, s["pos"], table, s["max_pos"] if c["rotate"] else 0, fmt, s["dst"],
                                s["n_rows"], s["codes"], s["scales"], ws, ws.numel(), st)
        if c["fmt"] == "fp8":
            return {"q": s["out"], "latents": s["codes"].view(torch.float8_e4m3fn)}

        def pairs():  # the two values of a byte
            v = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda", dtype=torch.bfloat16)
            b = torch.arange(256, device="cuda")
            return torch.stack((v[b & 15], v[b >> 4]), 1)
        values = _kept(s, "pairs", pairs)[s["codes"].int()].view(-1, D)
        return {"q": s["out"], "latents": values, "scales": s["scales"].view(torch.float8_e4m3fn)}
    if c["op"] == "tree":
        R = c["requests"]
        ws = _kept(s, "ws", lambda: _bytes(abi.csa2_tree_attn_workspace_bytes(s["tokens"], c["heads"], R, s["max_q"], s["max_kv"],
                                                                             c["window"])))
        abi.csa2_tree_plan(s["parent"], s["q_start"], s["kv_len"], R, s["tokens"], s["max_q"], c["window"], s["pos"], s["mask"],
                           s["words"], ws, ws.numel(), st)
        abi.csa2_tree_attn(s["q"], s["tokens"], c["heads"], s["q_start"], s["kv_len"], R, s["max_q"], s["max_kv"], s["pos"], s["mask"],
                           s["words"], fmt, s["codes"], s["scales"], s["n_rows"], s["table"], s["max_pages"], c["page"], c["window"],
                           1.0 / math.sqrt(D), s["out"], s["lse"], ws, ws.numel(), st)
        return {"pos": s["pos"], "mask": s["mask"], "out": s["out"], "lse": s["lse"]}
    if c["op"] == "logprobs":
        ws = _kept(s, "ws", lambda: _bytes(abi.STATUS_BYTES))
        abi.csa2_token_logprobs(s["logits"], abi.OUT_BF16 if c["dtype"] == "bf16" else abi.OUT_F32, s["logits"].stride(0), c["rows"],
                                c["vocab"], c["scale"], s["tokens"] if c["given"] else None, c["given"],
                                s["logprobs"] if c["given"] else None, s["lse"], s["entropy"], c["top"],
                                s["ids"] if c["top"] else None, s["best"] if c["top"] else None, ws, ws.numel(), st)
        got = {"lse": s["lse"], "entropy": s["entropy"]}
        if c["given"]:
            got["logprobs"] = s["logprobs"]
        if c["top"]:
            got["ids"], got["best"] = s["ids"], s["best"]
        return got
    ws = _kept(s, "ws", lambda: _bytes(abi.STATUS_BYTES))
    abi.csa2_tree_commit(s["parent"], s["token"], s["choice"], s["q_start"], s["kv_len"], c["requests"], s["tokens"], s["max_q"], fmt,
                         s["codes"], s["scales"], s["n_rows"], s["table"], s["max_pages"], c["page"], s["free"], s["n_pages"],
                         s["n_free"], s["n_free_out"], s["cached"], s["path"], s["accepted"], s["next"], ws, ws.numel(), st)
    return {"path": s["path"], "accepted": s["accepted"], "next": s["next"], "cached": s["cached"], "free": s["free"],
            "n_free": s["n_free_out"], "codes": s["codes"], **({} if s["scales"] is None else {"scales": s["scales"]})}


PLAIN = {"heads": _heads_plain, "tree": _tree_plain, "logprobs": _logprobs_plain, "commit": _commit_plain}


def run(state):
    if own:
        return _run_own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------- work and 64 bits
def _host_lengths(case):
    """What _lengths() gives, as numbers: the mean cached length and every request's nodes."""
    n = case["requests"]
    part = [0.25 + 0.75 * i / n for i in range(1, n + 1)]
    nodes = [1 if case.get("mixed") and (n - 1 - i) % 2 else max(1, round(case["nodes"] * p)) for i, p in enumerate(part)]
    return case["cached"] * sum(part) / n, nodes


def work(case):
    op = case["op"]
    if op == "heads":
        T, H = case["tokens"], case["heads"]
        live = T - T // 16
        entry = 288 if case["fmt"] == "fp4" else 512
        return {"bytes": live * (H * 4 * D + 2 * D + entry + 16), "flops": live * (H + 1) * D * 8}
    if op == "tree":
        H, W = case["heads"], case["window"]
        entry = 288 if case["fmt"] == "fp4" else 512
        cached, lengths = _host_lengths(case)
        byte = flop = 0.0
        for n in lengths:
            # ancestors of a node, itself among them: all before it in a chain, a quarter by levels of four, a logarithm at random
            above = n / 2 if case["shape"] == "chain" else n / 8 + 1 if case["shape"] == "beam" else math.log(n) + 1
            old = min(cached, W) if W else cached
            byte += (old + n) * entry + n * H * (4 * D + 4) + 16 * n
            flop += n * H * min(old + above, W or math.inf) * 4 * D
        return {"bytes": byte, "flops": flop}
    if op == "logprobs":
        n, V = case["rows"], case["vocab"]
        return {"bytes": n * (V * (2 if case["dtype"] == "bf16" else 4) + 12 * case["given"] + 8 + 8 * case["top"]), "flops": 5 * n * V}
    _, lengths = _host_lengths(case)
    entry = 288 if case["fmt"] == "fp4" else 512
    # of a random tree's path about a logarithm of its nodes is kept, of a chain about five (0.8 each)
    moved = sum(0 if case["shape"] == "chain" else min(n / 4, 4) if case["shape"] == "beam" else math.log(n) for n in lengths)
    return {"bytes": 24 * sum(lengths) + 24 * len(lengths) + moved * 2 * entry, "flops": 0}


def _exact_rows(codes, scales, at):
    """float64 values of the rows `at`: sign, exponent and mantissa of each code spelled out."""
    if scales is None:
        return codes[at].view(torch.float8_e4m3fn).double()
    b = codes[at].to(torch.int32)
    c = torch.stack((b % 16, b // 16), 2).flatten(1)
    e, m = (c // 2) % 4, c % 2
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.pow(2.0, (e - 1).double()))
    sign = torch.where(c >= 8, -1.0, 1.0).double()
    return sign * mag * scales[at].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)


def _exact_heads(s):
    c, T = s["case"], s["case"]["tokens"]
    alive = int((s["pos"] >= 0).sum())  # the padded ones stand behind

    def whole(x, w, pos):
        y = x.double()
        if w is not None:
            y = w.double() * y / (y.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt()
        if c["rotate"]:  # as complex numbers
            i = torch.arange(D // 2, device="cuda", dtype=torch.float64)
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos.double()[:, None] * torch.exp(-2 * i / D * math.log(THETA)))
            y = torch.view_as_real(torch.view_as_complex(y.unflatten(-1, (-1, 2)).contiguous()) * turn.view(len(pos), *[1] * (y.dim() - 2), D // 2)).flatten(-2)
        return y

    q = torch.zeros(T, c["heads"], D, dtype=torch.float64, device="cuda")
    for i in range(0, alive, 512):
        j = min(alive, i + 512)
        q[i:j] = whole(s["q"][i:j], s["q_weight"], s["pos"][i:j])
    z = torch.zeros(s["n_rows"], D, dtype=torch.float64, device="cuda")
    z[s["dst"][:alive]] = whole(s["latents"][:alive], s["l_weight"], s["pos"][:alive])
    if c["fmt"] == "fp8":
        return {"q": q, "latents": z}
    return {"q": q, "latents": None, "scales": z.unflatten(1, (-1, 16)).abs().max(2).values / 6.0}  # (a code of 4 bits is no approximation of a number)


def _exact_tree(s):
    c = s["case"]
    H, P, W = c["heads"], c["page"], c["window"]
    starts, lens, parent = s["q_start"].tolist(), s["kv_len"].tolist(), s["parent"].tolist()
    outs, lses = [], []
    for r in range(c["requests"]):
        a, n, L = starts[r], starts[r + 1] - starts[r], lens[r]
        at = torch.cat([torch.arange(p * P, p * P + P, device="cuda") for p in s["table"][r, :_ceil(L, P)].tolist()])[:L]
        k = _exact_rows(s["codes"], s["scales"], at)
        first = L - n
        lines = []  # every node's way down to it
        for i in range(n):
            up = parent[a + i]
            lines.append((lines[up] if up >= 0 else []) + [i])
        for i in range(0, n, 64):
            m = min(64, n - i)
            see = torch.zeros(m, L, dtype=torch.bool)
            for j in range(m):
                line = lines[i + j]
                see[j, max(0, first + len(line) - W) if W else 0:first] = True
                see[j, [first + x for x in (line[-W:] if W else line)]] = True
            q = s["q"][a + i:a + i + m].double().flatten(0, 1)
            x = (q @ k.T / math.sqrt(D)).masked_fill(~see.cuda().repeat_interleave(H, 0), -math.inf)
            lse = torch.logsumexp(x, 1)
            outs.append((torch.exp(x - lse[:, None]) @ k).view(m, H, D))
            lses.append(lse.view(m, H))
    return {"pos": None, "mask": None, "out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_logprobs(s):
    c = s["case"]
    got = {"lse": [], "entropy": [], "logprobs": [], "best": []}
    for i in range(0, c["rows"], 128):
        x = s["logits"][i:i + 128].double() * c["scale"]
        lse = torch.logsumexp(x, 1)
        lp = x - lse[:, None]
        p = lp.exp()
        got["lse"].append(lse)
        got["entropy"].append(-(p * lp.clamp(min=-1e5)).sum(1))
        tok = s["tokens"][i:i + 128]
        got["logprobs"].append(lp.gather(1, tok.clamp(min=0)).masked_fill(tok < 0, -math.inf))
        got["best"].append(lp.topk(c["top"], 1).values)
    got = {k: torch.cat(v) for k, v in got.items()}
    if c["masked"]:  # where a logit is the type's lowest value, its log probability depends on how that is scaled
        low = torch.finfo(s["logits"].dtype).min / 4
        if bool((got["logprobs"] < low).logical_and(got["logprobs"] > -math.inf).any()) or bool(
                (got["best"] < low).logical_and(got["best"] > -math.inf).any()):
            got["logprobs"] = got["best"] = None
    if not c["given"]:
        del got["logprobs"]
    if c["top"]:
        got["ids"] = None
    else:
        del got["best"]
    return got


def exact(case, seed):
    if case["op"] == "commit":
        return None
    return {"heads": _exact_heads, "tree": _exact_tree, "logprobs": _exact_logprobs}[case["op"]](prepare(case, seed))
