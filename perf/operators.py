"""The operators of a layer step over a paged latent cache, as cases to measure:

* plan   - block tables, slot maps and positions of a step, from the requests' lengths
* attn   - causal attention of each request's new tokens over its pages (512-wide latents, keys = values)
* norm   - residual addition, root-mean-square norm and an E4M3 output with scales
* matvec - products of a few rows with FP4 weights (E2M1, one E4M3 scale per 16 channels)

run() computes an operator from elementary torch operations, or through the library where `own` is true.
"""
import math

import torch

own = False

D = 512  # latent width
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 16 requests with up to 128K cached entries: pure latency
        {"name": "plan decode 16", "op": "plan", "requests": 16, "page": 64, "cached": 131072, "added": 1, "mixed": False},
        # a step that takes in many prompts' chunks beside decoding requests
        {"name": "plan chunks 192", "op": "plan", "requests": 192, "page": 64, "cached": 16384, "added": 4096, "mixed": True},
        # single tokens of 16 requests, 64 heads, FP4 pages: the decode form
        {"name": "attn decode 16x8k", "op": "attn", "requests": 16, "heads": 64, "added": 1, "cached": 8192, "page": 64,
         "fmt": "fp4", "window": 0, "mixed": False},
        # one request takes in 512 tokens over 8K cached entries
        {"name": "attn chunk 512 on 8k", "op": "attn", "requests": 1, "heads": 64, "added": 512, "cached": 8192, "page": 64,
         "fmt": "fp4", "window": 0, "mixed": False},
        # decoding requests beside odd chunks, a quarter of the heads, E4M3 window latents
        {"name": "attn mixed window", "op": "attn", "requests": 12, "heads": 16, "added": 333, "cached": 3001, "page": 16,
         "fmt": "fp8", "window": 128, "mixed": True},
        # a long prompt's chunk: 1024 tokens over 16K cached entries
        {"name": "attn chunk 1024 on 16k", "op": "attn", "requests": 1, "heads": 64, "added": 1024, "cached": 15360, "page": 128,
         "fmt": "fp4", "window": 0, "mixed": False},
        # the hidden state of a decode batch, one scale per row (what the FP4 products take)
        {"name": "norm decode 16", "op": "norm", "rows": 16, "dim": 5120, "group": 0, "residual": True},
        # latents of a prompt's chunk, no residual
        {"name": "norm latents 8191", "op": "norm", "rows": 8191, "dim": 512, "group": 0, "residual": False},
        # the hidden state of a prompt's chunk, scales per 128 channels
        {"name": "norm chunk 4096", "op": "norm", "rows": 4096, "dim": 7168, "group": 128, "residual": True},
        # one token's latent projection
        {"name": "matvec 1 to 512", "op": "matvec", "rows": 1, "k": 5120, "n": 512, "x": "bf16", "out": "bf16"},
        # 16 tokens' queries of 64 heads x 512 from a compressed query, E4M3 activations
        {"name": "matvec 16 to 32768", "op": "matvec", "rows": 16, "k": 1536, "n": 32768, "x": "fp8", "out": "bf16"},
        # a wide projection for a few tokens
        {"name": "matvec 4 to 28672", "op": "matvec", "rows": 4, "k": 8192, "n": 28672, "x": "bf16", "out": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("plan", "attn", "attn", "norm", "matvec", "matvec"))
    if op == "plan":
        requests = _log(rng, 1, 256)
        return {"op": op, "requests": requests, "page": rng.choice((8, 16, 64, 128, 200)), "cached": _log(rng, 64, 131072),
                "added": _log(rng, 1, max(2, 400000 // requests)) if requests > 100 else _log(rng, 1, 4096),
                "mixed": rng.random() < 0.5}
    if op == "attn":
        heads = rng.choice((5, 8, 16, 24, 32, 64, 64, 128))
        requests = _log(rng, 1, 32)
        added = 1 if rng.random() < 0.35 else _log(rng, 2, 1024)
        cached = _log(rng, 16, 15360)
        # a drawn case stays below the largest listed one, padded to its longest request
        while requests * added * heads * (cached + added) > 1024 * 64 * 16384 // 2:
            if requests > 1 and added > 1:
                requests = max(1, requests // 2)
            elif added > 1:
                added = max(1, added // 2)
            else:
                cached //= 2
        return {"op": op, "requests": requests, "heads": heads, "added": added, "cached": cached,
                "page": rng.choice((8, 16, 64, 128, 200)), "fmt": rng.choice(("fp4", "fp4", "fp8")),
                "window": rng.choice((0, 0, 0, 100, 128, 1000)), "mixed": rng.random() < 0.6}
    if op == "norm":
        group = rng.choice((0, 128))
        dim = 128 * _log(rng, 2, 64) if group else 8 * _log(rng, 16, 1024)
        return {"op": op, "rows": min(_log(rng, 1, 8192), 4096 * 7168 // dim), "dim": dim, "group": group,
                "residual": rng.random() < 0.7}
    k, n = 128 * _log(rng, 2, 96), _log(rng, 64, 32768)
    return {"op": op, "rows": rng.choice((1, 1, 2, 3, 5, 8, 11, 16)), "k": k, "n": min(n, 8192 * 28672 // k),
            "x": rng.choice(("bf16", "fp8")), "out": rng.choice(("bf16", "f32"))}


# ----------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _lengths(case, g):
    """Per request (cached, added): spread evenly from about a quarter of the case's sizes to all of them and, where
    the case is mixed, every other request decodes one token; which request has which goes by the seed."""
    n = case["requests"]
    part = 0.25 + 0.75 * torch.arange(1, n + 1, device="cuda", dtype=torch.float64) / n
    cached = (case["cached"] * part).round().to(torch.int32)
    added = (case["added"] * part).round().to(torch.int32).clamp(min=1)
    if case["mixed"]:
        added[(n - 1 - torch.arange(n, device="cuda")) % 2 == 1] = 1
    return cached[torch.randperm(n, device="cuda", generator=g)], added[torch.randperm(n, device="cuda", generator=g)]


def _ceil(a, b):
    return (a + b - 1) // b


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


def prepare(case, seed):
    g = _gen(seed)
    op, dev = case["op"], "cuda"
    s = {"case": dict(case)}
    if op in ("plan", "attn"):
        P = case["page"]
        cached, added = _lengths(case, g)
        s["max_pages"] = max_pages = _ceil(case["cached"] + case["added"], P)
        total = int(added.sum())
    if op == "plan":
        n_req = case["requests"]
        held, after = _ceil(cached, P), _ceil(cached + added, P)
        n_pages = int(after.sum()) + 37
        ids = torch.randperm(n_pages, device=dev, generator=g).to(torch.int32)
        # the pages held so far, in each request's row; the rest are free
        j = torch.arange(max_pages, device=dev)
        base = torch.cumsum(held, 0) - held
        own_page = j[None, :] < held[:, None]
        table = torch.where(own_page, ids[(base[:, None] + j).clamp(max=n_pages - 1)], torch.full((), -1, dtype=torch.int32, device=dev))
        n_held = int(held.sum())
        free = torch.zeros(n_pages, dtype=torch.int32, device=dev)
        free[:n_pages - n_held] = ids[n_held:]
        s.update(cached=cached, added=added, table=table, free=free, n_pages=n_pages,
                 n_free=torch.tensor([n_pages - n_held], dtype=torch.int32, device=dev),
                 n_free_out=torch.zeros(1, dtype=torch.int32, device=dev),
                 q_start=torch.zeros(n_req + 1, dtype=torch.int32, device=dev),
                 kv_len=torch.zeros(n_req, dtype=torch.int32, device=dev),
                 max_new=total + 5)  # a step's buffers are a little larger than it needs
        s["slots"] = torch.zeros(s["max_new"], dtype=torch.int64, device=dev)
        s["pos"] = torch.zeros(s["max_new"], dtype=torch.int64, device=dev)
    elif op == "attn":
        n_req, H = case["requests"], case["heads"]
        pages = _ceil(cached + added, P)
        n_pages = int(pages.sum()) + 3
        ids = torch.randperm(n_pages, device=dev, generator=g).to(torch.int32)
        base = torch.cumsum(pages, 0) - pages
        j = torch.arange(max_pages, device=dev)
        s["table"] = torch.where(j[None, :] < pages[:, None], ids[(base[:, None] + j).clamp(max=n_pages - 1)],
                                 torch.full((), -1, dtype=torch.int32, device=dev))
        s["n_rows"] = n_rows = n_pages * P
        lat = torch.randn(n_rows, D, device=dev, generator=g)
        if case["fmt"] == "fp4":
            s["codes"], s["scales"] = _quantize_fp4(lat)
        else:
            s["codes"], s["scales"] = lat.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), None
        del lat
        s["kv_len"] = cached + added
        s["q_start"] = torch.zeros(n_req + 1, dtype=torch.int32, device=dev)
        s["q_start"][1:] = torch.cumsum(added, 0)
        s["tokens"], s["max_q"], s["max_kv"] = total, int(added.max()), int(s["kv_len"].max())
        s["q"] = torch.randn(total, H, D, device=dev, generator=g).to(torch.bfloat16)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(total, H, device=dev)
    elif op == "norm":
        n, d = case["rows"], case["dim"]
        amp = torch.exp(torch.randn(n, 1, device=dev, generator=g))
        s["x"] = (amp * torch.randn(n, d, device=dev, generator=g)).to(torch.bfloat16)
        s["res"] = (2 * amp * torch.randn(n, d, device=dev, generator=g)).to(torch.bfloat16) if case["residual"] else None
        s["res_out"] = torch.zeros_like(s["x"]) if case["residual"] else None
        s["w"] = (1 + 0.2 * torch.randn(d, device=dev, generator=g)).to(torch.bfloat16)
        s["codes"] = torch.zeros(n, d, dtype=torch.uint8, device=dev)
        s["scales"] = torch.zeros(n, d // 128 if case["group"] else 1, device=dev)
    else:
        n, k, m = case["rows"], case["k"], case["n"]
        s["codes"], s["wscales"] = _quantize_fp4(torch.randn(m, k, device=dev, generator=g))
        x = torch.randn(n, k, device=dev, generator=g) * torch.exp(torch.randn(n, 1, device=dev, generator=g))
        if case["x"] == "fp8":
            s["xscale"] = x.abs().amax(1) / 448.0
            s["x"] = (x / s["xscale"][:, None]).to(torch.float8_e4m3fn)
        else:
            s["x"], s["xscale"] = x.to(torch.bfloat16), None
        s["alpha"] = 1.0 / math.sqrt(k)
        s["out"] = torch.zeros(n, m, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device=dev)
    return s


# ------------------------------------------------------------- plain forms
def _values(codes, scales):
    """fp32 values [rows][2 * bytes] of FP4 rows, or of E4M3 rows where scales is None."""
    if scales is None:
        return codes.view(torch.float8_e4m3fn).float()
    mags = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = torch.stack((mags[(codes & 15).long()], mags[(codes >> 4).long()]), -1).view(codes.shape[0], -1)
    return (v.view(codes.shape[0], -1, 16) * scales.view(torch.float8_e4m3fn).float().unsqueeze(2)).view(codes.shape[0], -1)


def _plan_plain(s):
    P, cached, added = s["case"]["page"], s["cached"], s["added"]
    held, after = _ceil(cached, P), _ceil(cached + added, P)
    need = after - held
    first = torch.cumsum(need, 0) - need
    j = torch.arange(s["max_pages"], device="cuda")
    fresh = (j[None, :] >= held[:, None]) & (j[None, :] < after[:, None])
    at = (s["n_free"] - 1 - (first[:, None] + j[None, :] - held[:, None])).clamp(0, s["n_pages"] - 1)
    table = torch.where(fresh, s["free"][at.long()], s["table"])
    end = torch.cumsum(added, 0)
    i = torch.arange(s["max_new"], device="cuda")
    r = torch.searchsorted(end, i, right=True).clamp(max=len(cached) - 1)
    pos = cached[r].long() + i - (end[r] - added[r])
    inside = i < end[-1]
    safe = torch.where(inside, pos, 0)
    slots = table[r, safe // P].long() * P + safe % P
    q_start = torch.cat((torch.zeros(1, dtype=torch.int32, device="cuda"), end.to(torch.int32)))
    return {"table": table, "slots": torch.where(inside, slots, -1), "pos": torch.where(inside, pos, -1), "q_start": q_start,
            "kv_len": cached + added, "n_free": (s["n_free"] - need.sum()).to(torch.int32)}


def _attn_plain(s):
    c = s["case"]
    P, H, R = c["page"], c["heads"], c["requests"]
    added = s["q_start"][1:] - s["q_start"][:-1]
    p = torch.arange(s["max_kv"], device="cuda")
    page = s["table"][:, p // P].clamp(min=0).long()
    rows = page * P + p % P
    scales = None if s["scales"] is None else s["scales"][rows.view(-1)]
    k = _values(s["codes"][rows.view(-1)], scales).view(R, -1, D)
    i = torch.arange(s["max_q"], device="cuda")
    token = (s["q_start"][:-1, None] + i).clamp(max=s["tokens"] - 1)
    q = s["q"][token].float().view(R, -1, D)
    t = (s["kv_len"] - added)[:, None] + i  # the last position that new token i sees
    seen = p[None, None, :] <= t[:, :, None]
    if c["window"]:
        seen = seen & (p[None, None, :] > t[:, :, None] - c["window"])
    x = torch.matmul(q, k.transpose(1, 2)).mul_(1.0 / math.sqrt(D)).view(R, s["max_q"], H, -1)
    x.masked_fill_(~seen[:, :, None, :], -math.inf)
    top = x.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x.sub_(top).exp_()
    total = x.sum(3, keepdim=True)
    o = torch.matmul(x.view(R, -1, s["max_kv"]), k).view(R, s["max_q"], H, D) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).squeeze(3)
    live = i[None, :] < added[:, None]
    return {"out": o[live].to(torch.bfloat16), "lse": lse[live]}


def _norm_plain(s):
    c = s["case"]
    h = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(torch.bfloat16)
    f = h.double()  # codes next to a border between two E4M3 values
    y = f / torch.sqrt(f.square().mean(1, keepdim=True) + 1e-6) * s["w"].double()
    yg = y.view(y.shape[0], -1, 128 if c["group"] else y.shape[1])
    scale = (yg.abs().amax(2) / 448.0).float()
    safe = torch.where(scale == 0, 1.0, scale).double()
    codes = (yg / safe.unsqueeze(2)).clamp(-448, 448).to(torch.float8_e4m3fn).view(y.shape)
    got = {"codes": codes, "scales": scale}
    if s["res"] is not None:
        got["residual"] = h
    return got


def _matvec_plain(s):
    x = s["x"].float()
    if s["xscale"] is not None:
        x = x * s["xscale"][:, None]
    w = _values(s["codes"], s["wscales"])
    return (torch.matmul(x, w.t()) * s["alpha"]).to(s["out"].dtype)


# ------------------------------------------------------------ the library
def _workspace(s, size):
    if "ws" not in s:  # kept by a program for all its steps
        s["ws"] = torch.zeros(size(), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _run_own(s):
    from csa2_sparse_attention_gb300 import abi
    c, st = s["case"], torch.cuda.current_stream()
    if c["op"] == "plan":
        ws = _workspace(s, lambda: abi.STATUS_BYTES)
        abi.csa2_page_plan(s["cached"], s["added"], c["requests"], c["page"], s["table"], s["max_pages"], s["free"], s["n_pages"],
                           s["n_free"], s["n_free_out"], s["q_start"], s["kv_len"], s["slots"], s["pos"], s["max_new"],
                           ws, ws.numel(), st)
        return {"table": s["table"], "slots": s["slots"], "pos": s["pos"], "q_start": s["q_start"], "kv_len": s["kv_len"],
                "n_free": s["n_free_out"]}
    if c["op"] == "attn":
        ws = _workspace(s, lambda: abi.csa2_paged_attn_workspace_bytes(s["tokens"], c["heads"], c["requests"], s["max_q"], s["max_kv"],
                                                                       c["window"]))
        fmt = abi.FMT_FP4 if c["fmt"] == "fp4" else abi.FMT_FP8
        abi.csa2_paged_attn(s["q"], s["tokens"], c["heads"], s["q_start"], s["kv_len"], c["requests"], s["max_q"], s["max_kv"], fmt,
                            s["codes"], s["scales"], s["n_rows"], s["table"], s["max_pages"], c["page"], c["window"],
                            1.0 / math.sqrt(D), s["out"], s["lse"], ws, ws.numel(), st)
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "norm":
        n, d = c["rows"], c["dim"]
        abi.csa2_rmsnorm_fp8(s["x"], d, s["res"], s["res_out"], s["w"], n, d, 1e-6, c["group"], s["codes"], s["scales"], None, st)
        got = {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]}
        if s["res"] is not None:
            got["residual"] = s["res_out"]
        return got
    ws = _workspace(s, lambda: abi.csa2_fp4_matvec_workspace_bytes(c["rows"], c["k"], c["n"]))
    abi.csa2_fp4_matvec(s["x"], abi.X_BF16 if c["x"] == "bf16" else abi.X_E4M3, s["xscale"], c["k"], c["rows"], c["k"], s["codes"],
                        s["wscales"], c["n"], s["alpha"], s["out"], abi.OUT_BF16 if c["out"] == "bf16" else abi.OUT_F32,
                        ws, ws.numel(), st)
    return s["out"]


PLAIN = {"plan": _plan_plain, "attn": _attn_plain, "norm": _norm_plain, "matvec": _matvec_plain}


def run(state):
    if own:
        return _run_own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------- work and 64 bits
def _host_lengths(case):
    """What _lengths() gives, as numbers: the mean cached length and every request's new tokens."""
    n = case["requests"]
    part = [0.25 + 0.75 * i / n for i in range(1, n + 1)]
    added = [1 if case["mixed"] and (n - 1 - i) % 2 else max(1, round(case["added"] * p)) for i, p in enumerate(part)]
    return case["cached"] * sum(part) / n, added


def work(case):
    op = case["op"]
    if op == "plan":
        _, added = _host_lengths(case)
        return {"bytes": 24 * len(added) + 8 * sum(added) / case["page"] + 16 * sum(added), "flops": 0}
    if op == "attn":
        H, W = case["heads"], case["window"]
        entry = 288 if case["fmt"] == "fp4" else 512
        cached, lengths = _host_lengths(case)
        byte = flop = 0.0
        for n in lengths:
            keys, seen = cached + n, cached + n / 2
            if W:
                keys, seen = min(W + n, keys), min(W, seen)
            byte += keys * entry + n * H * (4 * D + 4)
            flop += n * H * seen * 4 * D
        return {"bytes": byte, "flops": flop}
    if op == "norm":
        n, d = case["rows"], case["dim"]
        return {"bytes": n * d * (7 if case["residual"] else 3) + 2 * d + 4 * n * (d // 128 if case["group"] else 1), "flops": 6 * n * d}
    n, k, m = case["rows"], case["k"], case["n"]
    return {"bytes": m * k * 9 / 16 + n * k * (2 if case["x"] == "bf16" else 1) + n * m * (2 if case["out"] == "bf16" else 4),
            "flops": 2 * n * k * m}


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


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None
    if case["op"] == "attn":
        H, P, W = case["heads"], case["page"], case["window"]
        starts, lens = s["q_start"].tolist(), s["kv_len"].tolist()
        outs, lses = [], []
        for r in range(case["requests"]):
            n, L = starts[r + 1] - starts[r], lens[r]
            at = torch.cat([torch.arange(p * P, p * P + P, device="cuda") for p in s["table"][r, :_ceil(L, P)].tolist()])[:L]
            c = _exact_rows(s["codes"], s["scales"], at)
            for i in range(0, n, 64):
                m = min(64, n - i)
                q = s["q"][starts[r] + i:starts[r] + i + m].double().flatten(0, 1)
                t = torch.arange(L - n + i, L - n + i + m, device="cuda").repeat_interleave(H)[:, None]
                lo = max(0, L - n + i + 1 - W) if W else 0
                p = torch.arange(lo, L, device="cuda")[None, :]
                hidden = p > t
                if W:
                    hidden = hidden | (p <= t - W)
                x = (q @ c[lo:].T / math.sqrt(D)).masked_fill(hidden, -math.inf)
                lse = torch.logsumexp(x, 1)
                outs.append((torch.exp(x - lse[:, None]) @ c[lo:]).view(m, H, D))
                lses.append(lse.view(m, H))
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}
    if case["op"] == "norm":
        x = s["x"].double()
        if s["res"] is not None:
            x = (x + s["res"].double()).to(torch.bfloat16).double()
        y = s["w"].double() * x * torch.rsqrt((x * x).sum(1, keepdim=True) / case["dim"] + 1e-6)
        parts = y.unflatten(1, (-1, case["group"] or case["dim"]))
        scale = parts.abs().max(2).values / 448.0
        got = {"codes": (parts / scale[..., None]).flatten(1), "scales": scale}
        if s["res"] is not None:
            got["residual"] = x
        return got
    x = s["x"].double()
    if s["xscale"] is not None:
        x = x * s["xscale"].double()[:, None]
    step = max(1, (1 << 26) // case["k"])
    rows = [torch.arange(i, min(case["n"], i + step), device="cuda") for i in range(0, case["n"], step)]
    return torch.cat([x @ _exact_rows(s["codes"], s["wscales"], at).T for at in rows], 1) * s["alpha"]
