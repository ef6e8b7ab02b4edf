"""Calls of a step of trees at the ends of what they document: requests whose bounds do not hold, requests without keys,
steps without tokens, the smallest and largest values; the forms and bounds are those of test_gpu_tree.py."""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO
from oracle import tree_oracle as TO
from tests.test_gpu_paged import attn_inputs
from tests.test_gpu_tree import SM, U, Commit, Heads, Tree, abi, dev, f64, tree_layer, trees, walk_inputs  # noqa: F401

pytestmark = pytest.mark.gpu
D = 512


# ------------------------------------------------------------- head norms
def set_rows(h, q, lat):
    """The values of q [n][heads * 512] and lat [n][512] as the call's inputs."""
    h.q[:, :h.heads * D] = torch.from_numpy(q).to(torch.bfloat16).cuda()
    h.lat[:, :D] = torch.from_numpy(lat).to(torch.bfloat16).cuda()
    h.x64, h.lat64 = f64(h.q)[:h.n, :h.heads * D].reshape(h.n, h.heads, D), f64(h.lat)[:h.n, :D]


@pytest.mark.parametrize("fmt,turn", [("fp4", True), ("fp4", False), ("fp8", True)])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_heads_at_the_largest_values(abi, fmt, turn, eps):
    """Values up to 2^56: rows that are full of them, of one alone, and random ones; the bounds of Heads.check hold (sums of
    squares reach 512 * 2^112, far below fp32's largest number)."""
    rng = np.random.default_rng(23)
    h = Heads(abi, rng, 24, 3, fmt, turn=turn)
    most = 2.0 ** 56
    q, lat = (np.clip(2.0 ** 55 * rng.standard_normal((24, w)), -most, most) for w in (3 * D, D))
    for x in (q, lat):
        x[0] = most
        x[1] = np.where(rng.random(x.shape[1]) < 0.5, most, -most)
        x[2] = 0
        x[2, ::D] = -most
        x[3, 5::D] = most
    set_rows(h, q, lat)
    assert h.q.abs().max() == most and h.lat.abs().max() == most
    h.call(eps=eps).check(eps=float(np.float32(eps)))


@pytest.mark.parametrize("fmt,turn", [("fp4", True), ("fp4", False), ("fp8", True)])
def test_heads_at_the_smallest_rows_without_eps(abi, fmt, turn):
    """Rows whose largest value is 2^-60, eps 0.  The mean of the squares of k such values is k 2^-129, where fp32 steps by
    2^-149: off by 2^-21 / k relative, its root by 2^-22 / k.  Where k is small the sum of squares rounds less for it (k - 1
    times): root 2^-24 ((k - 1) / 2 + 4 / k) below the 5 * 2^-24 that are counted for it up to k = 10, and beyond that the
    mean's part is below 2^-25."""
    rng = np.random.default_rng(24)
    h = Heads(abi, rng, 24, 3, fmt, turn=turn)
    least = 2.0 ** -60
    q, lat = (np.clip(2.0 ** -61 * rng.standard_normal((24, w)), -least, least) for w in (3 * D, D))
    for x in (q, lat):
        x[:, 7::D] = least  # in every row and head
        x[0] = least
        x[1] = 0
        x[1, ::D] = -least
        for k in range(2, 12):
            x[k] = 0
            for j in range(k):
                x[k, 40 * j::D] = least * (1 if j else 1.5)
        x[12] = 2.0 ** -75 * rng.standard_normal(x.shape[1])
        x[12, 100::D] = least
        x[13] = 2.0 ** -120 * rng.standard_normal(x.shape[1])
        x[13, 200::D] = 1.25 * least
    set_rows(h, q, lat)
    h.call(eps=0.0).check(eps=0.0)


# ------------------------------------------------------------------ commit
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("what,value", [
    ("kv_len", 0), ("kv_len", 6), ("kv_len", 29), ("kv_len", -1), ("kv_len", -200), ("kv_len", -2 ** 31), ("kv_len", 2 ** 31 - 1),
    ("q_start", 970), ("q_start", 2 ** 31 - 1), ("q_start", -3), ("q_start", -2 ** 31)])
def test_commit_gives_no_pages_back_for_bad_requests(abi, fmt, what, value):
    """A request that begins many pages below its first entry, or whose tokens lie anywhere: its neighbours, the free list and
    the planes are as if it had brought nothing."""
    c = Commit(abi, np.random.default_rng(21), [20, 9, 4, 33], [30, 30, 7, 12], 8, fmt, vocab=2)
    q_start, kv_len = c.q_start.copy(), c.kv_len.copy()
    bad = (1,) if what == "kv_len" else (0, 1)  # q_start[1] ends request 0 and begins request 1
    getattr(c, what)[1] = value
    c.upload().call()
    torch.cuda.synchronize()
    path, acc, nxt, cached, free, n_free, planes = TO.tree_commit(
        c.parent, c.token, c.choice, q_start, kv_len, 8, c.planes, c.table, c.free, c.n_free, c.n_pages, c.cached0, c.T, bad)
    for got, want in ((c.accepted, acc), (c.next, nxt), (c.cached, cached), (c.nf, [n_free]), (c.d["free"], free), (c.d["table"], c.table)):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    for got, want in zip(c.dp, planes):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    got = c.path.cpu().numpy()
    held = q_start[1] if what == "kv_len" else q_start[2]  # (tokens whose bounds do not hold have no path)
    np.testing.assert_array_equal(got[held:c.T], path[held:])
    np.testing.assert_array_equal(got[:held], path[:held] if what == "kv_len" else np.full(held, -7))
    assert (got[c.T:] == -7).all()
    assert abi.csa2_status_fetch(c.ws)[0] == abi.ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("added", [[0, 0, 0], [4, 0, 6]])
def test_steps_without_tokens_are_committed(abi, added):
    """A step of no tokens, first of all and after one that had some, through the layer and the cache: nothing is accepted,
    lengths, pages and entries stay."""
    paged, g, cache, layer = tree_layer(abi, abi.FMT_FP4, 0, True)
    if any(added):
        n = sum(added)
        cache.added.copy_(torch.tensor(added, dtype=torch.int32))
        par = dev(trees(np.random.default_rng(0), added, "chain"))
        layer.step(torch.randn(n, 256, generator=g).to(torch.bfloat16).cuda(), n, max(added), max(added), parent=par)
        tok = torch.zeros(n, dtype=torch.int64, device="cuda")
        cache.commit(par, tok, tok, n, max(added))
        torch.cuda.synchronize()
        assert cache.accepted.tolist() == added and cache.next.tolist() == [0, -1, 0]
    before = [x.clone() for x in (cache.cached, cache.n_free, cache.free, cache.codes, cache.scales, cache.table, cache.path)]
    assert cache.cached.tolist() == added
    cache.added.zero_()
    none = lambda t: torch.zeros(0, dtype=t, device="cuda")  # noqa: E731
    out, lse = layer.step(torch.zeros((0, 256), dtype=torch.bfloat16, device="cuda"), 0, 0, 10, parent=none(torch.int32))
    path, accepted, nxt = cache.commit(none(torch.int32), none(torch.int64), none(torch.int64), 0, 0)
    torch.cuda.synchronize()
    assert len(out) == len(path) == 0 and accepted.tolist() == [0, 0, 0] and nxt.tolist() == [-1, -1, -1]
    for a, b in zip((cache.cached, cache.n_free, cache.free, cache.codes, cache.scales, cache.table, cache.path), before):
        assert torch.equal(a, b)
    for name, st in cache.status().items():
        assert st[0] == abi.OK, (name, st)


def test_step_of_a_view_off_a_boundary_changes_nothing(abi):
    """parents that the masks' call would refuse, once residual and pages had changed: refused before, and the next step is as
    if nothing had been."""
    paged, g, cache, layer = tree_layer(abi, abi.FMT_FP4, 0, True)
    nodes = [5, 0, 7]
    cache.added.copy_(torch.tensor(nodes, dtype=torch.int32))
    par = torch.zeros(16, dtype=torch.int32, device="cuda")
    par[3:15] = dev(trees(np.random.default_rng(0), nodes))
    x = torch.randn(12, 256, generator=g).to(torch.bfloat16).cuda()
    held = (layer.residual, cache.cached, cache.n_free, cache.free, cache.table, cache.kv_len, cache.q_start, cache.pos, cache.codes)
    before = [t.clone() for t in held]
    with pytest.raises(ValueError, match="not 16-byte aligned"):
        layer.step(x, 12, 7, 10, parent=par[3:])
    torch.cuda.synchronize()
    for a, b in zip(held, before):
        assert torch.equal(a, b)
    layer.step(x, 12, 7, 10, parent=par[3:].clone())
    torch.cuda.synchronize()
    assert cache.kv_len.tolist() == nodes


def test_commit_of_no_tokens_records_what_is_left_of_others(abi):
    """Without tokens, token bounds of an earlier step do not hold: recorded, and nothing is read or moved."""
    c = Commit(abi, np.random.default_rng(22), [20, 9], [3, 7], 8, "fp4").upload()
    a, d = abi, c.d
    a.csa2_tree_commit(None, None, None, d["q_start"], d["kv_len"], 2, 0, 7, a.FMT_FP4, c.dp[0], c.dp[1], c.planes[0].shape[0], d["table"],
                       c.max_pages, 8, d["free"], c.n_pages, c.nf, c.nf, c.cached, None, c.accepted, c.next, c.ws, c.ws.numel())
    torch.cuda.synchronize()
    assert c.accepted.tolist() == [0, 0] and c.next.tolist() == [-1, -1] and c.cached.tolist() == c.cached0.tolist()
    assert int(c.nf.item()) == c.n_free and (d["free"].cpu().numpy() == c.free).all()
    for got, want in zip(c.dp, c.planes):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    assert a.csa2_status_fetch(c.ws)[0] == a.ERR_DEVICE_BOUNDS


# --------------------------------------------------------------- attention
def requests_of(q_start, r):
    return slice(int(q_start[r]), int(q_start[r + 1]))


# (the few-row kernel twice, row tiles; all by shares)
@pytest.mark.parametrize("n_req,nodes,cached,spread", [(32, 8, 2048, 1), (32, 8, 2048, 40), (24, 16, 3100, 40)])
@pytest.mark.parametrize("empty", ["no entries", "too many", "negative"])
def test_attention_writes_requests_without_keys(abi, n_req, nodes, cached, spread, empty):
    """Several requests' trees laid out by their lengths, one of them without keys, each in turn: its rows are zeros and -inf
    wherever a group's share ends, and the others' are as with all of them."""
    rng = np.random.default_rng(n_req)
    n = [nodes] * n_req
    s = attn_inputs(rng, cached - rng.integers(0, spread, n_req) + n, n, 64, 64, "fp4", tail=1)
    t = Tree(abi, s, trees(rng, n)).call()
    assert t.check()[0] == abi.OK
    out, lse = t.out.clone(), t.lse.clone()
    big = float(out[:s["q_start"][-1]].abs().max())
    for r in range(n_req):
        kv = s["kv_len"].copy()
        kv[r] = {"no entries": 0, "too many": s["max_kv"] + 1 + r, "negative": -1 - 300 * r}[empty]
        t.kv_len.copy_(dev(kv))
        t.out.fill_(7.0)
        t.lse.fill_(7.0)
        t.call()
        torch.cuda.synchronize()
        own = requests_of(s["q_start"], r)
        assert (t.out[own] == 0).all() and torch.isneginf(t.lse[own]).all(), r
        others = torch.ones(s["T"], dtype=torch.bool, device="cuda")
        others[own] = False
        assert (t.out[others].float() - out[others].float()).abs().max() <= 2.0 ** -6 * big, r
        assert (t.lse[others] - lse[others]).abs().max() <= 2.0 ** -14, r
        assert abi.csa2_status_fetch(t.ws)[0] == abi.ERR_DEVICE_BOUNDS
        abi.csa2_status_reset(t.ws)


@pytest.mark.parametrize("n_req,H,kind,longest,window", [
    (40, 8, "few", 1300, 0), (33, 64, "few", 1200, 1050), (150, 8, "few", 1100, 0), (12, 64, "tiles", 3300, 0), (35, 32, "tiles", 3300, 3200)])
@pytest.mark.parametrize("seed", range(3))
def test_attention_walks_over_many_requests_without_keys(abi, n_req, H, kind, longest, window, seed):
    """Half of the requests have fewer entries than nodes or none, at random, beside short and long ones."""
    rng = np.random.default_rng(seed)
    s, parent = walk_inputs(rng, n_req, H, kind, longest, 16, "fp4")
    nodes = np.diff(s["q_start"])
    for r in np.flatnonzero(rng.random(n_req) < 0.5):
        if r != n_req // 2 and nodes[r] > 0:
            s["kv_len"][r] = 0 if rng.random() < 0.7 else rng.integers(0, nodes[r])
    t = Tree(abi, s, parent, window).call()
    t.check()


@pytest.mark.parametrize("n_req,H,kind,longest,page,fmt,window", [
    (3, 16, "few", 5000, 64, "fp8", 0), (33, 8, "few", 1500, 8, "fp4", 0), (40, 8, "few", 1300, 8, "fp8", 1050),
    (600, 8, "few", 1200, 8, "fp4", 0), (2, 64, "tiles", 3400, 64, "fp4", 0), (5, 64, "tiles", 4100, 16, "fp8", 3200),
    (35, 32, "tiles", 3300, 16, "fp4", 0)])
def test_attention_walks_write_every_row_again(abi, n_req, H, kind, longest, page, fmt, window):
    """A second call over outputs that hold something else gives the first one's bits."""
    rng = np.random.default_rng(n_req + H)
    s, parent = walk_inputs(rng, n_req, H, kind, longest, page, fmt)
    t = Tree(abi, s, parent, window).call()
    torch.cuda.synchronize()
    out, lse = t.out.clone(), t.lse.clone()
    t.out.fill_(5.0)
    t.lse.fill_(5.0)
    t.call()
    torch.cuda.synchronize()
    T = int(s["q_start"][-1])
    assert torch.equal(out[:T], t.out[:T]) and torch.equal(lse[:T], t.lse[:T]) and (t.out[T:] == 5).all() and (t.lse[T:] == 5).all()


@pytest.mark.parametrize("cached,nodes,H,window", [
    ([130, 301], [40, 9], 16, 20), ([700], [16], 64, 100), ([1500, 1290, 40], [12, 40, 3], 8, 1050), ([900, 1000], [90, 70], 64, 300),
    ([3500, 3300], [70, 66], 64, 3100)])
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_attention_positions_of_the_caller(abi, cached, nodes, H, window, fmt):
    """Positions that csa2_tree_plan does not give: below the request's first node, where they count as that one's, and above
    the node's place, where they count as it.  (Both kernels, split as for one request and for several.)"""
    rng = np.random.default_rng(25)
    s = attn_inputs(rng, np.asarray(cached) + nodes, nodes, H, 16, fmt)
    parent = trees(rng, nodes)
    t = Tree(abi, s, parent, window).plan()
    mask = np.zeros((s["T"], t.words), np.uint64)
    see, low = [], []
    for r, n in enumerate(nodes):
        a, first = int(s["q_start"][r]), cached[r]
        for i in range(n):
            p = int(rng.choice([0, max(0, first - window), max(0, first - 9), first - 1, first, first + i // 2, first + i, first + i + 1, 1 << 40]))
            t.pos[a + i] = p
            own = np.flatnonzero(rng.random(i + 1) < 0.3)
            for j in own:
                mask[a + i, j // 32] |= np.uint64(1 << (j % 32))
            low.append(max(0, min(max(p, first), first + i) + 1 - window))
            see.append(np.concatenate([np.arange(low[-1], first), first + own]))
    t.mask.copy_(dev(mask.astype(np.uint32).view(np.int32)))
    t.plan = lambda stream=None: t
    t.call()
    torch.cuda.synchronize()
    assert abi.csa2_status_fetch(t.ws)[0] == abi.OK
    out, lse, q = f64(t.out), f64(t.lse), f64(t.q)
    for r, n in enumerate(nodes):
        a = int(s["q_start"][r])
        p = np.arange(cached[r] + n)
        rows = s["table"][r, p // 16].astype(np.int64) * 16 + p % 16
        c = PO.latent_rows(s["codes"][rows], None if s["scales"] is None else s["scales"][rows])
        for i in range(a, a + n):
            k = c[see[i]]
            x = SM * q[i] @ k.T
            m = x.max(1, keepdims=True)
            e = np.exp(x - m)
            want, wl = e / e.sum(1, keepdims=True) @ k, (m + np.log(e.sum(1, keepdims=True)))[:, 0]
            d = 64 * U * np.max(np.abs(q[i]) @ np.abs(k).T) * SM + 2.0 ** -21  # (as in Tree.check)
            big = np.abs(k).max()
            assert (np.abs(out[i] - want) <= (2 * d + 2.0 ** -11 + len(p) * U) * big + (2.0 ** -8 + len(p) * U) * np.abs(want)).all(), (r, i - a)
            assert (np.abs(lse[i] - wl) <= d + len(p) * U + 2.0 ** -22 * (1 + np.abs(wl))).all(), (r, i - a)
