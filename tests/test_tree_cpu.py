"""Refusals of the calls of a step of trees (every bad argument returns before any launch; the pointers are never
valid), what the Python layer refuses, and the 64-bit forms by hand-worked values."""
import numpy as np
import pytest
import torch

from oracle import tree_oracle as TO


@pytest.fixture(scope="module")
def abi():
    from csa2_sparse_attention_gb300 import build
    build.build()
    from csa2_sparse_attention_gb300 import abi as A
    return A


F = 1 << 20  # never dereferenced
FAR = 1 << 40


def args(defaults, **kw):
    d = dict(defaults)
    d.update(kw)
    return [d[k] for k in defaults]


HEADS = dict(q=F, q_stride=64 * 512, heads=64, qw=F, q_out=FAR, lat=2 * FAR, lat_stride=512, lw=F, n=4, eps=1e-6, pos=F, table=F,
             max_pos=100, fmt=0, dst=F, n_rows=64, codes=3 * FAR, scales=4 * FAR, ws=F, ws_bytes=256, stream=None)
PLAN = dict(parent=F, q_start=F, kv_len=F, n_req=2, n_tokens=40, max_q=33, window=0, pos=FAR, mask=2 * FAR, words=2, ws=F, ws_bytes=256,
            stream=None)
ATTN = dict(q=F, n_tokens=4, heads=64, q_start=F, kv_len=F, n_req=2, max_q=2, max_kv=100, pos=F, mask=F, words=1, fmt=0, codes=F,
            scales=F, n_rows=128, table=F, max_pages=8, page=16, window=0, sm_scale=0.04, out=FAR, lse=F, ws=F, ws_bytes=1 << 40,
            stream=None)
LOGP = dict(x=F, dtype=0, stride=1000, n=3, vocab=1000, scale=1.0, tokens=F, given=2, logprobs=FAR, lse=2 * FAR, entropy=3 * FAR, top=5,
            ids=4 * FAR, best=5 * FAR, ws=F, ws_bytes=256, stream=None)
COMMIT = dict(parent=F, token=F, choice=F, q_start=F, kv_len=F, n_req=2, n_tokens=9, max_q=5, fmt=0, codes=5 * FAR, scales=6 * FAR, n_rows=64,
              table=F, max_pages=4, page=16, free=7 * FAR, n_pages=4, n_free=8 * FAR, n_free_out=8 * FAR, cached=FAR, path=2 * FAR,
              accepted=3 * FAR, next=4 * FAR, ws=F, ws_bytes=256, stream=None)
STATUS = {"I": 1, "U": 2, "W": 6}


def refused(abi, name, defaults, kw, status):
    c0 = abi.csa2_launch_count()
    assert getattr(abi.lib, name)(*args(defaults, **kw)) == STATUS[status]
    assert abi.csa2_launch_count() == c0


@pytest.mark.parametrize("kw,status", [
    (dict(heads=0), "U"), (dict(heads=129, q_stride=129 * 512), "U"), (dict(q_stride=64 * 512 - 8), "I"), (dict(q_stride=64 * 512 + 4), "I"),
    (dict(q_out=None), "I"), (dict(q=None), "I"), (dict(q=None, q_out=None), "I"), (dict(q=None, q_out=None, qw=None, lat=None, lw=None), "I"),
    (dict(lat=None), "I"), (dict(q=F + 8), "I"), (dict(qw=F + 2), "I"), (dict(lat=F + 4), "I"), (dict(lw=F + 8), "I"), (dict(pos=F + 8), "I"),
    (dict(dst=F + 8), "I"), (dict(table=F + 8), "I"), (dict(pos=None), "I"), (dict(max_pos=0), "I"), (dict(max_pos=(1 << 31) + 1), "I"),
    (dict(n=-1), "I"), (dict(n=(1 << 22) + 1), "U"), (dict(n_rows=-1), "I"), (dict(eps=-1.0), "I"), (dict(eps=float("nan")), "I"),
    (dict(eps=float("inf")), "I"), (dict(lat_stride=504), "I"), (dict(lat_stride=516), "I"), (dict(fmt=2), "U"), (dict(fmt=1), "I"),
    (dict(scales=None), "I"), (dict(codes=None), "I"), (dict(dst=None, n_rows=3), "I"), (dict(ws=None), "W"), (dict(ws_bytes=255), "W"),
    (dict(ws=F + 8), "W"),
    (dict(q_out=F + 1024), "I"), (dict(q_out=F, q_stride=65 * 512), "I"), (dict(q_out=2 * FAR + 16), "I"), (dict(q_out=2 * FAR - 16), "I"),
    (dict(codes=2 * FAR), "I"), (dict(codes=FAR + 64), "I"), (dict(scales=3 * FAR + 64 * 256 - 16), "I"), (dict(scales=F), "I"),
    (dict(pos=FAR + 32), "I"), (dict(dst=3 * FAR), "I"), (dict(qw=FAR + 4096), "I"), (dict(table=4 * FAR - 64), "I")])
def test_head_refusals(abi, kw, status):
    refused(abi, "csa2_head_norm_rope", HEADS, kw, status)


@pytest.mark.parametrize("kw,status", [
    (dict(parent=None), "I"), (dict(parent=F + 4), "I"), (dict(q_start=None), "I"), (dict(kv_len=F + 8), "I"), (dict(pos=None), "I"),
    (dict(mask=None), "I"), (dict(mask=F + 4), "I"), (dict(words=1), "I"), (dict(words=3), "I"), (dict(window=-1), "I"), (dict(n_req=-1), "I"),
    (dict(n_tokens=-1), "I"), (dict(max_q=-1), "I"), (dict(max_q=1025, words=33), "U"), (dict(n_tokens=(1 << 22) + 1), "U"),
    (dict(n_req=(1 << 20) + 1), "U"), (dict(ws=None), "W"), (dict(ws_bytes=0), "W"), (dict(pos=F), "I"), (dict(mask=F + 16), "I"),
    (dict(mask=FAR + 8 * 40 - 16), "I"), (dict(q_start=FAR), "I"), (dict(kv_len=2 * FAR + 8 * 40 - 16), "I")])
def test_plan_refusals(abi, kw, status):
    refused(abi, "csa2_tree_plan", PLAN, kw, status)


@pytest.mark.parametrize("kw,status", [
    (dict(heads=0), "U"), (dict(heads=129), "U"), (dict(page=4), "U"), (dict(fmt=2), "U"), (dict(scales=None), "I"), (dict(fmt=1), "I"),
    (dict(q=None), "I"), (dict(pos=None), "I"), (dict(mask=None), "I"), (dict(pos=F + 8), "I"), (dict(mask=F + 4), "I"), (dict(words=2), "I"),
    (dict(words=0), "I"), (dict(max_q=-1), "I"), (dict(max_q=1025, words=33), "U"), (dict(out=F), "I"), (dict(window=-1), "I"),
    (dict(sm_scale=0.0), "I"), (dict(ws_bytes=255), "W"), (dict(max_kv=(1 << 30) + 1), "U")])
def test_attention_refusals(abi, kw, status):
    refused(abi, "csa2_tree_attn", ATTN, kw, status)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), "I"), (dict(x=F + 1), "I"), (dict(x=F + 2, dtype=1), "I"), (dict(dtype=2), "U"), (dict(stride=999), "I"), (dict(n=-1), "I"), (dict(vocab=0), "I"),
    (dict(vocab=(1 << 21) + 1, stride=1 << 22), "U"), (dict(n=(1 << 24) + 1), "U"), (dict(scale=0.0), "I"), (dict(scale=-1.0), "I"),
    (dict(scale=float("nan")), "I"), (dict(scale=float("inf")), "I"), (dict(scale=2.0 ** -21), "U"), (dict(scale=2.0 ** 21), "U"),
    (dict(given=-1), "I"), (dict(given=65), "U"), (dict(top=-1), "I"), (dict(top=65), "U"), (dict(tokens=None), "I"), (dict(logprobs=None), "I"),
    (dict(ids=None), "I"), (dict(best=None), "I"), (dict(tokens=F + 4), "I"), (dict(lse=FAR + 4), "I"), (dict(best=FAR + 8), "I"),
    (dict(ws=None), "W"), (dict(ws_bytes=255), "W"), (dict(lse=F), "I"), (dict(ids=F + 5984), "I"), (dict(entropy=F - 0 + 16), "I"),
    (dict(best=F - 32), "I"), (dict(logprobs=F + 2000), "I"), (dict(tokens=2 * FAR), "I"), (dict(entropy=2 * FAR), "I"),
    (dict(best=4 * FAR + 48), "I"), (dict(stride=(1 << 36) + 4), "I")])
def test_logprobs_refusals(abi, kw, status):
    refused(abi, "csa2_token_logprobs", LOGP, kw, status)


@pytest.mark.parametrize("kw,status", [
    *[({k: None}, "I") for k in ("parent", "token", "choice", "q_start", "kv_len", "table", "free", "n_free", "n_free_out", "cached", "path",
                                 "accepted", "next")],
    *[({k: F + 8}, "I") for k in ("parent", "token", "choice", "table", "free", "path", "next", "codes", "scales")],
    (dict(scales=None), "I"), (dict(codes=None), "I"), (dict(fmt=1), "I"), (dict(fmt=2), "U"), (dict(page=12), "U"), (dict(page=0), "U"),
    (dict(n_req=-1), "I"), (dict(n_tokens=-1), "I"), (dict(max_q=-1), "I"), (dict(n_rows=-1), "I"), (dict(max_pages=-1), "I"),
    (dict(n_pages=1 << 31), "I"), (dict(max_q=1025), "U"), (dict(n_req=(1 << 20) + 1), "U"), (dict(ws=None), "W"), (dict(ws_bytes=255), "W"),
    (dict(cached=F), "I"), (dict(accepted=F), "I"), (dict(accepted=FAR), "I"), (dict(path=F + 16), "I"), (dict(next=F + 64), "I"),
    (dict(free=F), "I"), (dict(codes=F - 64), "I"), (dict(scales=5 * FAR + 64 * 256 - 16), "I"), (dict(n_free_out=7 * FAR + 12), "I"),
    (dict(n_free=FAR + 4), "I"), (dict(table=2 * FAR + 32), "I"), (dict(next=3 * FAR), "I")])
def test_commit_refusals(abi, kw, status):
    refused(abi, "csa2_tree_commit", COMMIT, kw, status)


def test_empty_calls_launch_nothing(abi):
    c0 = abi.csa2_launch_count()
    for name, d, kws in (("csa2_head_norm_rope", HEADS, [dict(n=0)]), ("csa2_tree_plan", PLAN, [dict(n_req=0), dict(n_tokens=0), dict(max_q=0, words=0)]),
                         ("csa2_tree_attn", ATTN, [dict(n_req=0), dict(n_tokens=0), dict(max_q=0, words=0)]), ("csa2_token_logprobs", LOGP, [dict(n=0)]),
                         ("csa2_tree_commit", COMMIT, [dict(n_req=0)])):
        for kw in kws:
            assert getattr(abi.lib, name)(*args(d, **kw)) == abi.OK, (name, kw)
    assert abi.csa2_launch_count() == c0


def test_workspace_sizes(abi):
    size = abi.csa2_tree_attn_workspace_bytes
    assert size(0, 64, 0, 0, 0, 0) >= abi.STATUS_BYTES
    assert size(16, 64, 1, 16, 8192, 0) == abi.csa2_paged_attn_workspace_bytes(16, 64, 1, 16, 8192, 0)
    assert size(64, 64, 4, 16, 8192, 0) >= size(16, 64, 1, 16, 8192, 0)
    for bad in ((-1, 64, 1, 1, 1, 0), (1, 0, 1, 1, 1, 0), (1, 129, 1, 1, 1, 0), (1, 64, 1, 1025, 1, 0), (1, 64, 1, 1, -1, 0), (1, 64, 1, 1, 1, -1)):
        assert size(*bad) == 0, bad
    assert size(1 << 22, 128, 1 << 20, 1024, 1 << 30, 2 ** 31 - 1) >= 256


def test_cache_refusals(abi):
    """What does not fit the cache's buffers is refused before any call."""
    from csa2_sparse_attention_gb300 import paged
    c = paged.PagedLatents(2, 8, 4, 16, 2, heads=4, fmt=abi.FMT_FP8, device="cpu")
    bf, i32, i64 = torch.bfloat16, torch.int32, torch.int64
    q, lat = torch.zeros(8, 4, 512, dtype=bf), torch.zeros(8, 512, dtype=bf)
    par, tok = torch.zeros(8, dtype=i32), torch.zeros(8, dtype=i64)
    c0 = abi.csa2_launch_count()
    for bad in (lambda: c.append_heads(q, lat, 9), lambda: c.append_heads(q[:, :3], lat, 8), lambda: c.append_heads(q.float(), lat, 8),
                lambda: c.append_heads(q, lat[:, :256], 8), lambda: c.append_heads(q, lat, 8, q_norm=torch.zeros(256, dtype=bf)),
                lambda: c.append_heads(q, lat, 8, latent_norm=torch.zeros(512)), lambda: c.append_heads(q, lat, 8, eps=-1.0),
                lambda: c.append_heads(q, lat.to("meta"), 8), lambda: c.tree(par, 9, 4), lambda: c.tree(par, 8, 9), lambda: c.tree(par, 8, -1),
                lambda: c.tree(tok, 8, 4), lambda: c.tree(par[:4], 8, 4), lambda: c.attend_tree(q, 8, 9, 16), lambda: c.attend_tree(q, 9, 4, 16),
                lambda: c.attend_tree(q[:, :2], 8, 4, 16), lambda: c.attend_tree(q, 8, 4, 16), lambda: c.workspace(8, 4, (1 << 31) - 1, tree=True), lambda: c.workspace(8, 1025, 16, tree=True),
                lambda: c.commit(par, tok, tok[:3], 8, 4), lambda: c.commit(par, par, tok, 8, 4), lambda: c.commit(par, tok, tok, 8, 9),
                lambda: c.commit(tok, tok, tok, 8, 4), lambda: c.commit(par.to("meta"), tok, tok, 8, 4)):
        with pytest.raises(ValueError):
            bad()
    assert abi.csa2_launch_count() == c0


def test_layer_and_logprobs_refusals(abi):
    from csa2_sparse_attention_gb300 import paged
    bf = torch.bfloat16
    c = paged.PagedLatents(1, 4, 1, 8, 1, heads=1, fmt=abi.FMT_FP8, device="cpu")
    w = lambda *shape: torch.zeros(shape, dtype=bf)  # noqa: E731
    for kw in (dict(q_norm=w(256)), dict(latent_norm=torch.zeros(512)), dict(q_norm=w(512).to("meta"))):
        with pytest.raises(ValueError, match="_norm"):
            paged.PagedLayer(c, 256, w(256), w(512, 256), w(512, 256), **kw)
    for kw in (dict(max_rows=0), dict(max_rows=1, given=65), dict(max_rows=1, top=-1), dict(max_rows=1, top=65)):
        with pytest.raises(ValueError):
            paged.TokenLogprobs(device="cpu", **kw)
    p, g = paged.TokenLogprobs(4, top=2, device="cpu"), paged.TokenLogprobs(4, given=2, device="cpu")
    x, t = torch.zeros(4, 100), torch.zeros(4, 2, dtype=torch.int64)
    c0 = abi.csa2_launch_count()
    for bad in (lambda: p(torch.zeros(5, 100)), lambda: p(x.half()), lambda: p(x[0]), lambda: p(x.t()), lambda: p(x[:1].expand(4, 100)),
                lambda: p(x, tokens=t), lambda: g(x), lambda: g(x, tokens=t[:3]), lambda: g(x, tokens=t.int()), lambda: g(x, tokens=t[:, :1]),
                lambda: p(x.to("meta")), lambda: p(torch.zeros(4, 0))):
        with pytest.raises(ValueError):
            bad()
    assert abi.csa2_launch_count() == c0


# ------------------------------------------------- the 64-bit forms by hand
def test_plan_form_by_hand():
    #            0
    #          1   2        request 1: two roots, a bad parent and its child
    #         3     4
    parent = np.array([-1, 0, 0, 1, 2, -1, -1, 2, 2], np.int32)
    parent[7] = 5
    q_start, kv_len = np.array([0, 5, 9]), np.array([25, 4])
    pos, mask = TO.tree_plan(parent, q_start, kv_len, 0, 1, np.full(9, -9), np.full((9, 1), -9, np.int32))
    assert pos.tolist() == [20, 21, 21, 22, 22, 0, 0, -1, -1]
    assert mask[:, 0].tolist() == [1, 3, 5, 11, 21, 1, 2, 0, 0]
    pos, mask = TO.tree_plan(parent, q_start, kv_len, 2, 1, pos, mask)
    assert mask[:, 0].tolist() == [1, 3, 5, 10, 20, 1, 2, 0, 0]


def test_attention_form_of_a_chain_is_the_causal_one():
    from oracle import paged_oracle as PO
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 120, (40, 512)).astype(np.uint8)
    table = np.array([[3, 0, 4]], np.int32)
    q = rng.standard_normal((6, 2, 512)).astype(np.float32)
    for window in (0, 3, 9):
        a = TO.tree_attention(q, np.arange(-1, 5), [0, 6], [20], codes, None, table, 8, window, 0.04)
        b = PO.paged_attention(q, [0, 6], [20], codes, None, table, 8, window, 0.04)
        for x, y in zip(a[:2] + a[2], b[:2] + b[2]):
            np.testing.assert_array_equal(x, y)


def test_logprobs_form_by_hand():
    x = np.array([[0.0, np.log(3.0), -np.inf, np.log(3.0), 0.0], [-np.inf] * 5, [0, 1, np.nan, 0, 0]])
    lp, lse, ent, ids, best = TO.token_logprobs(x, 1.0, np.array([[1, -1], [0, 0], [0, 0]]), 5)
    assert ids.tolist() == [[1, 3, 0, 4, -1], [-1] * 5, [-1] * 5]
    np.testing.assert_allclose(np.exp(best[0]), [3 / 8, 3 / 8, 1 / 8, 1 / 8, 0])
    np.testing.assert_allclose([np.exp(lp[0, 0]), np.exp(lse[0])], [3 / 8, 8])
    np.testing.assert_allclose(ent[0], -(2 * 3 / 8 * np.log(3 / 8) + 2 / 8 * np.log(1 / 8)))
    assert np.isneginf(lp[0, 1]) and np.isneginf(lse[1]) and ent[1] == 0 and np.isnan(lse[2]) and np.isnan(best[2]).all()


def test_commit_form_by_hand():
    parent = np.array([-1, 0, 0, 2, 2, 4, -1, 0], np.int32)   # request 0: 0 -> {1, 2}, 2 -> {3, 4}, 4 -> 5; request 1: 0 -> 1
    token = np.array([9, 7, 8, 5, 6, 6, 1, 2])
    choice = np.array([8, 0, 6, 0, 6, 3, 4, 0])
    q_start, kv_len = np.array([0, 6, 8]), np.array([10, 9])
    table = np.array([[2, 0], [1, 3]], np.int32)
    plane = np.arange(32)[:, None]
    path, acc, nxt, cached, free, n_free, (moved,) = TO.tree_commit(parent, token, choice, q_start, kv_len, 8, [plane], table,
                                                                    np.full(4, -7), 0, 4, np.zeros(2), 8)
    assert path.tolist() == [0, 2, 4, 5, -1, -1, 0, -1] and acc.tolist() == [4, 1] and nxt.tolist() == [3, 4]
    assert cached.tolist() == [8, 8] and free.tolist() == [3, 0, -7, -7] and n_free == 2
    # request 0's entries 4 .. 7 are rows 20 .. 23; nodes 0, 2, 4, 5 lay in entries 4, 6, 8, 9: rows 20, 22, 0, 1
    assert moved[20:24, 0].tolist() == [20, 22, 0, 1]
