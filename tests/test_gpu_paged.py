"""The operators of a step over a paged cache against their 64-bit forms:
page planning, causal attention of a chunk of new tokens over the pages,
residual norm to E4M3, and FP4 products, at the sizes and masks where they
can go wrong; graphs, streams and a whole step of them together."""
import math

import numpy as np
import pytest
import torch

from oracle import csa2_oracle as O
from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu
D = 512
SM = 1.0 / math.sqrt(D)


@pytest.fixture(scope="module")
def abi():
    from csa2_sparse_attention_gb300 import abi as A
    return A


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def fresh_ws(abi, n):
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    abi.csa2_status_reset(ws)
    return ws


# --------------------------------------------------------------- page plan
def plan_inputs(rng, cached, added, page, spare=3, extra_pages=2):
    cached, added = np.asarray(cached, np.int32), np.asarray(added, np.int32)
    pages = lambda n: -(-n.astype(np.int64) // page)  # noqa: E731
    held, after = pages(cached), pages(cached + added)
    max_pages = int(after.max(initial=1)) + extra_pages
    n_pages = int(after.sum()) + spare
    ids = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(cached), max_pages), -7, np.int32)
    at = 0
    for r in range(len(cached)):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    free = np.full(n_pages, -9, np.int32)
    free[:n_pages - at] = ids[at:]
    return cached, added, table, free, n_pages - at, n_pages


def run_plan(abi, cached, added, page, table, free, n_free, n_pages, max_new, alias=True, stream=None):
    R = len(cached)
    t, nf = dev(table), dev(np.array([n_free], np.int32))
    nfo = nf if alias else torch.full((1,), -5, dtype=torch.int32, device="cuda")
    qs = torch.full((R + 1,), -5, dtype=torch.int32, device="cuda")
    kl = torch.full((max(R, 1),), -5, dtype=torch.int32, device="cuda")
    sl = torch.full((max(max_new, 1),), -5, dtype=torch.int64, device="cuda")
    po = torch.full((max(max_new, 1),), -5, dtype=torch.int64, device="cuda")
    ws = fresh_ws(abi, abi.STATUS_BYTES)
    c, a = dev(cached), dev(added)
    abi.csa2_page_plan(c if R else None, a if R else None, R, page, t if t.numel() else None, table.shape[1], dev(free) if n_pages else None, n_pages,
                       nf, nfo, qs, kl if R else None, sl if max_new else None, po if max_new else None, max_new, ws,
                       ws.numel(), stream)
    torch.cuda.synchronize()
    return (t.cpu().numpy(), qs.cpu().numpy(), kl.cpu().numpy()[:R], sl.cpu().numpy()[:max_new],
            po.cpu().numpy()[:max_new], int(nfo.item()), abi.csa2_status_fetch(ws))


def check_plan(got, want):
    for g, w in zip(got[:5], want[:5]):
        np.testing.assert_array_equal(g, w)
    assert got[5] == want[5]


@pytest.mark.parametrize("case", [
    ("one token", [0], [1], 8, 0), ("page full", [16, 15, 17], [1, 1, 1], 16, 2), ("nothing new", [5, 0, 9], [0, 0, 0], 8, 3),
    ("zeros between", [0, 40, 8, 7, 0], [3, 0, 9, 0, 65], 8, 1), ("page of 200", [199, 200, 401], [2, 400, 1], 200, 0),
    ("no room behind", [3, 100], [50, 28], 64, 0)])
@pytest.mark.parametrize("alias", [True, False])
def test_plan_small(abi, case, alias):
    _, cached, added, page, tail = case
    rng = np.random.default_rng(len(cached) + page)
    args = plan_inputs(rng, cached, added, page)
    cached, added, table, free, n_free, n_pages = args
    max_new = int(added.sum()) + tail
    got = run_plan(abi, cached, added, page, table, free, n_free, n_pages, max_new, alias)
    check_plan(got, PO.page_plan(cached, added, page, table, free, n_free, n_pages, max_new))
    assert got[6][0] == abi.OK


@pytest.mark.parametrize("R,page,top", [(1, 64, 70000), (257, 16, 300), (600, 128, 90), (1030, 8, 40)])
def test_plan_many(abi, R, page, top):
    rng = np.random.default_rng(R)
    cached, added = rng.integers(0, 500, R), rng.integers(0, top + 1, R)
    added[rng.random(R) < 0.3] = 0
    if R == 1:
        added[0] = top
    cached, added, table, free, n_free, n_pages = plan_inputs(rng, cached, added, page)
    max_new = int(added.sum()) + 1000
    got = run_plan(abi, cached, added, page, table, free, n_free, n_pages, max_new)
    check_plan(got, PO.page_plan(cached, added, page, table, free, n_free, n_pages, max_new))
    assert got[6][0] == abi.OK


@pytest.mark.parametrize("what", ["pages", "tokens", "negative", "row", "free count"])
def test_plan_that_cannot_be_served_takes_nothing(abi, what):
    rng = np.random.default_rng(5)
    cached, added, table, free, n_free, n_pages = plan_inputs(rng, [9, 30, 2], [20, 1, 3000], 8, extra_pages=0)
    max_new = int(added.sum()) + 4
    if what == "pages":
        n_free = 100
    elif what == "tokens":
        max_new = int(added.sum()) - 1
    elif what == "negative":
        added[1] = -1
    elif what == "row":
        added[1] = 4000
        max_new = 8000
    else:
        n_free = n_pages + 1
    got = run_plan(abi, cached, added, 8, table, free, n_free, n_pages, max_new)
    want = PO.page_plan(cached, added, 8, table, free, n_free, n_pages, max_new)
    assert not want[6]
    check_plan(got, want)
    assert got[6][0] == abi.ERR_DEVICE_BOUNDS


def test_plan_bad_page_ids_give_no_slots(abi):
    rng = np.random.default_rng(6)
    cached, added, table, free, n_free, n_pages = plan_inputs(rng, [9, 30], [20, 5], 8)
    table[0, 1] = n_pages       # the half-filled page of request 0
    free[n_free - 1] = -3       # its first new page
    got = run_plan(abi, cached, added, 8, table, free, n_free, n_pages, 40)
    want = PO.page_plan(cached, added, 8, table, free, n_free, n_pages, 40)
    check_plan(got, want)
    assert (want[3][:7] == -1).all() and got[6][0] == abi.ERR_DEVICE_BOUNDS


def test_plan_empty(abi):
    z = np.zeros(0, np.int32)
    got = run_plan(abi, z, z, 8, np.zeros((0, 4), np.int32), np.arange(5, dtype=np.int32), 5, 5, 3)
    assert got[1].tolist() == [0] and got[3].tolist() == [-1] * 3 and got[5] == 5


# --------------------------------------------------------------- attention
def cache_rows(rng, n_rows, fmt, amp=1.0):
    x = amp * rng.standard_normal((n_rows, D)).astype(np.float32)
    if fmt == "fp8":
        return O.e4m3_encode(x.astype(np.float64)).astype(np.uint8), None
    t = torch.from_numpy(x).view(n_rows, D // 16, 16)
    s = (t.abs().amax(2) / 6.0).to(torch.float8_e4m3fn)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    c = torch.bucketize((t / s.float().clamp(min=2.0 ** -9).unsqueeze(2)).abs(), mids) | ((t < 0).long() << 3)
    c = c.view(n_rows, D).numpy().astype(np.uint8)
    return (c[:, 0::2] | (c[:, 1::2] << 4)), s.view(torch.uint8).numpy()


def attn_inputs(rng, kv_len, new, heads, page, fmt, q_amp=1.0, c_amp=1.0, tail=0):
    kv_len, new = np.asarray(kv_len, np.int32), np.asarray(new, np.int32)
    pages = -(-kv_len // page)
    n_pages, max_pages = int(pages.sum()) + 2, max(1, int(pages.max()))
    ids = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(kv_len), max_pages), -1, np.int32)
    at = 0
    for r, n in enumerate(pages):
        table[r, :n] = ids[at:at + n]
        at += n
    codes, scales = cache_rows(rng, n_pages * page, fmt, c_amp)
    q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(q_start[-1]) + tail
    q = bf16(q_amp * rng.standard_normal((max(T, 1), heads, D)))[:T]
    return dict(q=q, q_start=q_start, kv_len=kv_len, codes=codes, scales=scales, table=table, page=page, fmt=fmt, T=T, H=heads,
                max_q=int(new.max(initial=0)), max_kv=int(kv_len.max(initial=0)))


class Attn:
    """The device side of one attention call."""

    def __init__(self, abi, s, window=0, max_q=None, max_kv=None, ws=None, fill=7.0):
        self.abi, self.s, self.window = abi, s, window
        self.q, self.q_start, self.kv_len = s["q"].cuda(), dev(s["q_start"]), dev(s["kv_len"])
        self.codes, self.scales = dev(s["codes"]), None if s["scales"] is None else dev(s["scales"])
        self.table = dev(s["table"])
        self.max_q = s["max_q"] if max_q is None else max_q
        self.max_kv = s["max_kv"] if max_kv is None else max_kv
        self.out = torch.full((s["T"], s["H"], D), fill, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((s["T"], s["H"]), fill, device="cuda")
        size = abi.csa2_paged_attn_workspace_bytes(s["T"], s["H"], len(s["kv_len"]), self.max_q, self.max_kv, window)
        assert size >= abi.STATUS_BYTES
        self.ws = fresh_ws(abi, size) if ws is None else ws

    def call(self, stream=None, lse=True):
        s, abi = self.s, self.abi
        abi.csa2_paged_attn(self.q, s["T"], s["H"], self.q_start, self.kv_len, len(s["kv_len"]), self.max_q, self.max_kv,
                            abi.FMT_FP4 if s["fmt"] == "fp4" else abi.FMT_FP8, self.codes, self.scales,
                            self.codes.shape[0], self.table, s["table"].shape[1], s["page"], self.window, SM, self.out,
                            self.lse if lse else None, self.ws, self.ws.numel(), stream)

    def result(self):
        torch.cuda.synchronize()
        return self.out.float().cpu().numpy().astype(np.float64), self.lse.cpu().numpy().astype(np.float64)


def check_attn(out, lse, s, window, bad_page=None, tokens=None):
    """Against the 64-bit form.  With u = 2^-24: a logit is a 512-term fp32 sum of exact products, off by at most
    512 u sum|q||c| sm_scale (the true error grows with the square root; the bound is taken at 64 u), so the
    probabilities by a factor 1 + d, d = 64 u dot sm + 2^-21 (the exponential); they enter the product rounded to
    f16 (2^-11 relative, 2^-24 absolute below f16's normal range, against a sum of at least 1 for a largest
    probability of at least 1), whose sums are over |c| <= big: |o - o*| <= (2 d + 2^-11 + n 2^-24) big, then bf16
    rounds once: 2^-8 relative.  The sum of n positive terms in fp32 is off by at most n u relative in any order
    (each partial sum rounds once), which enters the logarithm as n u and the outputs as n u |o|."""
    T = int(s["q_start"][-1]) if tokens is None else tokens
    want, wlse, (dot, big) = PO.paged_attention(s["q"].float().numpy(), s["q_start"], s["kv_len"], s["codes"], s["scales"],
                                                s["table"], s["page"], window, SM, bad_page)
    d = 64 * 2.0 ** -24 * dot * SM + 2.0 ** -21
    tol = ((2 * d + 2.0 ** -11 + s["max_kv"] * 2.0 ** -24) * big)[..., None] + (2.0 ** -8 + s["max_kv"] * 2.0 ** -24) * np.abs(want)
    err = np.abs(out - want)[:T]
    assert np.isfinite(out[:T]).all()
    assert (err <= tol[:T]).all(), (err - tol[:T]).max()
    live = np.isfinite(wlse[:T])
    assert np.array_equal(np.isneginf(lse[:T]), ~live)
    assert (out[:T][~live] == 0).all()
    ltol = d + s["max_kv"] * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(np.where(np.isfinite(wlse), wlse, 0)))
    assert (np.abs(lse[:T][live] - wlse[:T][live]) <= ltol[:T][live]).all()


ATTN = [
    # kv_len, new, heads, page, fmt, window
    ([1], [1], 64, 8, "fp4", 0),
    ([1, 2, 127, 128, 129, 640], [1, 1, 1, 1, 1, 1], 64, 16, "fp4", 0),
    ([700], [130], 64, 64, "fp4", 0),
    ([300, 17, 64], [300, 17, 1], 5, 8, "fp4", 0),
    ([515, 1, 260], [3, 1, 2], 128, 128, "fp4", 0),
    ([900, 33], [1, 33], 1, 200, "fp8", 0),
    ([257, 400, 80], [7, 1, 80], 16, 16, "fp8", 128),
    ([500, 90], [40, 3], 24, 64, "fp4", 1),
    ([385, 129], [9, 129], 40, 8, "fp8", 100),
    ([0, 5, 0, 260], [0, 5, 0, 2], 64, 8, "fp4", 0),
    ([2000, 1500, 1800], [1, 2, 1], 8, 64, "fp4", 1000),
    ([3, 2], [9, 2], 64, 8, "fp4", 0),        # more tokens than entries: the first rows see nothing
    ([0, 4], [3, 4], 64, 8, "fp8", 0),        # a request without entries
]


@pytest.mark.parametrize("i", range(len(ATTN)))
def test_attention(abi, i):
    kv, new, H, page, fmt, window = ATTN[i]
    s = attn_inputs(np.random.default_rng(100 + i), kv, new, H, page, fmt)
    a = Attn(abi, s, window)
    a.call()
    check_attn(*a.result(), s, window)
    assert abi.csa2_status_fetch(a.ws)[0] == abi.OK


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("new", [1, 37])
def test_attention_long_and_looser_bounds(abi, fmt, new):
    """Long ragged requests (keys split over blocks), with host bounds above the lengths."""
    s = attn_inputs(np.random.default_rng(9), [3000, 5, 1311], [new, 1, min(new, 3)], 64, 64, fmt)
    a = Attn(abi, s, 0, max_q=new + 5, max_kv=9000)
    a.call()
    check_attn(*a.result(), s, 0)


@pytest.mark.parametrize("q_amp", [2.0 ** -20, 2.0 ** 14, 40.0])
def test_attention_query_ranges(abi, q_amp):
    """Tiny and huge queries keep their precision; at 40 the softmax is one-hot and its maximum moves."""
    s = attn_inputs(np.random.default_rng(3), [450, 130], [4, 1], 64, 16, "fp4", q_amp=q_amp, c_amp=1.0 if q_amp < 1e3 else 2.0 ** -5)
    a = Attn(abi, s)
    a.call()
    check_attn(*a.result(), s, 0)


def test_attention_growing_logits(abi):
    """Keys ordered so that each is seen as a new maximum, by more and more: every step rescales."""
    s = attn_inputs(np.random.default_rng(4), [1024], [1], 64, 8, "fp8")
    base = s["q"][0, 0].float().numpy()
    rows = (s["table"][0, np.arange(1024) // 8].astype(np.int64) * 8 + np.arange(1024) % 8)
    s["codes"][rows] = O.e4m3_encode((np.linspace(-8, 8, 1024)[:, None] * base[None]).astype(np.float64))
    a = Attn(abi, s)
    a.call()
    check_attn(*a.result(), s, 0)


@pytest.mark.parametrize("new,reqs", [(1, 152), (152, 1)])
def test_attention_many_small_probabilities(abi, new, reqs):
    """Half a million keys of probability 2^-25.3 next to one of about 1: each is below f16's range, together they are
    1.3 % of the output.  (As many rows as there are multiprocessors, so that the keys are not split: in a split of
    their own their probabilities are not small.)  The cache holds two pages: all but the first are the same one.

    Such a key enters the products with an error of at most 2^-25 against a largest probability of at least 2^7
    (2^-32 each, n 2^-32 = 2^-13 for all), the sums and the rest as in check_attn."""
    n = 1 << 19
    codes = np.zeros((128, D), np.uint8)
    codes[:64, 2] = 0x38    # page 0: 1.0 in channel 2
    codes[64, [0, 1]] = 0x38  # page 1: 1.0 in channels 0 and 1, at its first entry
    codes[65:, 2] = 0x38
    table = np.zeros((reqs, n // 64), np.int32)
    table[:, 0] = 1
    q = torch.zeros(reqs * new, 64, D, dtype=torch.bfloat16)
    q[:, :, 0] = 25.3 * np.log(2.0) / SM
    q0 = float(q[0, 0, 0])
    s = dict(q=q, q_start=np.arange(reqs + 1, dtype=np.int32) * new, kv_len=np.full(reqs, n, np.int32), codes=codes, scales=None,
             table=table, page=64, fmt="fp8", T=reqs * new, H=64, max_q=new, max_kv=n)
    a = Attn(abi, s)
    a.call()
    out, lse = a.result()
    others = n - new + np.arange(new, dtype=np.float64)  # keys that a token sees besides the first
    p = others * np.exp(-q0 * SM)
    want = np.zeros((reqs, new, 64, D))
    want[..., :2] = (1 / (1 + p))[None, :, None, None]
    want[..., 2] = (p / (1 + p))[None, :, None]
    d = 64 * 2.0 ** -24 * q0 * SM + 2.0 ** -21
    tol = 2 * d + 2.0 ** -11 * want + n * 2.0 ** -32 + (2.0 ** -8 + n * 2.0 ** -24) * want
    assert 0.012 < want[..., 2].min() and (np.abs(out.reshape(want.shape) - want) <= tol).all()
    wlse = np.broadcast_to((q0 * SM + np.log1p(p))[None, :, None], (reqs, new, 64))
    assert (np.abs(lse.reshape(wlse.shape) - wlse) <= d + n * 2.0 ** -24 + 2.0 ** -22 * (1 + wlse)).all()


@pytest.mark.parametrize("more,window", [(0, 100), (700, 600)])  # (the few-row kernel, decoded tiles)
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_attention_leaves_out_what_is_masked(abi, fmt, more, window):
    """NaN and the largest values in rows behind the sequence, outside the window, in later tokens' entries and in
    other pages do not reach rows that do not see them; a token that sees a NaN entry is NaN as a whole."""
    rng = np.random.default_rng(8)
    s = attn_inputs(rng, [201 + more, 77 + more], [6, 2], 64, 16, fmt)
    clean = {**s, "codes": s["codes"].copy(), "scales": None if s["scales"] is None else s["scales"].copy()}
    row = lambda r, p: int(s["table"][r, p // 16]) * 16 + p % 16  # noqa: E731

    def spoil(at):
        if fmt == "fp8":
            s["codes"][at, ::3] = 0x7F
            s["codes"][at, 1::3] = 0xFE
        else:
            s["scales"][at, ::2] = 0x7F
            s["scales"][at, 1::2] = 0x7E
    end = [16 * (-(-n // 16)) for n in s["kv_len"]]
    for p in list(range(201 + more, end[0])) + [199 + more, 200 + more, 3, 64]:
        spoil(row(0, p))
    for p in range(77 + more, end[1]):
        spoil(row(1, p))
    # request 0's tokens sit at 195 .. 200 + more: 3 and 64 are outside, 199 + more is seen by the last two
    a = Attn(abi, s, window)
    a.call()
    out, lse = a.result()
    assert np.isnan(out[4:6]).all() and np.isnan(lse[4:6]).all()
    out[4:6], lse[4:6] = 0, 0
    want = Attn(abi, clean, window)
    want.call()
    wout, wlse = want.result()
    wout[4:6], wlse[4:6] = 0, 0
    assert np.array_equal(out, wout) and np.array_equal(lse, wlse)


def test_attention_pages_and_lengths_outside_are_recorded(abi):
    s = attn_inputs(np.random.default_rng(11), [100, 60, 40, 50], [2, 2, 2, 2], 64, 8, "fp4")
    n_pages = len(s["codes"]) // 8
    s["table"][0, 3] = n_pages
    s["table"][0, 5] = -2
    bad = lambda i: i < 0 or i >= n_pages  # noqa: E731
    a = Attn(abi, s)
    a.call()
    check_attn(*a.result(), s, 0, bad_page=bad)
    st = abi.csa2_status_fetch(a.ws)
    assert st[0] == abi.ERR_DEVICE_BOUNDS and st[1] == 8 and st[2] == 0
    # a length above the bound, below zero: that request sees nothing
    for wrong in (101, -1):
        s2 = dict(s, kv_len=np.array([100, wrong, 40, 50], np.int32))
        s2["table"] = np.where(bad_ids(s2["table"], n_pages), 0, s2["table"]).astype(np.int32)
        b = Attn(abi, s2, max_kv=100)
        b.call()
        out, lse = b.result()
        assert (out[2:4] == 0).all() and np.isneginf(lse[2:4]).all()
        ref = dict(s2, kv_len=np.array([100, 0, 40, 50], np.int32))
        check_attn(out, lse, ref, 0)
        st = abi.csa2_status_fetch(b.ws)
        assert st[:3] == [abi.ERR_DEVICE_BOUNDS, 9, 1]
    # tokens above the bound: that request's rows are left as they are
    s3 = dict(s2, kv_len=np.array([100, 60, 40, 50], np.int32), q_start=np.array([0, 2, 7, 8, 8], np.int32))
    c = Attn(abi, s3, max_q=2)
    c.call()
    out, lse = c.result()
    assert (out[2:7] == 7).all() and (lse[2:7] == 7).all()
    assert abi.csa2_status_fetch(c.ws)[:3] == [abi.ERR_DEVICE_BOUNDS, 9, 1]


def test_attention_over_tiles_records_pages_and_lengths(abi):
    """The same for requests whose keys are decoded to tiles."""
    s = attn_inputs(np.random.default_rng(11), [100, 60, 40, 50], [6, 7, 5, 9], 64, 8, "fp4")
    n_pages = len(s["codes"]) // 8
    good = s["table"].copy()
    s["table"][0, 3] = n_pages
    s["table"][0, 5] = -2
    a = Attn(abi, s, max_kv=1000)
    a.call()
    check_attn(*a.result(), s, 0, bad_page=lambda i: i < 0 or i >= n_pages)
    st = abi.csa2_status_fetch(a.ws)
    assert st[0] == abi.ERR_DEVICE_BOUNDS and st[1] == 8 and st[2] == 0
    for wrong in (105, -1):  # the table's rows hold 104 entries
        b = Attn(abi, dict(s, table=good, kv_len=np.array([100, wrong, 40, 50], np.int32)), max_kv=1000)
        b.call()
        out, lse = b.result()
        assert (out[6:13] == 0).all() and np.isneginf(lse[6:13]).all()
        check_attn(out, lse, dict(s, table=good, kv_len=np.array([100, 0, 40, 50], np.int32)), 0)
        assert abi.csa2_status_fetch(b.ws)[:3] == [abi.ERR_DEVICE_BOUNDS, 9, 1]
    c = Attn(abi, dict(s, table=good, q_start=np.array([0, 6, 18, 18, 27], np.int32)), max_q=9, max_kv=1000)
    c.call()
    out, lse = c.result()
    assert (out[6:18] == 7).all() and (lse[6:18] == 7).all() and (out[:6] != 7).any()
    assert abi.csa2_status_fetch(c.ws)[:3] == [abi.ERR_DEVICE_BOUNDS, 9, 1]


@pytest.mark.parametrize("i", range(len(ATTN)))
def test_attention_with_a_loose_bound(abi, i):
    """The cases of test_attention with a bound that takes chunks to the decoded tiles (without a window)."""
    kv_len, new, heads, page, fmt, window = ATTN[i]
    s = attn_inputs(np.random.default_rng(200 + i), kv_len, new, heads, page, fmt)
    a = Attn(abi, s, window, max_kv=max(kv_len) + 600)
    a.call()
    check_attn(*a.result(), s, window)
    assert abi.csa2_status_fetch(a.ws)[0] == abi.OK


def test_attention_of_both_kinds_on_two_streams(abi):
    """Calls that run both kernels, on two streams at once with workspaces of their own, give the same bits as alone."""
    calls = []
    for k in range(2):
        s = attn_inputs(np.random.default_rng(50 + k), [2600, 2300, 900, 2100], [40 + k, 1, 2, 1], 64, 16, ("fp4", "fp8")[k])
        a = Attn(abi, s)
        a.call()
        calls.append((a, a.result()))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for (a, _), st in zip(calls, streams):
            a.call(st)
    torch.cuda.synchronize()
    for a, (out, lse) in calls:
        got = a.result()
        assert np.array_equal(got[0], out) and np.array_equal(got[1], lse) and abi.csa2_status_fetch(a.ws)[0] == abi.OK


def bad_ids(t, n):
    return (t < 0) | (t >= n)


@pytest.mark.parametrize("bound", [300, 1000])
def test_attention_rows_behind_the_last_token_stay(abi, bound):
    s = attn_inputs(np.random.default_rng(12), [90, 300], [3, 70], 16, 8, "fp4", tail=19)
    a = Attn(abi, s, max_kv=bound)
    a.call()
    out, lse = a.result()
    check_attn(out, lse, s, 0)
    assert (out[73:] == 7).all() and (lse[73:] == 7).all()


def test_attention_without_lse_and_twice(abi):
    s = attn_inputs(np.random.default_rng(13), [1300, 40], [2, 40], 64, 64, "fp4")
    a = Attn(abi, s)
    a.call()
    one, _ = a.result()
    a.out.fill_(1.0)
    a.lse.fill_(3.0)
    a.call(lse=False)
    two, lse = a.result()
    assert np.array_equal(one, two) and (lse == 3).all()


def test_attention_graphs_streams_and_one_workspace(abi):
    """Two captured graphs that share a workspace, replayed in order on a stream of their own with lengths and
    inputs that change between replays, give what eager calls give."""
    s1 = attn_inputs(np.random.default_rng(14), [2100, 700], [1, 1], 64, 64, "fp4")
    s2 = attn_inputs(np.random.default_rng(15), [640, 1900], [5, 3], 64, 16, "fp8")
    a, b = Attn(abi, s1), Attn(abi, s2, 128)
    size = max(a.ws.numel(), b.ws.numel())
    a.ws = b.ws = fresh_ws(abi, size)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graphs = []
    for x in (a, b):
        x.call(st)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            x.call(torch.cuda.current_stream())
        graphs.append(g)
    for k in range(3):
        a.kv_len.copy_(torch.tensor([2100 - 500 * k, 700], dtype=torch.int32))
        b.q.mul_(-1)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for g in graphs:
                g.replay()
        st.synchronize()
        check_attn(*a.result(), dict(s1, kv_len=np.array([2100 - 500 * k, 700], np.int32)), 0)
        check_attn(*b.result(), dict(s2, q=b.q.cpu()), 128)
    assert abi.csa2_status_fetch(a.ws)[0] == abi.OK


def test_attention_is_the_sparse_attention_of_all_entries(abi):
    """Over at most 512 contiguous entries the paged call equals csa2_sparse_attn with every entry selected."""
    n = 500
    s = attn_inputs(np.random.default_rng(16), [n], [1], 64, 8, "fp4")
    order = np.arange(-(-n // 8), dtype=np.int32)
    s["table"][0, :len(order)] = order
    a = Attn(abi, s)
    a.call()
    out, lse = a.result()
    topk = torch.full((1, 512), -1, dtype=torch.int32, device="cuda")
    topk[0, :n] = torch.arange(n, dtype=torch.int32)
    ws = fresh_ws(abi, abi.csa2_workspace_bytes(abi.OP_SPARSE_ATTN, 1, n, 1, 512))
    o = torch.empty(1, 64, D, dtype=torch.float32, device="cuda")
    ls = torch.empty(1, 64, device="cuda")
    abi.csa2_sparse_attn(a.q, 1, a.codes, a.scales, a.codes.shape[0], torch.zeros(1, dtype=torch.int64, device="cuda"),
                         torch.tensor([n], dtype=torch.int32, device="cuda"), topk, 512, None, None, 0, SM, o, abi.OUT_F32,
                         ls, ws, ws.numel())
    torch.cuda.synchronize()
    check_attn(o.cpu().numpy().astype(np.float64), ls.cpu().numpy().astype(np.float64), s, 0)
    check_attn(out, lse, s, 0)


# -------------------------------------------------------------------- norm
def norm_call(abi, x, res, w, group, y=True, in_place=False, stride=None, stream=None):
    n, dim = x.shape
    stride = stride or dim
    xd = torch.full((n, stride), 3.0, dtype=torch.bfloat16, device="cuda")
    xd[:, :dim] = x.cuda()
    rd = None if res is None else res.cuda()
    ro = None if res is None else (rd if in_place else torch.zeros_like(rd))
    codes = torch.zeros(n, dim, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(n, dim // 128 if group else 1, device="cuda")
    yo = torch.zeros(n, dim, dtype=torch.bfloat16, device="cuda") if y else None
    abi.csa2_rmsnorm_fp8(xd, stride, rd, ro, w.cuda(), n, dim, 1e-6, group, codes, scales, yo, stream)
    torch.cuda.synchronize()
    return (None if ro is None else ro.cpu()), codes.view(torch.float8_e4m3fn).float().cpu().numpy(), scales.cpu().numpy(), \
        None if yo is None else yo.float().cpu().numpy()


def check_norm(h, w, group, codes, scales, y):
    """y is off by a few fp32 roundings, e = (dim/2 + 8) 2^-24 relative at most for a serial sum's share; the sum
    here is over a tree of at most 64-long chains: e = 48 * 2^-24.  The scale by e + 2^-24, a code's value by half
    a step (2^-4 relative, 2^-10 absolute below E4M3's normal range) plus e of y/s."""
    want = PO.rmsnorm(h, w, 1e-6)
    n, dim = want.shape
    e = 48 * 2.0 ** -24
    g = want.reshape(n, -1, 128 if group else dim)
    s = np.abs(g).max(axis=2) / 448.0
    assert (np.abs(scales - s) <= (e + 2.0 ** -24) * s + 2.0 ** -150).all()
    r = np.divide(g, s[..., None], out=np.zeros_like(g), where=s[..., None] > 0).reshape(n, dim)
    assert (np.abs(codes - r) <= np.maximum(2.0 ** -4 * np.abs(r), 2.0 ** -10) + 4 * e * np.abs(r)).all()
    if y is not None:
        assert (np.abs(y - want) <= (2.0 ** -8 + e) * np.abs(want)).all()


@pytest.mark.parametrize("n,dim,group,res", [(1, 8, 0, True), (3, 128, 128, True), (9, 512, 0, False), (17, 520, 0, True),
                                             (5, 1024, 128, False), (4, 1032, 0, True), (2, 5120, 0, True),
                                             (3, 7168, 128, True), (1, 16384, 0, True), (1300, 640, 128, True),
                                             (2500, 16, 0, False), (1, 16256, 128, False)])
def test_norm(abi, n, dim, group, res):
    rng = np.random.default_rng(dim + n)
    amp = np.exp(rng.standard_normal((n, 1)))
    x, w = bf16(amp * rng.standard_normal((n, dim))), bf16(1 + 0.2 * rng.standard_normal(dim))
    r = bf16(amp * rng.standard_normal((n, dim))) if res else None
    ro, codes, scales, y = norm_call(abi, x, r, w, group)
    h = x if r is None else (x.float() + r.float()).to(torch.bfloat16)
    if res:
        assert torch.equal(ro, h)
    check_norm(h.double().numpy(), w.double().numpy(), group, codes, scales, y)


def test_norm_in_place_strided_and_without_bf16(abi):
    rng = np.random.default_rng(2)
    x, w, r = bf16(rng.standard_normal((6, 512))), bf16(rng.standard_normal(512)), bf16(rng.standard_normal((6, 512)))
    a = norm_call(abi, x, r, w, 0, stride=600, in_place=True, y=False)
    b = norm_call(abi, x, r, w, 0)
    assert torch.equal(a[0], b[0]) and np.array_equal(a[1], b[1]) and np.array_equal(a[2], b[2])


@pytest.mark.parametrize("group", [0, 128])
def test_norm_extremes(abi, group):
    """Zero rows, one huge element, tiny rows (subnormal scales), zero weights."""
    x = np.zeros((5, 256), np.float32)
    x[1, 7] = 2.0 ** 50
    x[2] = 2.0 ** -120
    x[3, :128] = 1.0
    x[4] = np.linspace(-3, 3, 256)
    w = np.ones(256, np.float32)
    _, codes, scales, y = norm_call(abi, bf16(x), None, bf16(w), group)
    check_norm(bf16(x).double().numpy(), w.astype(np.float64), group, codes, scales, y)
    assert (codes[0] == 0).all() and (scales[0] == 0).all()
    w[:] = 2.0 ** -126
    _, codes, scales, _ = norm_call(abi, bf16(x), None, bf16(w), group, y=False)
    assert np.isfinite(codes).all() and np.isfinite(scales).all()
    assert np.abs(codes[1]).max() >= 256  # a subnormal scale keeps the largest code near 448


def test_norm_nan_and_infinity(abi):
    x = np.ones((3, 256), np.float32)
    x[0, 5] = np.nan
    x[1, 200] = np.inf
    _, codes, scales, _ = norm_call(abi, bf16(x), None, bf16(np.ones(256)), 128)
    assert np.isnan(scales[0]).all() and np.isnan(codes[0]).all()
    assert np.isnan(scales[1, 1]) and np.isnan(codes[1, 128:]).all()
    assert scales[1, 0] == 0 and (codes[1, :128] == 0).all()
    assert np.isfinite(scales[2]).all() and np.isfinite(codes[2]).all()


# ------------------------------------------------------------------ matvec
def weight(rng, n_out, k, amp=1.0):
    c, s = [], []
    for i in range(0, n_out * k, D * 4096):
        m = min(4096, (n_out * k - i + D - 1) // D)
        a, b = cache_rows(rng, m, "fp4", amp)
        c.append(a.reshape(-1))
        s.append(b.reshape(-1))
    return np.concatenate(c)[:n_out * k // 2].reshape(n_out, k // 2), np.concatenate(s)[:n_out * k // 16].reshape(n_out, k // 16)


def matvec_call(abi, x, xs, codes, scales, alpha, out_dtype, stride=None):
    n, k = x.shape
    stride = stride or k
    xd = torch.zeros(max(n, 1), stride, dtype=x.dtype).view(torch.uint8 if x.dtype == torch.float8_e4m3fn else x.dtype)
    xd[:n, :k] = x.view(xd.dtype)
    xd = xd.cuda()
    out = torch.full((max(n, 1), len(codes)), 9.0, dtype=out_dtype, device="cuda")
    ws = fresh_ws(abi, abi.csa2_fp4_matvec_workspace_bytes(n, k, len(codes)))
    abi.csa2_fp4_matvec(xd, abi.X_BF16 if xs is None else abi.X_E4M3, None if xs is None else dev(xs), stride, n, k, dev(codes),
                        dev(scales), len(codes), alpha, out, abi.OUT_BF16 if out_dtype == torch.bfloat16 else abi.OUT_F32, ws,
                        ws.numel())
    torch.cuda.synchronize()
    return out[:n].double().cpu().numpy()


def check_matvec(got, x, xs, codes, scales, alpha, out_dtype):
    """Products are exact; k terms are added in fp32 in chains of at most 512 and trees (bounded at 64 * 2^-24 of the
    absolute sum), scaled by alpha and the row's scale in fp32, rounded once."""
    want, reach = PO.matvec(x.double().numpy(), xs, codes, scales, alpha)
    tol = 64 * 2.0 ** -24 * reach + (2.0 ** -8 if out_dtype == torch.bfloat16 else 0) * np.abs(want)
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / np.maximum(tol, 1e-30)).max()


@pytest.mark.parametrize("n,k,n_out", [(1, 128, 1), (1, 5120, 512), (2, 256, 63), (3, 1536, 130), (8, 384, 1000), (9, 640, 65),
                                       (16, 1536, 2048), (17, 128, 33), (40, 2048, 100), (1, 65536, 3), (5, 12288, 257),
                                       (1, 8192, 4099)])
@pytest.mark.parametrize("fp8", [False, True])
def test_matvec(abi, n, k, n_out, fp8):
    rng = np.random.default_rng(n * k + n_out)
    codes, scales = weight(rng, n_out, k)
    x = np.exp(rng.standard_normal((n, 1))) * rng.standard_normal((n, k))
    if fp8:
        xs = (np.abs(x).max(axis=1) / 448).astype(np.float32)
        xt = torch.from_numpy(x / xs[:, None]).float().to(torch.float8_e4m3fn)
    else:
        xs, xt = None, bf16(x)
    for dt in (torch.bfloat16, torch.float32):
        got = matvec_call(abi, xt, xs, codes, scales, 0.37, dt, stride=k + 16 if n_out % 2 else None)
        check_matvec(got, xt, xs, codes, scales, 0.37, dt)


@pytest.mark.parametrize("n,k,n_out", [(1, 4096, 6000), (5, 896, 20000), (16, 768, 32768), (3, 1408, 9333), (12, 640, 14592)])
def test_matvec_splits_of_the_warps(abi, n, k, n_out):
    """Sizes whose warps are no powers of two each way, or not all in use."""
    rng = np.random.default_rng(n + k)
    codes, scales = weight(rng, n_out, k)
    x = bf16(rng.standard_normal((n, k)))
    got = matvec_call(abi, x, None, codes, scales, 1.0, torch.float32)
    check_matvec(got, x, None, codes, scales, 1.0, torch.float32)


def test_matvec_ranges(abi):
    """Rows of very different size side by side, a zero row, the largest and smallest weights."""
    rng = np.random.default_rng(1)
    codes, scales = weight(rng, 96, 512)
    scales[:32] = 0x7E   # 448
    scales[32:64] = 0x01  # 2^-9
    codes[10] = 0x77
    x = bf16(rng.standard_normal((4, 512)) * np.array([2.0 ** 90, 2.0 ** -90, 1.0, 0.0])[:, None])
    got = matvec_call(abi, x, None, codes, scales, 1.0, torch.float32)
    check_matvec(got, x, None, codes, scales, 1.0, torch.float32)
    assert (got[3] == 0).all()


def test_matvec_nan_stays_in_its_row(abi):
    rng = np.random.default_rng(1)
    codes, scales = weight(rng, 64, 256)
    x = bf16(rng.standard_normal((5, 256)))
    clean = matvec_call(abi, x, None, codes, scales, 1.0, torch.float32)
    x[1, 3], x[3, 200] = float("nan"), float("inf")
    scales = scales.copy()
    scales[7, 2] = 0x7F
    got = matvec_call(abi, x, None, codes, scales, 1.0, torch.float32)
    assert np.isnan(got[1]).all() and np.isnan(got[:, 7]).all() and not np.isfinite(got[3]).any()
    keep = np.ones(64, bool)
    keep[7] = False
    assert np.array_equal(got[[0, 2, 4]][:, keep], clean[[0, 2, 4]][:, keep])


def test_matvec_weights_beyond_two_gigabytes(abi):
    """Row offsets past 2^31 bytes: only the last rows are not zero."""
    k, n_out = 65536, 66000
    codes = torch.zeros(n_out, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((n_out, k // 16), 0x38, dtype=torch.uint8, device="cuda")
    codes[-3:] = 0x22  # ones
    x = torch.ones(2, k, dtype=torch.bfloat16, device="cuda")
    out = torch.full((2, n_out), 9.0, device="cuda")
    ws = fresh_ws(abi, abi.csa2_fp4_matvec_workspace_bytes(2, k, n_out))
    abi.csa2_fp4_matvec(x, abi.X_BF16, None, k, 2, k, codes, scales, n_out, 1.0, out, abi.OUT_F32, ws, ws.numel(), None)
    torch.cuda.synchronize()
    assert (out[:, :-3] == 0).all() and (out[:, -3:] == k).all()


# ------------------------------------------------- the attention once more
@pytest.mark.parametrize("new,fmt", [(2, "fp4"), (2, "fp8"), (40, "fp4"), (40, "fp8")])
def test_attention_cache_beyond_two_gigabytes(abi, new, fmt):
    """Rows past 2^31 bytes of the latent planes, in the few-row kernel and over decoded tiles."""
    s = attn_inputs(np.random.default_rng(21), [300], [new], 16, 64, fmt)
    shift = (1 << 31) // (256 if fmt == "fp4" else 512) // 64 + 17  # pages
    n_rows = len(s["codes"]) + 64 * shift
    a = Attn(abi, s, max_kv=1000)
    codes = torch.empty((n_rows, s["codes"].shape[1]), dtype=torch.uint8, device="cuda")
    codes[64 * shift:] = a.codes
    a.codes = codes
    if fmt == "fp4":
        scales = torch.empty((n_rows, 32), dtype=torch.uint8, device="cuda")
        scales[64 * shift:] = a.scales
        a.scales = scales
    a.table = a.table + shift
    a.call()
    check_attn(*a.result(), s, 0)
    assert abi.csa2_status_fetch(a.ws)[0] == abi.OK


@pytest.mark.parametrize("kv,new,bound", [([500, 300], [2, 1], 500), ([500, 300], [40, 1], 500), ([500, 300], [40, 1], 1000),
                                          ([2600, 2300, 900], [40, 1, 1], 2600)])  # few rows, few tiles, tiles, both kernels
def test_attention_gives_up_and_recovers(abi, kv, new, bound):
    """With a wait limit of 1 ns every bounded wait gives up: the status says so, copies and MMAs in flight are
    waited for, and the next call is right."""
    s = attn_inputs(np.random.default_rng(22), kv, new, 16, 16, "fp4")
    a = Attn(abi, s, max_kv=bound)
    a.call()
    one = a.result()
    check_attn(*one, s, 0)
    abi.csa2_debug_wait_limit(1)
    try:
        a.call()
        torch.cuda.synchronize()
    finally:
        abi.csa2_debug_wait_limit(0)
    assert abi.csa2_status_fetch(a.ws)[0] == abi.ERR_TIMEOUT
    abi.csa2_status_reset(a.ws)
    a.out.fill_(3.0)
    a.call()
    two = a.result()
    assert np.array_equal(one[0], two[0]) and np.array_equal(one[1], two[1])
    assert abi.csa2_status_fetch(a.ws)[0] == abi.OK


def test_attention_of_many_requests(abi):
    """More requests than a warp's scan step, some without tokens, some without entries."""
    rng = np.random.default_rng(23)
    R = 150
    new = rng.integers(0, 3, R)
    kv = np.where(new > 0, rng.integers(0, 200, R), rng.integers(0, 50, R))
    s = attn_inputs(rng, kv, new, 3, 8, "fp4")
    a = Attn(abi, s)
    a.call()
    check_attn(*a.result(), s, 0)


@pytest.mark.parametrize("reqs,new,heads,longest", [(1, 1, 64, 8192), (5, 3, 64, 5000), (33, 1, 64, 3000), (60, 1, 128, 1500),
                                                    (200, 1, 5, 2000), (3, 40, 64, 2100), (40, 6, 16, 1100), (257, 1, 64, 700)])
def test_attention_splits_by_the_requests_lengths(abi, reqs, new, heads, longest):
    """Lengths from one entry to the longest, so that the splits are far from those planned for the longest alone; the
    same calls with host bounds far above the lengths, and with a second set of lengths in the same workspace."""
    rng = np.random.default_rng(31)
    lens = lambda: np.maximum(rng.integers(0, 1 + longest * np.arange(1, reqs + 1) // reqs), 1)  # noqa: E731
    kv_len = lens()
    kv_len[-1] = longest
    s = attn_inputs(rng, kv_len, np.minimum(new, kv_len), heads, 16, "fp4")
    a = Attn(abi, s)
    a.call()
    check_attn(*a.result(), s, 0)
    b = Attn(abi, s, max_kv=4 * longest)
    b.call()
    check_attn(*b.result(), s, 0)
    assert abi.csa2_status_fetch(a.ws)[0] == 0 and abi.csa2_status_fetch(b.ws)[0] == 0
    short = np.minimum(s["kv_len"], np.maximum(lens(), np.diff(s["q_start"]))).astype(np.int32)
    s2 = {**s, "kv_len": short}
    c = Attn(abi, s2, max_kv=longest, ws=a.ws)
    c.call()
    check_attn(*c.result(), s2, 0)


@pytest.mark.parametrize("kv_len,new,heads,window,fmt", [
    ([900, 2300, 2200, 40, 1, 0, 2100, 2049], [1, 300, 1, 4, 1, 0, 2, 1], 64, 0, "fp4"),   # both kernels, the short ones' keys split
    ([2600, 2300, 2048, 2500, 700], [40, 1, 1, 1, 2], 100, 0, "fp8"),                     # both, keys of both split
    ([600, 90, 31, 600, 80, 300, 300, 300], [90, 1, 1, 3, 2, 1, 1, 1], 32, 100, "fp4"),   # both, short window
    ([300, 90, 31, 600], [90, 90, 1, 3], 32, 0, "fp8")])                                  # tiles alone
def test_attention_long_and_short_requests_together(abi, kv_len, new, heads, window, fmt):
    """Short requests beside long ones may take a kernel of their own; tokens behind the last request stay as they are,
    a request with bad bounds is recorded and skipped, and a replayed graph gives the same bits."""
    s = attn_inputs(np.random.default_rng(21), kv_len, new, heads, 16, fmt, tail=3)
    a = Attn(abi, s, window)
    a.call()
    out, lse = a.result()
    check_attn(out, lse, s, window)
    T = int(s["q_start"][-1])
    assert (out[T:] == 7).all() and (lse[T:] == 7).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.call(torch.cuda.current_stream())
    a.out.fill_(5), a.lse.fill_(5)
    g.replay(), g.replay()
    out2, lse2 = a.result()
    assert np.array_equal(out2[:T], out[:T]) and np.array_equal(lse2[:T], lse[:T]) and (out2[T:] == 5).all()
    assert abi.csa2_status_fetch(a.ws)[0] == 0
    a.kv_len[0] = 1 << 20  # outside the table row: sees nothing
    a.call()
    out3, lse3 = a.result()
    n = int(s["q_start"][1])
    assert (out3[:n] == 0).all() and np.isneginf(lse3[:n]).all() and np.array_equal(out3[n:T], out[n:T])
    assert abi.csa2_status_fetch(a.ws)[0] == abi.ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("kv,new,window", [(512, 30, 0), (513, 30, 0), (900, 40, 250), (900, 40, 400), (2000, 300, 128)])
def test_attention_on_both_sides_of_few_tiles(abi, kv, new, window):
    """Long chunks that see four key tiles or fewer go to the few-row kernel, others to the decoded tiles."""
    s = attn_inputs(np.random.default_rng(kv + new), [kv, kv // 2, 7], [new, min(new, kv // 2), 7], 32, 16, "fp8")
    a = Attn(abi, s, window)
    a.call()
    check_attn(*a.result(), s, window)


@pytest.mark.parametrize("new,kv,window,fmt,loose", [(152, 1700, 0, "fp4", 0), (156, 1700, 0, "fp8", 0), (161, 2100, 1600, "fp4", 0),
                                                     (199, 1650, 0, "fp4", 0), (227, 1600, 0, "fp4", 0), (30, 1600, 0, "fp4", 169),
                                                     (153, 155, 0, "fp4", 1700), (100, 2000, 0, "fp8", 100)])
def test_attention_of_one_long_chunk(abi, new, kv, window, fmt, loose):
    """One request of whole waves of rows and some more, whose last rows' keys may be split: 38 items of 256 rows and 0,
    1, 3, 12 (and a broken one) and 19 more, fewer than a wave under looser bounds, and too few keys to split."""
    s = attn_inputs(np.random.default_rng(new), [kv], [new], 64, 16, fmt, tail=loose if loose < 1000 else 0)
    a = Attn(abi, s, window, max_q=new + (loose if loose < 1000 else 0), max_kv=max(kv, loose))
    for _ in range(2):
        a.out.fill_(7), a.lse.fill_(7)
        a.call()
        out, lse = a.result()
        check_attn(out, lse, s, window)
        assert (out[new:] == 7).all() and (lse[new:] == 7).all() and abi.csa2_status_fetch(a.ws)[0] == abi.OK


@pytest.mark.parametrize("heads,new", [(64, 4), (64, 5), (128, 2), (1, 256), (1, 257), (100, 3)])
def test_attention_on_both_sides_of_the_kernels_border(abi, heads, new):
    """256 rows of a request go to the few-row kernel, more to the decoded tiles."""
    s = attn_inputs(np.random.default_rng(heads + new), [new + 150, 140], [new, 1], heads, 16, "fp4")
    a = Attn(abi, s)
    a.call()
    check_attn(*a.result(), s, 0)


# ------------------------------------------------------------ a whole step
def layer_case(abi, fmt, window, seed=31):
    from csa2_sparse_attention_gb300 import paged
    g = torch.Generator().manual_seed(seed)
    R, hidden, heads, page = 3, 256, 4, 16
    cache = paged.PagedLatents(R, 64, 40, page, 12, heads=heads, fmt=fmt, window=window)
    w = lambda *sh: torch.randn(*sh, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    layer = paged.PagedLayer(cache, hidden, (1 + 0.1 * torch.randn(hidden, generator=g)).to(torch.bfloat16).cuda(),
                             w(heads * D, hidden), w(D, hidden))
    return paged, g, cache, layer


@pytest.mark.parametrize("fmt,window", [("fp4", 0), ("fp8", 20)])
def test_step_over_a_paged_cache(abi, fmt, window):
    """Prompt chunks, then decoding steps beside another chunk: every stage of the step against its 64-bit form on
    what the stage before it left, and the plan against the whole history."""
    paged, g, cache, layer = layer_case(abi, abi.FMT_FP4 if fmt == "fp4" else abi.FMT_FP8, window)
    hidden, heads, page = layer.hidden, cache.heads, cache.page_size
    table, n_free = cache.table.cpu().numpy(), cache.n_pages
    free = cache.free.cpu().numpy()
    cached = np.zeros(3, np.int32)
    for added in ([30, 0, 17], [1, 25, 1], [1, 1, 1], [0, 1, 31]):
        added = np.array(added, np.int32)
        n = int(added.sum())
        cache.added.copy_(torch.from_numpy(added))
        layer.residual[:n] = torch.randn(n, hidden, generator=g).to(torch.bfloat16)
        res = layer.residual[:n].cpu()
        x = torch.randn(n, hidden, generator=g).to(torch.bfloat16)
        out, lse = layer.step(x.cuda(), n, int(added.max()), int((cached + added).max()))
        torch.cuda.synchronize()
        for name, st in cache.status().items():
            assert st[0] == abi.OK, (name, st)
        # norm
        h = (x.float() + res.float()).to(torch.bfloat16)
        assert torch.equal(layer.residual[:n].cpu(), h)
        codes = layer.x[:n].view(torch.float8_e4m3fn).cpu()
        xs = layer.x_scales[:n].cpu().numpy()
        check_norm(h.double().numpy(), layer.norm_weight.double().cpu().numpy(), 0, codes.float().numpy(), xs[:, None], None)
        # projections
        for wt, got in ((layer.wq, layer.q[:n].flatten(1)), (layer.wlatent, layer.latents[:n])):
            check_matvec(got.double().cpu().numpy(), codes, xs, wt[0].cpu().numpy(), wt[1].cpu().numpy(), 1.0, torch.bfloat16)
        # plan
        want = PO.page_plan(cached, added, page, table, free, n_free, cache.n_pages, cache.max_tokens)
        table, n_free = want[0], want[5]
        check_plan((cache.table.cpu().numpy(), cache.q_start.cpu().numpy(), cache.kv_len.cpu().numpy(), cache.slots.cpu().numpy(),
                    cache.pos.cpu().numpy(), int(cache.n_free.item())), want)
        # append
        slots, pos = want[3][:n], want[4][:n]
        lat = layer.latents[:n].double().cpu().numpy()
        cc = cache.codes.cpu().numpy()
        cs = None if cache.scales is None else cache.scales.cpu().numpy()
        if fmt == "fp4":
            oc, os_ = O.append_main_latent(lat, pos)
            assert np.mean(cc[slots] != oc) < 1e-3 and np.mean(cs[slots] != os_) < 1e-3  # ties next to a border
        else:
            assert np.array_equal(cc[slots], O.append_swa_fp8(lat))
        # attention
        s = dict(q=layer.q[:n].cpu(), q_start=want[1], kv_len=want[2], codes=cc, scales=cs, table=table, page=page, fmt=fmt, T=n,
                 H=heads, max_q=int(added.max()), max_kv=int(want[2].max()))
        check_attn(out.double().cpu().numpy(), lse.double().cpu().numpy(), s, window)
        cache.advance()
        cached = want[2].copy()


def test_step_captured_and_replayed_is_the_eager_step(abi):
    """A decoding step in a CUDA graph, replayed over growing lengths (the plan takes pages inside the graph), equals
    eager steps of another cache byte for byte."""
    runs = []
    for captured in (False, True):
        paged, g, cache, layer = layer_case(abi, abi.FMT_FP4, 0)
        chunk = torch.tensor([30, 9, 17], dtype=torch.int32)
        cache.added.copy_(chunk)
        x = torch.randn(56, layer.hidden, generator=g).to(torch.bfloat16).cuda()
        layer.step(x, 56, 30, 30)
        cache.advance()
        cache.added.fill_(1)
        tok = torch.zeros(3, layer.hidden, dtype=torch.bfloat16, device="cuda")
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        cache.workspace(3, 1, 64)
        graph = torch.cuda.CUDAGraph()
        if captured:
            with torch.cuda.graph(graph, stream=st):
                layer.step(tok, 3, 1, 64, torch.cuda.current_stream())
                cache.advance()
        got = []
        for _ in range(5):
            tok.copy_(torch.randn(3, layer.hidden, generator=g))
            layer.residual.zero_()
            torch.cuda.synchronize()
            if captured:
                with torch.cuda.stream(st):
                    graph.replay()
            else:
                layer.step(tok, 3, 1, 64)
                cache.advance()
            torch.cuda.synchronize()
            got += [cache.out[:3].clone(), cache.lse[:3].clone(), cache.table.clone(), cache.kv_len.clone(), cache.codes.clone()]
        for name, s in cache.status().items():
            assert s[0] == abi.OK, (name, s)
        runs.append(got)
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_captured_step_keeps_its_workspace(abi):
    """A larger eager step between replays takes a workspace of its own; a step that would need a larger one inside a
    capture is refused."""
    paged, g, cache, layer = layer_case(abi, abi.FMT_FP4, 0)
    cache.added.copy_(torch.tensor([30, 9, 17], dtype=torch.int32))
    x = torch.randn(56, layer.hidden, generator=g).to(torch.bfloat16).cuda()
    layer.step(x, 56, 30, 30)
    cache.advance()
    q = layer.q[:3].clone()
    cache.added.fill_(0)
    cache.plan()
    cache.q_start.copy_(torch.tensor([0, 1, 2, 3], dtype=torch.int32))  # (a query over what is there)
    cache.workspace(3, 1, 32)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attend(q, 3, 1, 32)
    held = cache.ws_attn
    graph.replay()
    torch.cuda.synchronize()
    want = cache.out[:3].clone()
    need = abi.csa2_paged_attn_workspace_bytes(3, cache.heads, 3, 3, 1 << 16, 0)
    assert need > held.numel()
    with pytest.raises(RuntimeError):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            cache.attend(q, 3, 3, 1 << 16)
    cache.attend(q, 3, 3, 1 << 16)
    assert cache.ws_attn is not held and any(w is held for w in cache._kept)
    cache.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache.out[:3], want) and cache.status()["attn"][0] == abi.OK


def test_padded_step(abi):
    """More tokens than the lengths give: the rows behind change nothing but the append's status."""
    runs = []
    for pad in (0, 5):
        paged, g, cache, layer = layer_case(abi, abi.FMT_FP4, 0)
        cache.added.copy_(torch.tensor([20, 0, 7], dtype=torch.int32))
        x = torch.randn(32, layer.hidden, generator=g).to(torch.bfloat16).cuda()
        cache.out.fill_(3), cache.lse.fill_(3)
        layer.step(x, 27 + pad, 20, 20)
        torch.cuda.synchronize()
        assert (cache.out[27:] == 3).all() and (cache.lse[27:] == 3).all()
        st = cache.status()
        assert st["plan"][0] == st["attn"][0] == abi.OK
        assert st["append"][0] == (abi.ERR_DEVICE_BOUNDS if pad else abi.OK)
        runs.append((cache.out[:27].clone(), cache.codes.clone(), cache.scales.clone(), cache.table.clone()))
    for a, b in zip(*runs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bound", [200, 1000])
@pytest.mark.parametrize("new", [[10, 6, 1, 1], [130, 9, 1, 3]])
def test_attention_of_more_tokens_than_entries(abi, new, bound):
    """Lengths below the new tokens': the tokens before position 0 see nothing."""
    s = attn_inputs(np.random.default_rng(17), [3, 0, 1, 200], new, 64, 16, "fp4")
    a = Attn(abi, s, max_kv=bound)
    a.call()
    check_attn(*a.result(), s, 0)
    assert abi.csa2_status_fetch(a.ws)[0] == 0


@pytest.mark.parametrize("new,bound", [(2, 300), (9, 300), (9, 1000)])
def test_attention_nan_and_infinite_queries_stay_in_their_rows(abi, new, bound):
    s = attn_inputs(np.random.default_rng(19), [300, 150], [new, new], 64, 16, "fp4")
    a = Attn(abi, s, max_kv=bound)
    a.call()
    want, wlse = a.result()
    a.q[0, 5, 17] = float("nan")
    a.q[new - 1, 63, 300] = float("inf")
    a.q[new, 0, 0] = -float("inf")
    a.call()
    out, lse = a.result()
    for t, h in ((0, 5), (new - 1, 63), (new, 0)):
        assert np.isnan(out[t, h]).all() and np.isnan(lse[t, h])
        out[t, h], lse[t, h] = want[t, h], wlse[t, h]
    assert np.array_equal(out, want) and np.array_equal(lse, wlse)


def test_plan_over_several_blocks_shares_its_ticket(abi):
    """Many tokens (several blocks), the free count in place, call after call on one workspace."""
    rng = np.random.default_rng(41)
    cached, added, table, free, n_free, n_pages = plan_inputs(rng, [70] * 40, [700] * 40, 16, spare=5000)
    t, nf = dev(table), dev(np.array([n_free], np.int32))
    c, a, f = dev(cached), dev(added), dev(free)
    qs = torch.zeros(41, dtype=torch.int32, device="cuda")
    kl = torch.zeros(40, dtype=torch.int32, device="cuda")
    sl, po = (torch.zeros(30000, dtype=torch.int64, device="cuda") for _ in range(2))
    ws = fresh_ws(abi, abi.STATUS_BYTES)
    for _ in range(3):
        abi.csa2_page_plan(c, a, 40, 16, t, table.shape[1], f, n_pages, nf, nf, qs, kl, sl, po, 30000, ws, ws.numel(), None)
        torch.cuda.synchronize()
        want = PO.page_plan(cached, added, 16, table, free, n_free, n_pages, 30000)
        n_free = want[5]
        table = want[0]
        check_plan((t.cpu().numpy(), qs.cpu().numpy(), kl.cpu().numpy(), sl.cpu().numpy(), po.cpu().numpy(), int(nf.item())), want)


# ------------------------------------------------ what a call may be given
def at16(t):
    """The same tensor 16 bytes behind a 32-byte boundary."""
    v = torch.empty(t.numel() * t.element_size() + 16, dtype=torch.uint8, device="cuda")[16:].view(t.dtype).view(t.shape)
    assert v.data_ptr() % 32 == 16
    return v.copy_(t)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kv,new,window,bound", [
    ([500, 33, 300], [2, 1, 3], 0, 500), ([300, 90], [40, 9], 0, 300), ([700, 300], [40, 1], 0, 1000),
    ([2600, 2300, 900], [40, 1, 1], 0, 2600), ([900, 300], [40, 30], 400, 900)])  # few rows, few tiles, tiles, both, window
def test_attention_of_pointers_at_16_bytes(abi, kv, new, window, bound, fmt):
    """Every operand 16-byte aligned and no more: the bits of the call on 256-byte aligned ones."""
    s = attn_inputs(np.random.default_rng(61), kv, new, 64, 16, fmt)
    a = Attn(abi, s, window, max_kv=bound)
    a.call()
    want = a.result()
    check_attn(*want, s, window)
    for name in ("q", "q_start", "kv_len", "codes", "scales", "table", "out", "lse", "ws"):
        if getattr(a, name) is not None:
            setattr(a, name, at16(getattr(a, name)))
    a.out.fill_(7), a.lse.fill_(7)
    a.call()
    got = a.result()
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    assert abi.csa2_status_fetch(a.ws)[0] == abi.OK


def test_products_norms_and_plans_of_pointers_at_16_bytes(abi):
    rng = np.random.default_rng(62)
    codes, scales = (at16(dev(v)) for v in weight(rng, 300, 640))
    ws = fresh_ws(abi, abi.csa2_fp4_matvec_workspace_bytes(5, 640, 300) + 16)[16:]
    out = at16(torch.zeros(5, 300, device="cuda"))
    for xt, xs in ((bf16(rng.standard_normal((5, 640))), None),
                   (torch.randn(5, 640, generator=torch.Generator().manual_seed(1)).to(torch.float8_e4m3fn), np.ones(5, np.float32))):
        abi.csa2_fp4_matvec(at16(xt.cuda().view(torch.uint8)), abi.X_BF16 if xs is None else abi.X_E4M3,
                            None if xs is None else at16(dev(xs)), 640, 5, 640, codes, scales, 300, 1.0, out, abi.OUT_F32, ws,
                            ws.numel())
        torch.cuda.synchronize()
        check_matvec(out.double().cpu().numpy(), xt, xs, codes.cpu().numpy(), scales.cpu().numpy(), 1.0, torch.float32)
    x, w = bf16(rng.standard_normal((9, 640))), bf16(rng.standard_normal(640))
    res, y = at16(torch.zeros(9, 640, dtype=torch.bfloat16, device="cuda")), at16(torch.zeros(9, 640, dtype=torch.bfloat16, device="cuda"))
    c, sc = at16(torch.zeros(9, 640, dtype=torch.uint8, device="cuda")), at16(torch.zeros(9, 5, device="cuda"))
    abi.csa2_rmsnorm_fp8(at16(x.cuda()), 640, res, res, at16(w.cuda()), 9, 640, 1e-6, 128, c, sc, y)
    torch.cuda.synchronize()
    check_norm(x.double().numpy(), w.double().numpy(), 128, c.view(torch.float8_e4m3fn).double().cpu().numpy(),
               sc.cpu().numpy(), y.double().cpu().numpy())
    cached, added, table, free, n_free, n_pages = plan_inputs(rng, [9, 30], [20, 5], 8)
    t, q, k = at16(dev(table)), *(at16(torch.zeros(n, dtype=torch.int32, device="cuda")) for n in (3, 2))
    sl, po = (at16(torch.zeros(40, dtype=torch.int64, device="cuda")) for _ in range(2))
    nf, ws = at16(dev(np.array([n_free], np.int32))), fresh_ws(abi, abi.STATUS_BYTES + 16)[16:]
    abi.csa2_page_plan(at16(dev(cached)), at16(dev(added)), 2, 8, t, table.shape[1], at16(dev(free)), n_pages, nf, nf, q, k, sl, po, 40,
                       ws, ws.numel())
    torch.cuda.synchronize()
    check_plan(tuple(v.cpu().numpy() for v in (t, q, k, sl, po)) + (int(nf.item()),),
               PO.page_plan(cached, added, 8, table, free, n_free, n_pages, 40))


# -------------------------------------------------- the cache between steps
def cache_step(cache, g, added, captured=None):
    """One step of random latents and queries (n tokens in all) over the cache, eager or by replaying a graph."""
    q, lat = captured[1:] if captured else (torch.empty(16, cache.heads, D, dtype=torch.bfloat16, device="cuda"),
                                            torch.empty(16, D, dtype=torch.bfloat16, device="cuda"))
    q.copy_(torch.randn(q.shape, generator=g)), lat.copy_(torch.randn(lat.shape, generator=g))
    cache.added.copy_(torch.tensor(added, dtype=torch.int32))

    def calls():
        cache.plan()
        cache.append(lat, 16)
        cache.attend(q, 16, 16, 96)
        cache.advance()
    torch.cuda.synchronize()
    if captured is None:
        calls()
    elif captured[0] is None:
        cache.workspace(16, 16, 96)
        captured[0] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured[0]):
            calls()
    if captured:
        captured[0].replay()
    torch.cuda.synchronize()


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("refused", [[0, 97, 0], [16, 40, 16], [-1, 1, 1]])  # a table row too short, too few pages, a bad length
def test_refused_step_leaves_the_cache_as_it_was(abi, captured, refused):
    """A step that the plan refuses, advanced over like any other, changes nothing: the steps behind it are those of a
    cache that never saw it."""
    from csa2_sparse_attention_gb300 import paged
    runs = []
    for also in (False, True):
        cache = paged.PagedLatents(3, 97, 7, 16, 6, heads=4, fmt=abi.FMT_FP4)
        g, use = torch.Generator().manual_seed(3), [None, torch.zeros(16, 4, D, dtype=torch.bfloat16, device="cuda"),
                                                    torch.zeros(16, D, dtype=torch.bfloat16, device="cuda")] if captured else None
        cache_step(cache, g, [10, 4, 2], use)
        cache_step(cache, g, [6, 9, 1], use)
        if also:
            before = [t.clone() for t in (cache.cached, cache.table, cache.n_free, cache.codes, cache.scales)]
            assert cache.cached.tolist() == [16, 13, 3] and cache.status()["plan"][0] == abi.OK
            state = g.get_state()
            cache_step(cache, g, refused, use)
            g.set_state(state)
            assert cache.status()["plan"][0] == abi.ERR_DEVICE_BOUNDS
            for got, want in zip((cache.cached, cache.table, cache.n_free, cache.codes, cache.scales), before):
                assert torch.equal(got, want)
        cache_step(cache, g, [1, 14, 1], use)
        cache_step(cache, g, [0, 1, 15], use)
        cache.advance()  # once more changes nothing
        assert cache.cached.tolist() == [17, 28, 19]
        runs.append([t.clone() for t in (cache.cached, cache.table, cache.n_free, cache.kv_len, cache.codes, cache.scales, cache.out,
                                         cache.lse)])
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_advance_and_status_of_a_step_on_another_stream(abi):
    """The step's stream is held up by other work: what advance() and status() take from the step comes behind it."""
    runs = []
    for apart in (False, True):
        paged, g, cache, layer = layer_case(abi, abi.FMT_FP4, 0)
        st = torch.cuda.Stream() if apart else None
        x = torch.randn(56, layer.hidden, generator=g).to(torch.bfloat16).cuda()
        tok = torch.randn(3, layer.hidden, generator=g).to(torch.bfloat16).cuda()
        cache.workspace(56, 30, 64)
        torch.cuda.synchronize()
        for added, rows in (([30, 9, 17], x), ([1, 1, 1], tok)):
            cache.added.copy_(torch.tensor(added, dtype=torch.int32))
            layer.residual.zero_()
            torch.cuda.synchronize()
            if apart:
                with torch.cuda.stream(st):
                    torch.cuda._sleep(200_000_000)
            layer.step(rows, len(rows), 30, 64, st)
            cache.advance(st)
            torch.cuda.synchronize()
        cache.table[0, 1] = cache.n_pages
        assert cache.cached.tolist() == [31, 10, 18]
        cache.added.fill_(0)
        cache.added[0] = 1  # its page is the one outside
        torch.cuda.synchronize()
        if apart:
            with torch.cuda.stream(st):
                torch.cuda._sleep(200_000_000)
        layer.step(tok[:1], 1, 30, 64, st)
        assert cache.status(st)["plan"][0] == cache.status(st)["attn"][0] == abi.ERR_DEVICE_BOUNDS
        runs.append((cache.cached.clone(), cache.codes.clone(), cache.out[:3].clone()))
    for a, b in zip(*runs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("handle", [False, True])  # the stream as an object, as a number
def test_capture_on_the_given_stream(abi, handle):
    """A stream that is being captured while another one is current: its step's workspace stays in the graph, and one
    that would have to grow it is refused without ending the capture."""
    paged, g, cache, layer = layer_case(abi, abi.FMT_FP4, 0)
    cache.added.copy_(torch.tensor([30, 9, 17], dtype=torch.int32))
    layer.step(torch.randn(56, layer.hidden, generator=g).to(torch.bfloat16).cuda(), 56, 30, 64)
    cache.advance()
    cache.added.fill_(0)
    cache.plan()
    cache.q_start.copy_(torch.tensor([0, 1, 2, 3], dtype=torch.int32))  # (a query over what is there)
    q = layer.q[:3].clone()
    cache.attend(q, 3, 1, 64)
    torch.cuda.synchronize()
    want, held = cache.out[:3].clone(), cache.ws_attn
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    given = st.cuda_stream if handle else st
    with torch.cuda.stream(st):
        graph.capture_begin(capture_error_mode="thread_local")
    try:
        cache.attend(q, 3, 1, 64, given)
        with pytest.raises(RuntimeError, match="captured"):
            cache.attend(q, 3, 3, 1 << 16, given)
    finally:
        with torch.cuda.stream(st):
            graph.capture_end()
    cache.attend(q, 3, 3, 1 << 16)
    assert cache.ws_attn is not held and any(w is held for w in cache._kept)
    cache.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache.out[:3], want) and cache.status()["attn"][0] == abi.OK


def test_status_outlives_its_workspace(abi):
    """A problem that a step recorded is still there after a larger step took another workspace."""
    paged, g, cache, layer = layer_case(abi, abi.FMT_FP4, 0)
    cache.added.copy_(torch.tensor([30, 9, 17], dtype=torch.int32))
    x = torch.randn(56, layer.hidden, generator=g).to(torch.bfloat16).cuda()
    layer.step(x, 56, 20, 64)  # request 0 brings more than max_q
    first = cache.status()["attn"]
    assert first == [abi.ERR_DEVICE_BOUNDS, 9, 0, 30]
    held = cache.ws_attn
    for kv in (1000, 1 << 16):
        cache.attend(layer.q, 56, 30, kv)
        assert cache.ws_attn is not held and not cache._kept and cache.status()["attn"] == first
        held = cache.ws_attn
    abi.csa2_status_reset(cache.ws_attn)
    cache.attend(layer.q, 56, 30, 64)
    assert cache.ws_attn is held and cache.status()["attn"][0] == abi.OK


@pytest.mark.parametrize("captured", [False, True])
def test_refused_bounds_leave_the_step_undone(abi, captured):
    """A step whose bounds are refused (too large, or a capture that would need a larger workspace) has changed nothing."""
    paged, g, cache, layer = layer_case(abi, abi.FMT_FP4, 0)
    x = torch.randn(56, layer.hidden, generator=g).to(torch.bfloat16).cuda()
    cache.added.copy_(torch.tensor([30, 9, 17], dtype=torch.int32))
    layer.step(x, 56, 30, 64)
    cache.advance()
    cache.added.fill_(1)
    state = lambda: [t.clone() for t in (layer.residual, layer.x, layer.q, cache.table, cache.n_free, cache.kv_len, cache.q_start,  # noqa: E731
                                         cache.slots, cache.codes, cache.out)]
    before = state()
    torch.cuda.synchronize()
    if captured:
        with pytest.raises(RuntimeError, match="captured"):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                layer.step(x, 3, 1, 1 << 16)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):  # what was captured before the refusal, if a caller goes on
            with pytest.raises(RuntimeError, match="captured"):
                layer.step(x, 3, 1, 1 << 16)
        graph.replay()
    else:
        with pytest.raises(ValueError):
            layer.step(x, 3, 1, (1 << 30) + 1)
    torch.cuda.synchronize()
    for a, b in zip(state(), before):
        assert torch.equal(a, b)


def test_step_refuses_host_tensors(abi):
    paged, g, cache, layer = layer_case(abi, abi.FMT_FP4, 0)
    c0 = abi.csa2_launch_count()
    with pytest.raises(ValueError, match="hidden: on cpu"):
        layer.step(torch.zeros(3, layer.hidden, dtype=torch.bfloat16), 3, 1, 64)
    with pytest.raises(ValueError, match="q: on cpu"):
        cache.attend(torch.zeros(3, cache.heads, D, dtype=torch.bfloat16), 3, 1, 64)
    assert abi.csa2_launch_count() == c0


@pytest.mark.parametrize("n,kv", [(1, 3000), (4, 2000), (40, 4000)])  # few rows; tiles; with split keys
@pytest.mark.parametrize("order", ["behind it", "before it", "empty ones"])
def test_attention_of_good_requests_beside_token_bounds_out_of_order(abi, n, kv, order):
    """A request whose tokens run past the call's, or backwards, is recorded and skipped; the one beside it is whole."""
    rng = np.random.default_rng(71)
    if order == "before it":    # tokens n .. 2n - 1 are the last request's
        s = attn_inputs(rng, [30, 40, kv], [n, 0, n], 64, 16, "fp4")
        starts, mine = [0, 1000 + n, n, 2 * n], [n, n, n, 2 * n]
    elif order == "behind it":  # tokens 0 .. n - 1 are the first one's
        s = attn_inputs(rng, [kv, 50, 60, 0], [n, 0, 0, 0], 64, 16, "fp4")
        starts, mine = [0, n, -1, 0, 0], [0, n, n, n, n]
    else:
        s = attn_inputs(rng, [20, kv, 60, 70, 80, 90], [0, n, 0, 0, 0, 0], 64, 16, "fp4")
        starts, mine = [0, 0, n, -5, -5, -2, 0], [0, 0, n, n, n, n, n]
    a = Attn(abi, dict(s, q_start=np.array(starts, np.int32)), max_q=n)
    a.call()
    out, lse = a.result()
    first = mine[0]
    assert (out[:first] == 7).all() and (lse[:first] == 7).all()
    out[:first], lse[:first] = 0, -np.inf
    check_attn(out, lse, dict(s, q_start=np.array(mine, np.int32)), 0)
    assert abi.csa2_status_fetch(a.ws)[:2] == [abi.ERR_DEVICE_BOUNDS, 9]


def test_step_of_no_tokens(abi):
    """An idle step, with an empty tensor: nothing but the plan's outputs changes, and the next step goes on."""
    runs = []
    for idle in (False, True):
        paged, g, cache, layer = layer_case(abi, abi.FMT_FP4, 0)
        x = torch.randn(56, layer.hidden, generator=g).to(torch.bfloat16).cuda()
        cache.added.copy_(torch.tensor([30, 9, 17], dtype=torch.int32))
        layer.step(x, 56, 30, 64)
        cache.advance()
        if idle:
            cache.added.zero_()
            out, lse = layer.step(x[:0], 0, 0, 64)
            assert out.shape == (0, cache.heads, D) and lse.shape == (0, cache.heads)
            cache.append(layer.latents[:0], 0)
            cache.advance()
            assert cache.kv_len.tolist() == cache.cached.tolist() == [30, 9, 17] and not cache.q_start.any()
        cache.added.fill_(1)
        layer.step(x[:3], 3, 1, 64)
        torch.cuda.synchronize()
        assert all(st[0] == abi.OK for st in cache.status().values())
        runs.append([t.clone() for t in (cache.out, cache.lse, cache.codes, cache.table, cache.n_free, layer.residual)])
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def turned(q, pos, theta=10000.0):
    """Queries [n][heads][512] turned in place by their positions, pairs (2i, 2i+1), in 64 bits, rounded once."""
    ang = pos[:, None, None].double() * theta ** (-torch.arange(D // 2, device=q.device).double() * 2 / D)
    e, o = q[..., 0::2].double(), q[..., 1::2].double()
    q.copy_(torch.stack((e * ang.cos() - o * ang.sin(), e * ang.sin() + o * ang.cos()), -1).flatten(-2))


@pytest.mark.parametrize("captured", [False, True])
def test_step_with_rotated_queries(abi, captured):
    """Queries are turned by the plan's positions between the products and the attention: a chunk, then single tokens."""
    paged, g, cache, layer = layer_case(abi, abi.FMT_FP4, 0)
    tok = torch.zeros(56, layer.hidden, dtype=torch.bfloat16, device="cuda")
    for added in ([30, 9, 17], [1, 1, 1]):
        n, graph = sum(added), torch.cuda.CUDAGraph()
        cache.added.copy_(torch.tensor(added, dtype=torch.int32))
        tok[:n] = torch.randn(n, layer.hidden, generator=g).to(torch.bfloat16)
        layer.residual.zero_()
        if captured:
            cache.workspace(n, 30, 64)
            with torch.cuda.graph(graph):
                layer.step(tok[:n], n, 30, 64, rotate=turned)
            graph.replay()
        else:
            layer.step(tok[:n], n, 30, 64, rotate=turned)
        torch.cuda.synchronize()
        assert all(st[0] == abi.OK for st in cache.status().values()) and cache.pos[:n].min() >= 0
        xs, w = layer.x_scales[:n].cpu().numpy(), [t.cpu().numpy() for t in layer.wq]
        raw, reach = PO.matvec(layer.x[:n].view(torch.float8_e4m3fn).double().cpu().numpy(), xs, *w, 1.0)
        turn = lambda v: O.rope(v.reshape(-1, D), np.repeat(cache.pos[:n].cpu().numpy(), cache.heads)).reshape(n, -1)  # noqa: E731
        # the product's fp32 sum and its rounding to bf16 (2^-8 relative), times at most sqrt(2) for a turned pair, and one more
        pair = np.repeat(np.hypot(raw[:, 0::2], raw[:, 1::2]), 2, axis=1)
        tol = 1.5 * (2.0 ** -8 * pair + 64 * 2.0 ** -24 * np.repeat(np.maximum(reach[:, 0::2], reach[:, 1::2]), 2, axis=1)) + 2.0 ** -8 * pair
        q = layer.q[:n].double().cpu().numpy().reshape(n, -1)
        assert (np.abs(q - turn(raw)) <= tol).all() and (np.abs(q - raw) > tol).any()
        s = dict(q=layer.q[:n].cpu(), q_start=cache.q_start.cpu().numpy(), kv_len=cache.kv_len.cpu().numpy(),
                 codes=cache.codes.cpu().numpy(), scales=cache.scales.cpu().numpy(), table=cache.table.cpu().numpy(), page=cache.page_size,
                 fmt="fp4", T=n, H=cache.heads, max_q=30, max_kv=64)
        check_attn(cache.out[:n].double().cpu().numpy(), cache.lse[:n].double().cpu().numpy(), s, 0)
        cache.advance()


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_step_without_a_rotary_embedding_goes_by_distances(abi, fmt):
    """A cache that does not rotate: the same tokens behind 48 others, outside the window of all but the first ones, have
    the same latents and (up to the order of fp32 sums, bounded as in check_attn) the same outputs."""
    from csa2_sparse_attention_gb300 import paged
    R, hidden, window = 1, 256, 16
    g = torch.Generator().manual_seed(5)
    w = lambda *sh: torch.randn(*sh, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    weights = (w(hidden), w(4 * D, hidden), w(D, hidden))
    before, x = w(48, hidden), w(40, hidden)
    runs = []
    for shift in (False, True):
        cache = paged.PagedLatents(R, 64, 8, 16, 8, heads=4, fmt=abi.FMT_FP4 if fmt == "fp4" else abi.FMT_FP8, window=window, rope_theta=None)
        layer = paged.PagedLayer(cache, hidden, *weights)
        for rows in ([before, x] if shift else [x]):
            cache.added.fill_(len(rows))
            layer.residual.zero_()
            layer.step(rows, len(rows), 64, 128)
            cache.advance()
        torch.cuda.synchronize()
        assert all(st[0] == abi.OK for st in cache.status().values())
        slots = cache.slots[:40].cpu().numpy()
        codes, scales = cache.codes.cpu().numpy(), None if fmt == "fp8" else cache.scales.cpu().numpy()
        s = dict(q=layer.q[:40].cpu(), q_start=cache.q_start.cpu().numpy(), kv_len=cache.kv_len.cpu().numpy(), codes=codes, scales=scales,
                 table=cache.table.cpu().numpy(), page=16, fmt=fmt, T=40, H=4, max_q=40, max_kv=int(cache.kv_len[0]))
        check_attn(cache.out[:40].double().cpu().numpy(), cache.lse[:40].double().cpu().numpy(), s, window)
        want, wlse, _ = PO.paged_attention(s["q"].float().numpy(), s["q_start"], s["kv_len"], codes, scales, s["table"], 16, window, SM)
        runs.append((codes[slots], None if scales is None else scales[slots], want[window:], wlse[window:], layer.q[:40].cpu()))
    a, b = runs
    assert torch.equal(a[4], b[4]) and np.array_equal(a[0], b[0]) and (a[1] is None or np.array_equal(a[1], b[1]))
    np.testing.assert_allclose(a[2], b[2], rtol=0, atol=1e-12 * np.abs(a[2]).max())
    np.testing.assert_allclose(a[3], b[3], rtol=1e-12)


def test_step_on_another_stream_than_the_cache_was_made_on(abi):
    """The stream that fills a new cache and its weights is held up: a step on another one finds them filled."""
    from csa2_sparse_attention_gb300 import paged
    g = torch.Generator().manual_seed(2)
    w = lambda *sh: torch.randn(*sh, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    weights, x, added = (w(256), w(4 * D, 256), w(D, 256)), w(56, 256), torch.tensor([30, 9, 17], dtype=torch.int32).cuda()
    runs = []
    for apart in (False, True):
        torch.cuda.synchronize()
        st = torch.cuda.Stream() if apart else torch.cuda.current_stream()
        if apart:
            torch.cuda._sleep(200_000_000)
        cache = paged.PagedLatents(3, 64, 40, 16, 12, heads=4, fmt=abi.FMT_FP4)
        layer = paged.PagedLayer(cache, 256, *weights)
        with torch.cuda.stream(st):
            cache.added.copy_(added)
            layer.step(x, 56, 30, 30, st)
        torch.cuda.synchronize()
        assert all(s[0] == abi.OK for s in cache.status().values())
        runs.append([t.clone() for t in (cache.out, cache.lse, cache.codes, cache.table, cache.n_free, layer.residual)])
    for a, b in zip(*runs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n,dim,group", [(40, 16, 0), (30, 512, 0), (20, 1024, 128), (9, 1032, 0), (16, 5120, 0), (12, 7168, 128),
                                         (3, 16384, 0)])
@pytest.mark.parametrize("values", ["random", "whole numbers"])
def test_norm_codes_are_those_of_the_exact_quotient(abi, n, dim, group, values):
    """y / s = 448 h w / max|h w| whatever the root is: products of 16 bits, whose quotients lie on a border of two codes
    (then 64 bits have them exactly) or at least 2^-21 of it away.  So the codes can be compared for equality; whole
    numbers lie on borders often."""
    rng = np.random.default_rng(dim)
    if values == "random":
        x, w = bf16(np.exp(3 * rng.standard_normal((n, 1))) * rng.standard_normal((n, dim))), bf16(1 + 0.2 * rng.standard_normal(dim))
    else:
        x, w = bf16(rng.integers(-112, 113, (n, dim)) * 2.0 ** rng.integers(-20, 20, (n, 1))), bf16(2.0 ** rng.integers(-1, 2, dim))
    _, codes, scales, y = norm_call(abi, x, None, w, group)
    h, wd = x.double().numpy(), w.double().numpy()
    check_norm(h, wd, group, codes, scales, y)
    a = (h * wd).reshape(n, -1, group or dim)
    want = O.e4m3_decode(O.e4m3_encode(448.0 * a / np.abs(a).max(axis=2, keepdims=True))).reshape(n, dim)
    assert np.array_equal(codes, want)
