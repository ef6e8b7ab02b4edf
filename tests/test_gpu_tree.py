"""The operators of a step of trees against their 64-bit forms: head norms with rotation and append, positions and
masks, attention, log probabilities, the commit; graphs, streams, and whole steps of them together."""
import math

import numpy as np
import pytest
import torch

from oracle import csa2_oracle as O
from oracle import paged_oracle as PO
from oracle import tree_oracle as TO
from tests.test_gpu_paged import attn_inputs, bf16, check_attn, dev, fresh_ws

pytestmark = pytest.mark.gpu
D = 512
SM = 1.0 / math.sqrt(D)
U = 2.0 ** -24


@pytest.fixture(scope="module")
def abi():
    from csa2_sparse_attention_gb300 import abi as A
    return A


def f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------ head norms
class Heads:
    """One call: inputs, outputs filled with what is to stay where nothing is written."""

    def __init__(self, abi, rng, n, heads, fmt, qn=True, ln=True, turn=True, q_gap=0, l_gap=0, amp=1.0, pos=None, dst=None, extra=3,
                 in_place=False, shift=0, dst_null=False):
        self.abi, self.n, self.heads, self.fmt = abi, n, heads, fmt
        x = amp * rng.standard_normal((max(n, 1), heads * D + q_gap)) * np.exp(rng.standard_normal((max(n, 1), 1)))
        flat = torch.zeros(x.size + shift, dtype=torch.bfloat16)
        flat[shift:] = bf16(x).flatten()
        self.q_flat = flat.cuda()
        self.q_stride, self.l_stride = heads * D + q_gap, D + l_gap
        self.q = self.q_flat[shift:].view(max(n, 1), -1)
        self.lat = bf16(amp * rng.standard_normal((max(n, 1), self.l_stride))).cuda()
        self.x64, self.lat64 = f64(self.q)[:n, :heads * D].reshape(n, heads, D), f64(self.lat)[:n, :D]
        weight = lambda on: bf16(1 + 0.3 * rng.standard_normal(D)).cuda() if on else None  # noqa: E731
        self.qw, self.lw = weight(qn), weight(ln)
        self.max_pos = 5000
        self.pos64 = rng.integers(0, self.max_pos, n) if pos is None else np.asarray(pos)
        self.n_rows = n + extra
        self.dst64 = (np.arange(n) if dst_null else rng.permutation(self.n_rows)[:n]) if dst is None else np.asarray(dst)
        self.pos, self.dst = dev(self.pos64.astype(np.int64)), None if dst_null else dev(self.dst64.astype(np.int64))
        self.turn = turn
        self.table = None
        if turn:
            self.table = torch.zeros(abi.csa2_rope_table_bytes(D, self.max_pos), dtype=torch.uint8, device="cuda")
            abi.csa2_rope_table_init(10000.0, D, self.max_pos, self.table)
        out = torch.full((max(n, 1) * heads * D + shift,), 7.0, dtype=torch.bfloat16, device="cuda")
        self.out = self.q if in_place else out[shift:].view(max(n, 1), -1)
        fp4 = fmt == "fp4"
        self.codes = torch.full((self.n_rows, D // 2 if fp4 else D), 0x35, dtype=torch.uint8, device="cuda")
        self.scales = torch.full((self.n_rows, D // 16), 0x35, dtype=torch.uint8, device="cuda") if fp4 else None
        self.ws = fresh_ws(abi, abi.STATUS_BYTES)

    def call(self, stream=None, queries=True, latents=True, eps=1e-6):
        q, lat = queries, latents
        self.abi.csa2_head_norm_rope(
            self.q if q else None, self.q_stride, self.heads, self.qw if q else None, self.out if q else None, self.lat if lat else None,
            self.l_stride, self.lw if lat else None, self.n, eps, self.pos, self.table, self.max_pos if self.turn else 0,
            self.abi.FMT_FP4 if self.fmt == "fp4" else self.abi.FMT_FP8, self.dst, self.n_rows, self.codes if lat else None,
            self.scales if lat else None, self.ws, self.ws.numel(), stream)
        torch.cuda.synchronize()
        return self

    def check(self, queries=True, latents=True, eps=1e-6, live=None):
        """Queries: y is off by 2^-20 (|h0| + |h1|) of its pair at most (h the normed values; the kernel's own comment counts
        13 roundings of 2^-24), then bf16 rounds once, 2^-8 relative.  Latents are the codes of 64-bit arithmetic, which
        differ in the last bits only where a value lies within 2^-40 of a border."""
        live = np.ones(self.n, bool) if live is None else live
        pos = np.where(live, self.pos64, 0)
        if queries:
            h = TO.head_norm(self.x64, None if self.qw is None else f64(self.qw), eps)
            want = TO.turned(h, pos) if self.turn else h
            got = f64(self.out)[:self.n].reshape(self.n, self.heads, D)
            pair = np.repeat(np.abs(h[..., 0::2]) + np.abs(h[..., 1::2]), 2, -1)
            tol = 2.0 ** -20 * pair * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
            assert (np.abs(got - want) <= tol)[live].all(), (np.abs(got - want) - tol)[live].max()
            assert (got[~live] == (self.x64[~live] if self.out is self.q else 7.0)).all()
        codes = self.codes.cpu().numpy()
        left = np.ones(self.n_rows, bool)
        if latents:
            h = TO.head_norm(self.lat64, None if self.lw is None else f64(self.lw), eps)
            want = TO.turned(h, pos) if self.turn else h
            rows = self.dst64[live]
            left[rows] = False
            if self.fmt == "fp4":
                c, s = O.quantize_fp4(want[live])
                np.testing.assert_array_equal(self.scales.cpu().numpy()[rows], s)
                np.testing.assert_array_equal(O.e2m1_decode(O.unpack_codes(codes[rows])), O.e2m1_decode(c))
            else:
                np.testing.assert_array_equal(O.e4m3_decode(codes[rows]), O.e4m3_decode(O.e4m3_encode(want[live])))
        assert (codes[left] == 0x35).all()
        if self.scales is not None:
            assert (self.scales.cpu().numpy()[left] == 0x35).all()


@pytest.mark.parametrize("n,heads,fmt,kw", [
    (1, 1, "fp4", {}), (1, 64, "fp4", {}), (16, 64, "fp4", {}), (7, 5, "fp8", dict(turn=False)), (33, 128, "fp4", dict(ln=False)),
    (300, 64, "fp4", {}), (41, 16, "fp8", dict(q_gap=512, l_gap=16 * 512)), (9, 3, "fp4", dict(q_gap=8, l_gap=8, shift=8)),
    (25, 8, "fp8", dict(qn=False, ln=False)), (25, 8, "fp4", dict(qn=False, ln=False)), (12, 24, "fp4", dict(in_place=True)),
    (12, 24, "fp8", dict(in_place=True, shift=8)), (10, 2, "fp4", dict(turn=False, qn=False)), (6, 2, "fp8", dict(qn=False, ln=False, turn=False)),
    (14, 7, "fp4", dict(dst_null=True)), (1500, 9, "fp8", {}), (3000, 1, "fp4", {})])
def test_heads(abi, n, heads, fmt, kw):
    Heads(abi, np.random.default_rng(n + heads), n, heads, fmt, **kw).call().check()


@pytest.mark.parametrize("what", ["queries", "latents"])
def test_heads_of_one_kind(abi, what):
    h = Heads(abi, np.random.default_rng(1), 19, 6, "fp4")
    q = what == "queries"
    h.call(queries=q, latents=not q).check(queries=q, latents=not q)
    if not q:
        assert (h.out == 7.0).all()


def test_heads_leave_out_what_is_padded_and_record_what_is_not(abi):
    rng = np.random.default_rng(2)
    pos = np.array([5, -1, 4999, 0, 77, -1])
    h = Heads(abi, rng, 6, 3, "fp4", pos=pos, dst=[3, -1, 0, 8, 1, -1])
    h.call().check(live=pos >= 0)
    assert abi.csa2_status_fetch(h.ws)[0] == abi.OK
    for bad, kw in (("pos", dict(pos=[5, 5000, 9])), ("pos", dict(pos=[5, -2, 9])), ("dst", dict(dst=[0, 6, 1])), ("dst", dict(dst=[0, -2, 1]))):
        h = Heads(abi, rng, 3, 3, "fp8", **kw)
        if bad == "pos":
            h.call().check(live=np.array([True, False, True]))
        else:  # the token's queries are good
            h.call()
            got, alive = h.codes.cpu().numpy(), np.array([True, False, True])
            w = TO.turned(TO.head_norm(h.lat64, f64(h.lw), 1e-6), h.pos64)
            np.testing.assert_array_equal(O.e4m3_decode(got[[0, 1]]), O.e4m3_decode(O.e4m3_encode(w[alive])))
            assert (got[2:] == 0x35).all()
        st = abi.csa2_status_fetch(h.ws)
        assert st[0] == abi.ERR_DEVICE_BOUNDS and st[2] == 1, st


def test_heads_without_rotation_below_position_zero(abi):
    pos = np.array([-1, 3, 1 << 40])
    h = Heads(abi, np.random.default_rng(3), 3, 2, "fp4", turn=False, pos=pos)
    h.call().check(live=pos >= 0)
    assert abi.csa2_status_fetch(h.ws)[0] == abi.OK


def test_heads_far_positions(abi):
    """Angles of positions near a million, by the table's addition of two angles."""
    h = Heads(abi, np.random.default_rng(4), 64, 2, "fp4")
    h.max_pos = 1 << 20
    h.table = torch.zeros(abi.csa2_rope_table_bytes(D, h.max_pos), dtype=torch.uint8, device="cuda")
    abi.csa2_rope_table_init(10000.0, D, h.max_pos, h.table)
    h.pos64 = np.random.default_rng(5).integers((1 << 20) - 3000, 1 << 20, 64)
    h.pos = dev(h.pos64)
    h.call().check()


@pytest.mark.parametrize("amp,eps", [(2.0 ** 55, 1e-6), (2.0 ** -40, 1e-6), (2.0 ** -50, 0.0), (1.0, 0.0), (300.0, 100.0)])
def test_heads_ranges(abi, amp, eps):
    h = Heads(abi, np.random.default_rng(6), 20, 4, "fp4", amp=min(amp, 2.0 ** 50))
    h.call(eps=eps).check(eps=float(np.float32(eps)))


def test_heads_zeros_nan_and_infinity(abi):
    """A row of zeros stays one; NaN and infinity stay in their rows: NaN in a normed query, a NaN scale in FP4."""
    for fmt in ("fp4", "fp8"):
        h = Heads(abi, np.random.default_rng(7), 6, 2, fmt, dst_null=True)
        h.q[0, :D] = 0
        h.q[1, 5] = float("nan")
        h.q[2, D + 9] = float("inf")
        h.lat[0] = 0
        h.lat[1, 40] = float("nan")
        h.lat[2, 40] = float("-inf")
        h.call(eps=0.0)
        out = f64(h.out).reshape(6, 2, D)
        assert (out[0, 0] == 0).all() and np.isnan(out[1, 0]).all() and np.isnan(out[2, 1, 8:10]).all()
        assert np.isfinite(out[[0, 1, 2, 3, 4, 5], [1, 1, 0, 0, 0, 0]]).all() and np.isfinite(out[3:]).all()
        codes = h.codes.cpu().numpy()
        if fmt == "fp4":
            s = h.scales.cpu().numpy()
            assert (s[0] == 0).all() and (s[1] == 0x7F).all() and s[2, 2] == 0x7F and (s[3:] != 0x7F).all()
        else:
            assert np.isnan(O.e4m3_decode(codes[1])).all() and (O.e4m3_decode(codes[0]) == 0).all() and not np.isnan(O.e4m3_decode(codes[3:6])).any()


def test_heads_codes_next_to_borders(abi):
    """Values within the fp32 error of a border between two codes: the exact ones decide.  Rows of powers of two and
    small whole numbers, whose quotients lie on borders, normed by eps alone or not at all."""
    rng = np.random.default_rng(8)
    for fmt in ("fp4", "fp8"):
        h = Heads(abi, rng, 200, 1, fmt, turn=False)
        x = rng.integers(-24, 25, (200, D)) * 2.0 ** rng.integers(-3, 3, (200, 1))
        h.lat[:] = bf16(x).cuda()
        h.lat64 = f64(h.lat)
        h.lw = bf16(2.0 ** rng.integers(-1, 2, D)).cuda()
        h.call().check()
        h.lw = None
        h.call().check()


def test_heads_append_is_the_append(abi):
    """Without norms the rows are those of csa2_quantize_append, byte for byte where no value is minus zero."""
    h = Heads(abi, np.random.default_rng(9), 500, 1, "fp4", ln=False)
    h.call(queries=False)
    codes, scales, ws = torch.full_like(h.codes, 0x35), torch.full_like(h.scales, 0x35), fresh_ws(abi, abi.STATUS_BYTES)
    abi.csa2_quantize_append(h.lat, 500, D, abi.FMT_FP4, abi.LAYOUT_ROWS, h.pos, h.table, h.max_pos, h.dst, h.n_rows, codes, scales, ws,
                             ws.numel())
    torch.cuda.synchronize()
    assert torch.equal(scales, h.scales)
    np.testing.assert_array_equal(O.e2m1_decode(O.unpack_codes(codes.cpu().numpy())), O.e2m1_decode(O.unpack_codes(h.codes.cpu().numpy())))


# ---------------------------------------------------------- plan and mask
def trees(rng, nodes, shape="random"):
    parent = []
    for n in nodes:
        for i in range(n):
            if i == 0:
                parent.append(-1)
            elif shape == "chain":
                parent.append(i - 1)
            elif shape == "star":
                parent.append(0)
            elif shape == "roots":
                parent.append(int(rng.integers(-1, i)))
            else:
                parent.append(int(rng.integers(max(0, i - 6), i)))
    return np.array(parent, np.int32).reshape(-1)


class Plan:
    def __init__(self, abi, parent, q_start, kv_len, window=0, max_q=None, tail=3):
        self.abi, self.parent, self.window, self.tail = abi, parent, window, tail
        self.q_start, self.kv_len = np.asarray(q_start, np.int32), np.asarray(kv_len, np.int32)
        self.max_q = int(np.diff(q_start).max(initial=0)) if max_q is None else max_q
        self.n, self.words = len(parent), -(-self.max_q // 32)
        self.d = [dev(np.concatenate([parent, np.full(tail, 5, np.int32)])), dev(self.q_start), dev(self.kv_len)]
        self.pos = torch.full((self.n + tail,), -9, dtype=torch.int64, device="cuda")
        self.mask = torch.full((self.n + tail, max(self.words, 1)), -9, dtype=torch.int32, device="cuda")
        self.ws = fresh_ws(abi, abi.STATUS_BYTES)

    def call(self, stream=None):
        self.abi.csa2_tree_plan(*self.d, len(self.kv_len), self.n + self.tail, self.max_q, self.window, self.pos, self.mask, self.words,
                                self.ws, self.ws.numel(), stream)
        return self

    def check(self):
        torch.cuda.synchronize()
        T = self.n + self.tail
        pos, mask = TO.tree_plan(np.concatenate([self.parent, np.full(self.tail, 5)]), self.q_start, self.kv_len, self.window, self.words,
                                 np.full(T, -9, np.int64), np.full((T, max(self.words, 1)), -9, np.int32))
        np.testing.assert_array_equal(self.pos.cpu().numpy(), pos)
        np.testing.assert_array_equal(self.mask.cpu().numpy(), mask)
        return self.abi.csa2_status_fetch(self.ws)


def starts(nodes):
    return np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)


@pytest.mark.parametrize("nodes,shape", [([1], "chain"), ([1, 2, 31, 32, 33, 64, 65], "random"), ([1024], "chain"), ([1024, 3], "random"),
                                         ([200, 0, 7], "roots"), ([40, 129], "star"), ([0, 0, 5], "random"), ([300], "chain")])
@pytest.mark.parametrize("window", [0, 1, 5, 40])
def test_plan(abi, nodes, shape, window):
    rng = np.random.default_rng(len(nodes) + window)
    parent = trees(rng, nodes, shape)
    p = Plan(abi, parent, starts(nodes), np.asarray(nodes) + rng.integers(0, 100, len(nodes)), window)
    assert p.call().check()[0] == abi.OK


def test_plan_records_bad_parents_and_lengths(abi):
    rng = np.random.default_rng(0)
    nodes = [12, 9, 6]
    for place, value in ((3, 3), (4, 9), (5, -2), (0, 0), (2, 1 << 20)):
        parent = trees(rng, nodes)
        parent[12 + place] = value
        st = Plan(abi, parent, starts(nodes), np.asarray(nodes) + 5).call().check()
        assert st[0] == abi.ERR_DEVICE_BOUNDS and st[2:] == [12 + place, value]
    parent = trees(rng, nodes)
    st = Plan(abi, parent, starts(nodes), [20, 8, 6]).call().check()   # fewer entries than nodes
    assert st[0] == abi.ERR_DEVICE_BOUNDS and st[2] == 1
    p = Plan(abi, parent, starts(nodes), [20, 20, 20], max_q=11).call()  # a request above the bound is skipped
    torch.cuda.synchronize()
    assert (p.pos[:12] == -9).all() and (p.mask[:12] == -9).all() and (p.pos[12:27] >= 0).all() and (p.pos[27:] == -9).all()
    assert abi.csa2_status_fetch(p.ws)[0] == abi.ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("window", [0, 40])
def test_plan_loses_what_descends_from_a_bad_parent(abi, window):
    """Over several words of the mask, with nodes beside it that keep theirs."""
    parent = trees(np.random.default_rng(1), [200, 9], "chain")
    parent[70] = 71
    parent[150] = 30
    p = Plan(abi, parent, starts([200, 9]), [300, 9], window)
    assert p.call().check()[2:] == [70, 71]
    assert (p.pos[70:150] == -1).all() and (p.pos[:70] >= 0).all() and (p.pos[150:209] >= 0).all()


# --------------------------------------------------------------- attention
class Tree:
    """Plan and attention of trees over the pages of attn_inputs."""

    def __init__(self, abi, s, parent, window=0, max_q=None, max_kv=None, ws=None):
        self.abi, self.s, self.window, self.parent = abi, s, window, parent
        self.max_q = s["max_q"] if max_q is None else max_q
        self.max_kv = s["max_kv"] if max_kv is None else max_kv
        self.q, self.q_start, self.kv_len = s["q"].cuda(), dev(s["q_start"]), dev(s["kv_len"])
        self.codes, self.scales, self.table = dev(s["codes"]), None if s["scales"] is None else dev(s["scales"]), dev(s["table"])
        T = s["T"]
        self.par = dev(np.concatenate([parent, np.full(T - len(parent), -1, np.int32)]).astype(np.int32))
        self.words = -(-self.max_q // 32)
        self.pos = torch.full((T,), -1, dtype=torch.int64, device="cuda")
        self.mask = torch.zeros((T, max(self.words, 1)), dtype=torch.int32, device="cuda")
        self.out = torch.full((T, s["H"], D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((T, s["H"]), 7.0, device="cuda")
        size = abi.csa2_tree_attn_workspace_bytes(T, s["H"], len(s["kv_len"]), self.max_q, self.max_kv, window)
        assert size >= abi.STATUS_BYTES
        self.ws = fresh_ws(abi, size) if ws is None else ws

    def plan(self, stream=None):
        self.abi.csa2_tree_plan(self.par, self.q_start, self.kv_len, len(self.s["kv_len"]), self.s["T"], self.max_q, self.window, self.pos,
                                self.mask, self.words, self.ws, self.ws.numel(), stream)
        return self

    def call(self, stream=None):
        s = self.s
        self.plan(stream)
        self.abi.csa2_tree_attn(self.q, s["T"], s["H"], self.q_start, self.kv_len, len(s["kv_len"]), self.max_q, self.max_kv, self.pos,
                                self.mask, self.words, self.abi.FMT_FP4 if s["fmt"] == "fp4" else self.abi.FMT_FP8, self.codes, self.scales,
                                self.codes.shape[0], self.table, s["table"].shape[1], s["page"], self.window, SM, self.out, self.lse, self.ws,
                                self.ws.numel(), stream)
        return self

    def check(self, bad_page=None):
        """The bounds are those of the causal attention (tests/test_gpu_paged.py, check_attn): 64 u sum|q||c| sm of a logit, an
        exponential of 2^-21, probabilities in f16 (2^-11 relative, 2^-24 absolute), one rounding to bf16, sums of n terms."""
        torch.cuda.synchronize()
        s = self.s
        out, lse = f64(self.out), f64(self.lse)
        T = int(s["q_start"][-1])
        want, wlse, (dot, big) = TO.tree_attention(self.q.float().cpu().numpy(), self.parent, s["q_start"], s["kv_len"], s["codes"], s["scales"],
                                                   s["table"], s["page"], self.window, SM, bad_page)
        d = 64 * U * dot * SM + 2.0 ** -21
        tol = ((2 * d + 2.0 ** -11 + s["max_kv"] * U) * big)[..., None] + (2.0 ** -8 + s["max_kv"] * U) * np.abs(want)
        err = np.abs(out - want)[:T]
        assert np.isfinite(out[:T]).all()
        assert (err <= tol[:T]).all(), (err - tol[:T]).max()
        live = np.isfinite(wlse[:T])
        assert np.array_equal(np.isneginf(lse[:T]), ~live) and (out[:T][~live] == 0).all()
        ltol = d + s["max_kv"] * U + 2.0 ** -22 * (1 + np.abs(np.where(np.isfinite(wlse), wlse, 0)))
        assert (np.abs(lse[:T][live] - wlse[:T][live]) <= ltol[:T][live]).all()
        assert (out[T:] == 7).all() and (lse[T:] == 7).all()
        return self.abi.csa2_status_fetch(self.ws)


ATTN = [
    # cached, nodes, heads, page, fmt, window, shape
    ([0], [1], 64, 8, "fp4", 0, "chain"),
    ([0, 3, 200], [5, 9, 3], 64, 8, "fp4", 0, "random"),
    ([700, 130], [16, 1], 64, 64, "fp4", 0, "random"),
    ([2000], [16], 64, 64, "fp4", 0, "star"),
    ([90, 128, 127, 640, 1], [33, 32, 31, 64, 65], 8, 16, "fp4", 0, "random"),
    ([300, 17, 64], [3, 12, 1], 5, 8, "fp8", 0, "roots"),
    ([500, 90, 260], [40, 45, 3], 16, 16, "fp8", 128, "random"),
    ([500, 90], [40, 3], 24, 64, "fp4", 1, "random"),
    ([385, 129], [20, 70], 40, 8, "fp8", 3, "chain"),
    ([385, 2, 1000], [130, 90, 7], 5, 8, "fp4", 20, "chain"),
    ([1111], [200], 1, 200, "fp8", 0, "random"),
    ([600, 5], [260, 1], 2, 128, "fp4", 100, "random"),
    ([2500, 1900, 800], [60, 1, 64], 64, 64, "fp4", 0, "random"),
    ([900], [100], 128, 16, "fp8", 1000, "roots"),
    ([250], [1024], 3, 8, "fp4", 0, "random"),
]


@pytest.mark.parametrize("i", range(len(ATTN)))
@pytest.mark.parametrize("loose", [False, True])
def test_attention(abi, i, loose):
    """Both kernels: with bounds above the lengths short requests go beside or over the decoded tiles."""
    cached, nodes, H, page, fmt, window, shape = ATTN[i]
    rng = np.random.default_rng(100 + i)
    s = attn_inputs(rng, np.asarray(cached) + nodes, nodes, H, page, fmt, tail=2)
    parent = trees(rng, nodes, shape)
    t = Tree(abi, s, parent, window, max_q=min(1024, s["max_q"] + 300) if loose else None, max_kv=s["max_kv"] + 2000 if loose else None)
    assert t.call().check()[0] == abi.OK


@pytest.mark.parametrize("cached,nodes,H", [([700, 30], [16, 3], 64), ([1500], [100], 64), ([260, 5], [7, 1], 8)])
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_attention_of_chains_is_the_causal_one(abi, cached, nodes, H, fmt):
    s = attn_inputs(np.random.default_rng(7), np.asarray(cached) + nodes, nodes, H, 16, fmt)
    t = Tree(abi, s, trees(None, nodes, "chain")).call()
    out, lse = torch.zeros_like(t.out), torch.zeros_like(t.lse)
    ws = fresh_ws(abi, abi.csa2_paged_attn_workspace_bytes(s["T"], H, len(nodes), s["max_q"], s["max_kv"], 0))
    abi.csa2_paged_attn(t.q, s["T"], H, t.q_start, t.kv_len, len(nodes), s["max_q"], s["max_kv"], abi.FMT_FP4 if fmt == "fp4" else abi.FMT_FP8,
                        t.codes, t.scales, t.codes.shape[0], t.table, s["table"].shape[1], 16, 0, SM, out, lse, ws, ws.numel())
    assert t.check()[0] == abi.OK
    check_attn(f64(out), f64(lse), s, 0)  # the same bounds around the same values
    big = np.abs(f64(out)).max()
    assert np.abs(f64(out) - f64(t.out)).max() <= 2.0 ** -6 * big and (lse - t.lse).abs().max() <= 2.0 ** -14


@pytest.mark.parametrize("nodes", [[6, 4], [90, 70]])  # (the few-row kernel, decoded tiles)
@pytest.mark.parametrize("window", [0, 50])
def test_attention_leaves_out_what_is_masked(abi, nodes, window):
    """NaN latents in other branches, behind the sequence and outside the window reach no row that does not see them."""
    rng = np.random.default_rng(11)
    s = attn_inputs(rng, np.array([700, 230]) + nodes, nodes, 64, 16, "fp8")
    parent = np.concatenate([np.array([-1] + [0] * (n - 1), np.int32) for n in nodes])  # every node sees the root and itself
    row = lambda r, p: int(s["table"][r, p // 16]) * 16 + p % 16  # noqa: E731
    bad = [3, nodes[0] - 1]
    for j in bad:
        s["codes"][row(0, 700 + j)] = 0x7F
    if window:
        s["codes"][[row(0, p) for p in range(600)]] = 0x7F
    t = Tree(abi, s, parent, window).call()
    torch.cuda.synchronize()
    out = f64(t.out)
    assert np.isnan(out[bad]).all()
    s2 = dict(s, codes=s["codes"].copy())
    s2["codes"][(s2["codes"] & 0x7F) == 0x7F] = 0
    want, _, _ = TO.tree_attention(t.q.float().cpu().numpy(), parent, s["q_start"], s["kv_len"], s2["codes"], None, s["table"], 16, window, SM)
    good = np.setdiff1d(np.arange(s["T"]), bad)
    assert np.isfinite(out[good]).all() and np.abs(out[good] - want[good]).max() <= 2.0 ** -6 * np.abs(want).max()


@pytest.mark.parametrize("nodes", [[6, 4, 3], [90, 70, 80]])
def test_attention_rows_that_see_nothing(abi, nodes):
    """Nodes of a bad parent, what descends from them, and a request with fewer entries than nodes get zeros and -inf."""
    rng = np.random.default_rng(12)
    kv = np.array([300, 0, 500]) + nodes
    s = attn_inputs(rng, kv, nodes, 64, 16, "fp4")
    parent = trees(rng, nodes)
    parent[2] = 4
    parent[sum(nodes[:2]) + 1] = -5
    s["kv_len"][1] = nodes[1] - 1
    t = Tree(abi, s, parent).call()
    st = t.check()
    assert st[0] == abi.ERR_DEVICE_BOUNDS and np.isneginf(f64(t.lse)[2]).all() and np.isneginf(f64(t.lse)[nodes[0]]).all()


@pytest.mark.parametrize("nodes", [[5, 2], [80, 66]])
def test_attention_pages_outside_are_recorded(abi, nodes):
    s = attn_inputs(np.random.default_rng(13), np.array([400, 260]) + nodes, nodes, 64, 16, "fp4")
    n_pages = s["codes"].shape[0] // 16
    s["table"][0, 3], s["table"][1, -1 if nodes[1] > 60 else 16] = n_pages, -4
    t = Tree(abi, s, trees(np.random.default_rng(1), nodes))
    st = t.call().check(bad_page=lambda i: not 0 <= i < n_pages)
    assert st[0] == abi.ERR_DEVICE_BOUNDS


def test_attention_masks_of_the_caller(abi):
    """Masks that no tree has: any of the request's earlier nodes, or none at all (a row then has the cached entries)."""
    rng = np.random.default_rng(14)
    nodes = [40, 9]
    s = attn_inputs(rng, np.array([130, 0]) + nodes, nodes, 16, 8, "fp4")
    t = Tree(abi, s, trees(rng, nodes)).plan()
    see = np.tril(rng.random((2, 40, 40)) < 0.4)
    see[0, 5] = see[1, 3] = False
    words = np.zeros((49, 2), np.uint64)
    for r, n, a in ((0, 40, 0), (1, 9, 40)):
        for i in range(n):
            for j in np.flatnonzero(see[r, i, :n]):
                words[a + i, j // 32] |= np.uint64(1 << (j % 32))
    t.mask.copy_(dev(words.astype(np.uint32).view(np.int32)))
    t.plan = lambda stream=None: t
    t.call()
    torch.cuda.synchronize()
    out, lse = f64(t.out), f64(t.lse)
    q = t.q.float().cpu().numpy().astype(np.float64)
    for r, n, a, first in ((0, 40, 0, 130), (1, 9, 40, 0)):
        p = np.arange(first + n)
        rows = s["table"][r, p // 8].astype(np.int64) * 8 + p % 8
        c = PO.latent_rows(s["codes"][rows], s["scales"][rows])
        for i in range(n):
            seen = np.concatenate([np.arange(first), first + np.flatnonzero(see[r, i, :n])])
            if not len(seen):
                assert (out[a + i] == 0).all() and np.isneginf(lse[a + i]).all()
                continue
            x = SM * q[a + i] @ c[seen].T
            e = np.exp(x - x.max(1, keepdims=True))
            want = e / e.sum(1, keepdims=True) @ c[seen]
            dot = np.max(np.abs(q[a + i]) @ np.abs(c[seen]).T)
            assert (np.abs(out[a + i] - want) <= (2 * (64 * U * dot * SM + 2.0 ** -21) + 2.0 ** -11 + 200 * U) * np.abs(c).max() + 2.0 ** -7 * np.abs(want)).all()


def test_attention_graphs_share_a_workspace(abi):
    """Two captured steps of trees on one workspace, replayed with lengths that change, give what the 64-bit form gives."""
    rng = np.random.default_rng(15)
    s1 = attn_inputs(rng, [2100, 700], [6, 3], 64, 64, "fp4")
    s2 = attn_inputs(rng, [640, 1900], [70, 65], 64, 16, "fp8")
    a, b = Tree(abi, s1, trees(rng, [6, 3])), Tree(abi, s2, trees(rng, [70, 65]), 128)
    a.ws = b.ws = fresh_ws(abi, max(a.ws.numel(), b.ws.numel()))
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
        a.s = dict(s1, kv_len=np.array([2100 - 500 * k, 700], np.int32))
        b.q.mul_(-1)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for g in graphs:
                g.replay()
        st.synchronize()
        a.check()
        assert b.check()[0] == abi.OK


def test_attention_many_requests(abi):
    rng = np.random.default_rng(16)
    nodes = rng.integers(0, 9, 300)
    cached = rng.integers(0, 200, 300)
    s = attn_inputs(rng, cached + nodes, nodes, 8, 8, "fp4")
    assert Tree(abi, s, trees(rng, nodes)).call().check()[0] == abi.OK


def walk_inputs(rng, n_req, H, kind, longest, page, fmt):
    """Requests of very unequal numbers of nodes and entries, some without any; "few": with one of more than 256 rows (or
    very many), "tiles": of more than 512 rows on average."""
    if kind == "few":
        nodes = rng.integers(0, 4, n_req)
        nodes[n_req // 3] = 256 // H + 3
    else:
        nodes = rng.integers(0, 1024 // H + 6, n_req)
        nodes[-1] = 0
    cached = (longest * rng.random(n_req) ** 4).astype(np.int64)
    cached[n_req // 2], cached[0] = longest, 0
    nodes[n_req // 2] = max(nodes[n_req // 2], 1)
    s = attn_inputs(rng, cached + nodes, nodes, H, page, fmt, tail=1)
    return s, trees(rng, nodes)


@pytest.mark.parametrize("n_req,H,kind,longest,page,fmt,window", [
    (2, 64, "few", 1100, 16, "fp4", 0), (3, 16, "few", 5000, 64, "fp8", 0), (33, 8, "few", 1500, 8, "fp4", 0), (40, 8, "few", 1300, 8, "fp8", 1050),
    (150, 8, "few", 1100, 16, "fp4", 0), (600, 8, "few", 1200, 8, "fp4", 0), (2, 64, "tiles", 3400, 64, "fp4", 0),
    (5, 64, "tiles", 4100, 16, "fp8", 3200), (35, 32, "tiles", 3300, 16, "fp4", 0)])
def test_attention_walks(abi, n_req, H, kind, longest, page, fmt, window):
    """Several requests' items laid out by their real lengths: more of them than groups of CTAs and fewer, more requests than
    a warp and than a block look at at once."""
    rng = np.random.default_rng(n_req + H)
    s, parent = walk_inputs(rng, n_req, H, kind, longest, page, fmt)
    t = Tree(abi, s, parent, window).call()
    assert t.check()[0] == abi.OK
    first, lse = t.out.clone(), t.lse.clone()
    t.call()
    assert t.check()[0] == abi.OK and torch.equal(first, t.out) and torch.equal(lse, t.lse)


@pytest.mark.parametrize("n_req,H,kind,longest", [(40, 8, "few", 1300), (12, 64, "tiles", 3300)])
def test_attention_walks_around_bad_requests(abi, n_req, H, kind, longest):
    """Requests whose token bounds do not hold are skipped and recorded, and all others are as before."""
    rng = np.random.default_rng(18)
    s, parent = walk_inputs(rng, n_req, H, kind, longest, 16, "fp4")
    t = Tree(abi, s, parent).call()
    assert t.check()[0] == abi.OK
    out, lse = t.out.clone(), t.lse.clone()
    for place, value in ((n_req // 4, s["T"] + 9), (n_req - 2, -3)):
        bad = s["q_start"].copy()
        bad[place] = value
        t.q_start.copy_(dev(bad))
        t.out.fill_(7.0)
        t.lse.fill_(7.0)
        t.call()
        torch.cuda.synchronize()
        assert abi.csa2_status_fetch(t.ws)[0] == abi.ERR_DEVICE_BOUNDS
        abi.csa2_status_reset(t.ws)
        left = np.zeros(s["T"], bool)
        left[s["q_start"][place - 1]:s["q_start"][place + 1]] = True
        left[s["q_start"][-1]:] = True
        assert (t.out[left] == 7).all() and (t.lse[left] == 7).all()
        a, b = f64(t.out)[~left], f64(out)[~left]
        assert np.abs(a - b).max() <= 2.0 ** -6 * np.abs(b).max()
        a, b = f64(t.lse)[~left], f64(lse)[~left]
        assert np.array_equal(np.isneginf(a), np.isneginf(b)) and np.abs(a - b)[np.isfinite(b)].max() <= 2.0 ** -14


def test_attention_gives_up_and_recovers(abi):
    """Bounded waits that run out are recorded, and the next call is as if nothing had been."""
    rng = np.random.default_rng(17)
    for nodes, longest in (([5, 3], 900), ([70, 66], 900), ([70, 66], 3300)):
        s = attn_inputs(rng, np.array([longest, 400]) + nodes, nodes, 64, 16, "fp4")
        t = Tree(abi, s, trees(rng, nodes))
        t.call()
        torch.cuda.synchronize()
        want = t.out.clone()
        abi.csa2_debug_wait_limit(1)
        try:
            t.call()
            torch.cuda.synchronize()
        finally:
            abi.csa2_debug_wait_limit(0)
        assert abi.csa2_status_fetch(t.ws)[0] == abi.ERR_TIMEOUT
        abi.csa2_status_reset(t.ws)
        assert t.call().check()[0] == abi.OK and torch.equal(t.out, want)


# ------------------------------------------------------- log probabilities
class Logp:
    def __init__(self, abi, x, tokens, top, scale=1.0, gap=0, shift=0):
        """x: a CPU tensor [n][V] of bf16 or fp32; rows `gap` elements apart, the first one `shift` elements behind a 16-byte
        border, the tokens as many behind theirs."""
        self.abi, self.top, self.scale = abi, top, scale
        n, V = x.shape
        self.n, self.V, self.x64 = n, V, x.double().numpy()
        self.flat = torch.full((n * (V + gap) + 64 + shift,), float("nan"), dtype=x.dtype)
        self.flat[shift:shift + n * (V + gap)].view(n, V + gap)[:, :V] = x
        self.flat = self.flat.cuda()[shift:]
        self.stride = V + gap
        flat = np.concatenate([np.zeros(shift), np.ravel(tokens)]).astype(np.int64) if tokens is not None else None
        self.tokens = dev(flat)[shift:] if flat is not None and np.size(tokens) else None
        self.tok64 = np.asarray(tokens).reshape(n, -1) if tokens is not None else np.zeros((n, 0), np.int64)
        self.given = self.tok64.shape[1]
        f = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
        self.lp, self.lse, self.ent, self.best = f(n, self.given), f(n), f(n), f(n, top)
        self.ids = torch.full((n, top), -7, dtype=torch.int32, device="cuda")
        self.ws = fresh_ws(abi, abi.STATUS_BYTES)

    def call(self, stream=None):
        a = self.abi
        a.csa2_token_logprobs(self.flat, a.OUT_BF16 if self.flat.dtype == torch.bfloat16 else a.OUT_F32, self.stride, self.n, self.V,
                              self.scale, self.tokens, self.given, self.lp if self.given else None, self.lse, self.ent, self.top,
                              self.ids if self.top else None, self.best if self.top else None, self.ws, self.ws.numel(), stream)
        return self

    def check(self):
        """With u = 2^-24, Y = |y| weighted by the probabilities, Y2 likewise y^2 (natural logarithms): an exponent y is a
        difference, a product with a rounded constant and a product with it, off by 3 u |y| (|y| <= 4 ln 2 above its thread's
        base counts as well), the exponential by 2^-22, sums of 32 terms and over threads, warps and slices by 45 u in all
        (sums across groups keep their rests).  So S is off by dS = 3 u (Y + 3) + 2^-22 + 45 u relative, the weighted sum of y
        by 3 u (Y2 + 3 Y) + (2^-22 + 48 u) (Y + 3)."""
        torch.cuda.synchronize()
        lp, lse, ent, ids, best = TO.token_logprobs(self.x64, self.scale, self.tok64, self.top)
        with np.errstate(invalid="ignore", over="ignore"):
            y = (self.x64 - self.x64.max(1, keepdims=True)) * self.scale
            p = np.exp(y)
            p = np.where(np.isnan(p), 0, p / np.maximum(p.sum(1, keepdims=True), 1e-300))
            y = np.where(p > 0, y, 0)
        Y, Y2 = (p * np.abs(y)).sum(1), (p * y * y).sum(1)
        dS = 3 * U * (Y + 3) + 2.0 ** -22 + 45 * U
        dT = 3 * U * (Y2 + 3 * Y) + (2.0 ** -22 + 48 * U) * (Y + 3)
        some = np.isfinite(lse)
        near = lambda got, want, tol: self._near(f64(got), want, tol)  # noqa: E731
        near(self.lse, lse, 2 * U * np.abs(np.where(some, lse, 0)) + dS + 2 * U * (1 + np.log(self.V)))
        near(self.ent, ent, dS + dT + 4 * U * (np.log(self.V) + Y))
        for got, want in ((self.lp, lp), (self.best, best)):
            near(got, want, 3 * U * np.abs(np.where(np.isfinite(want), want, 0)) + (dS + 4 * U * (1 + np.log(self.V)))[:, None])
        np.testing.assert_array_equal(self.ids.cpu().numpy(), ids)
        return self.abi.csa2_status_fetch(self.ws)

    @staticmethod
    def _near(got, want, tol):
        np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
        np.testing.assert_array_equal(got[np.isinf(want)], want[np.isinf(want)])
        fine = np.isfinite(want)
        err = np.abs(got[fine] - want[fine])
        assert (err <= np.broadcast_to(tol, want.shape)[fine]).all(), (err - np.broadcast_to(tol, want.shape)[fine]).max()


def logits(rng, n, V, dtype=torch.float32, amp=2.0):
    x = amp * rng.standard_normal((n, V))
    return torch.from_numpy((x + 0.4 * x * np.abs(x)).astype(np.float32)).to(dtype)


def picks(rng, n, V, given):
    t = rng.integers(0, V, (n, given))
    if given:
        t[::3, 0] = -1
    return t


@pytest.mark.parametrize("n,V,given,top,gap", [
    (1, 1, 1, 1, 0), (3, 1, 2, 5, 7), (2, 2, 0, 2, 0), (5, 7, 1, 7, 0), (4, 63, 3, 64, 0), (9, 1000, 1, 20, 0), (7, 1001, 0, 0, 0),
    (3, 4096, 1, 1, 8), (2, 32000, 1, 5, 0), (1, 131072, 64, 64, 0), (33, 5003, 2, 20, 3), (400, 777, 1, 3, 0), (1, 100003, 1, 20, 0),
    (40, 50021, 4, 20, 13), (1, 300000, 1, 64, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logprobs(abi, n, V, given, top, gap, dtype):
    rng = np.random.default_rng(n + V)
    assert Logp(abi, logits(rng, n, V, dtype), picks(rng, n, V, given), top, gap=gap).call().check()[0] == abi.OK


@pytest.mark.parametrize("n,V,top,gap", [(700, 1000, 20, 0), (700, 3001, 24, 1), (2000, 260, 5, 0), (1900, 1, 1, 3), (1000, 5003, 25, 0),
                                         (640, 2500, 64, 4), (2500, 7, 64, 0), (930, 17001, 0, 0), (1830, 9001, 1, 0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logprobs_of_many_short_rows(abi, n, V, top, gap, dtype):
    """Blocks of fewer threads, which walk over several rows; masks of both kinds on some of them."""
    rng = np.random.default_rng(n + V)
    x = logits(rng, n, V, dtype)
    for r in range(n):
        if r % 5 < 2:
            kept = rng.random(V) < (1.0, 0.3, 0.02, 0.001)[r % 4]
            x[r][torch.from_numpy(~kept)] = -math.inf if r % 5 else torch.finfo(dtype).min
    x[2 % n] = 1.5
    x[7 % n] = torch.linspace(3.0, -3.0, V).to(dtype)
    x[8 % n, V // 2] = math.nan
    assert Logp(abi, x, picks(rng, n, V, 2), top, gap=gap).call().check()[0] == abi.OK


@pytest.mark.parametrize("dtype,shift", [(torch.float32, 1), (torch.float32, 3), (torch.bfloat16, 1), (torch.bfloat16, 6)])
@pytest.mark.parametrize("n,V,gap", [(1, 3, 0), (1, 5001, 0), (7, 8192, 0), (5, 40001, 2)])
def test_logprobs_of_rows_from_any_element(abi, dtype, shift, n, V, gap):
    rng = np.random.default_rng(n + V)
    Logp(abi, logits(rng, n, V, dtype), picks(rng, n, V, 1), 3, gap=gap, shift=shift).call().check()


@pytest.mark.parametrize("scale", [2.0 ** -20, 0.1, 1.25, 37.0, 2.0 ** 20])
def test_logprobs_scales(abi, scale):
    rng = np.random.default_rng(3)
    Logp(abi, logits(rng, 6, 9001), picks(rng, 6, 9001, 2), 9, scale).call().check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [500, 40000])
def test_logprobs_masks_and_ties(abi, dtype, V):
    """Rows of -inf, of the type's lowest value, of few others beside them; all equal; NaN and infinities; zeros of both signs;
    values in steps, so that the place of the last alternative is one of many equal ones."""
    rng = np.random.default_rng(4)
    x = logits(rng, 16, V, dtype)
    low = torch.finfo(dtype).min
    x[0], x[1], x[2] = -math.inf, low, 3.5
    x[3, 5:] = -math.inf
    x[4, 30:] = low
    x[5], x[6] = -math.inf, low
    x[5, V - 1], x[6, V // 2] = 1.0, 1.0
    x[7, V // 3] = math.nan
    x[8, V // 3] = math.inf
    x[9] = torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0).to(dtype)
    x[10] = torch.from_numpy(rng.integers(-3, 4, V).astype(np.float32)).to(dtype)
    x[11] = low
    x[11, ::3] = -math.inf
    x[12] = torch.arange(V).float().to(dtype) * 0.01
    x[13] = -x[12]
    x[14] = 2e4
    x[14, 7::11] = 2e4 + 256
    x[15, :V // 2] = -1e4
    Logp(abi, x, picks(rng, 16, V, 2), 20).call().check()
    Logp(abi, x, None, 64).call().check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [9, 320])
def test_logprobs_of_few_values_above_a_mask(abi, dtype, n):
    """Masks of the lowest value or -inf that leave less than there are alternatives, or hardly more; the lowest value
    itself among -inf; rows that fall and rise, so that neighbours hold the largest."""
    rng = np.random.default_rng(8)
    V = 30011
    x = logits(rng, n, V, dtype)
    low = torch.finfo(dtype).min
    for r in range(n):
        kept = rng.choice(V, (0, 3, 19, 20, 21, 33, 64, 200, 1500)[r % 9], replace=False)
        y = torch.full((V,), low if r % 2 else -math.inf, dtype=dtype)
        y[kept] = x[r, kept]
        x[r] = y
    x[0, 5:5 * 7:5] = low
    x[4 % n] = torch.linspace(9.0, -9.0, V).to(dtype)
    x[7 % n] = torch.linspace(-9.0, 9.0, V).to(dtype)
    Logp(abi, x, picks(rng, n, V, 1), 20).call().check()
    Logp(abi, x[:9], None, 64).call().check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logprobs_of_alternatives_in_few_places(abi, dtype):
    """The large values all lie in what a few threads see: more of them than are ranked at once."""
    E = 4 if dtype == torch.float32 else 8
    V = 512 * E * 4 * 30
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.uniform(-1, 0, (2, V)).astype(np.float32))
    at = (np.arange(V) // E % 512) < 7
    x[0, at] = torch.from_numpy(rng.uniform(1, 2, at.sum()).astype(np.float32))
    x[1, at] = 1.0
    n = 400  # (many rows: one block each)
    got = Logp(abi, x.to(dtype)[np.arange(n) % 2], None, 20)
    got.call()
    torch.cuda.synchronize()
    one = Logp(abi, x.to(dtype), None, 20).call()
    one.check()
    assert torch.equal(got.ids, one.ids[torch.arange(n) % 2]) and (got.best - one.best[torch.arange(n) % 2]).abs().max() < 1e-5


def test_logprobs_peaked_rows_keep_their_tail(abi):
    """One token of nearly all probability before, behind and among a long tail."""
    rng = np.random.default_rng(6)
    x = torch.from_numpy(rng.normal(0, 0.1, (4, 60000)).astype(np.float32))
    for r, (at, v) in enumerate(((0, 18.0), (59999, 18.0), (30000, 24.0), (77, 11.5))):
        x[r, at] = v
    Logp(abi, x, picks(rng, 4, 60000, 1), 3).call().check()


def test_logprobs_tokens_outside_are_recorded(abi):
    rng = np.random.default_rng(7)
    for bad in (500, -2, 1 << 40):
        tok = picks(rng, 3, 500, 2)
        tok[1, 1] = bad
        st = Logp(abi, logits(rng, 3, 500), tok, 2).call().check()
        assert st[0] == abi.ERR_DEVICE_BOUNDS and st[2] == 1


@pytest.mark.parametrize("dtype,gap,shift", [(torch.float32, 0, 0), (torch.float32, 1, 3), (torch.bfloat16, 3, 7)])
def test_logprobs_of_the_largest_vocabulary(abi, dtype, gap, shift):
    rng = np.random.default_rng(9)
    V = 1 << 21
    x = logits(rng, 2, V, dtype)
    x[0, V - 1], x[1, 0] = 40.0, 40.0
    Logp(abi, x, np.array([[V - 1], [0]]), 2, gap=gap, shift=shift).call().check()


def test_logprobs_beyond_two_gigabytes(abi):
    """Rows behind 2^31 bytes and elements, and the largest vocabulary."""
    V = 1 << 21
    x = torch.zeros(1100, V, dtype=torch.bfloat16, device="cuda")
    x[1099, V - 3] = 20.0
    x[1099, 9] = 12.0
    ids, best = torch.zeros(1100, 2, dtype=torch.int32, device="cuda"), torch.zeros(1100, 2, device="cuda")
    lse, ws = torch.zeros(1100, device="cuda"), fresh_ws(abi, abi.STATUS_BYTES)
    abi.csa2_token_logprobs(x, abi.OUT_BF16, V, 1100, V, 1.0, None, 0, None, lse, None, 2, ids, best, ws, ws.numel())
    torch.cuda.synchronize()
    assert ids[1099].tolist() == [V - 3, 9] and (ids[:1099] == torch.tensor([0, 1], device="cuda")).all()
    want = math.log(math.exp(20) + math.exp(12) + V - 2)
    assert abs(float(lse[1099]) - want) < 1e-5 and (lse[:1099] - math.log(V)).abs().max() < 1e-5
    assert abs(float(best[1099, 0]) - (20 - want)) < 1e-5


def test_logprobs_rows_do_not_depend_on_the_others(abi):
    """A row cut into slices for a cluster and the same row as one block's: the alternatives are the same, the sums within the
    bound of both."""
    rng = np.random.default_rng(8)
    x = logits(rng, 1, 131072, torch.bfloat16)
    one = Logp(abi, x, [[5]], 20).call()
    many = Logp(abi, x.expand(700, -1), [[5]] * 700, 20).call()
    one.check()
    assert torch.equal(many.ids, one.ids.expand(700, -1)) and (many.lse == many.lse[0]).all()
    assert (many.lse[0] - one.lse[0]).abs() < 4e-6 and (many.best - one.best).abs().max() < 8e-6


# ------------------------------------------------------------------ commit
class Commit:
    def __init__(self, abi, rng, cached, nodes, page, fmt, shape="random", vocab=3, spare=5, extra=2, tail=2):
        self.abi, self.page, self.fmt = abi, page, fmt
        cached, nodes = np.asarray(cached, np.int32), np.asarray(nodes, np.int32)
        self.kv_len, self.q_start = cached + nodes, starts(nodes)
        pages = -(-self.kv_len // page)
        self.n_pages, self.max_pages = int(pages.sum()) + spare, max(1, int(pages.max(initial=0))) + extra
        ids = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((len(nodes), self.max_pages), -3, np.int32)
        at = 0
        for r, n in enumerate(pages):
            self.table[r, :n] = ids[at:at + n]
            at += n
        self.free = np.full(self.n_pages, -9, np.int32)
        self.n_free = 2 if spare >= 2 else 0
        self.free[:self.n_free] = ids[at:at + self.n_free]
        self.T = int(self.q_start[-1])
        self.tail = tail
        self.parent = np.concatenate([trees(rng, nodes, shape), np.full(tail, 4, np.int32)])
        self.token, self.choice = rng.integers(0, vocab, self.T + tail), rng.integers(0, vocab, self.T + tail)
        rows = self.n_pages * page
        self.planes = [rng.integers(0, 256, (rows, w), dtype=np.uint8) for w in ((256, 32) if fmt == "fp4" else (512,))]
        self.max_q = int(nodes.max(initial=0))
        self.cached0 = rng.integers(0, 9, len(nodes)).astype(np.int32)

    def upload(self):
        self.d = {k: dev(np.asarray(getattr(self, k), t)) for k, t in (("parent", np.int32), ("token", np.int64), ("choice", np.int64),
                  ("q_start", np.int32), ("kv_len", np.int32), ("table", np.int32), ("free", np.int32))}
        self.dp = [dev(p) for p in self.planes]
        self.nf = torch.tensor([self.n_free], dtype=torch.int32, device="cuda")
        T, R = self.T + self.tail, len(self.kv_len)
        self.cached = dev(self.cached0)
        self.path = torch.full((T,), -7, dtype=torch.int32, device="cuda")
        self.accepted = torch.full((R,), -7, dtype=torch.int32, device="cuda")
        self.next = torch.full((R,), -7, dtype=torch.int64, device="cuda")
        self.ws = fresh_ws(self.abi, self.abi.STATUS_BYTES)
        return self

    def call(self, stream=None, move=True, max_q=None):
        d, a = self.d, self.abi
        a.csa2_tree_commit(d["parent"], d["token"], d["choice"], d["q_start"], d["kv_len"], len(self.kv_len), self.T + self.tail,
                           self.max_q if max_q is None else max_q, a.FMT_FP4 if self.fmt == "fp4" else a.FMT_FP8,
                           self.dp[0] if move else None, self.dp[1] if move and self.fmt == "fp4" else None, self.planes[0].shape[0],
                           d["table"], self.max_pages, self.page, d["free"], self.n_pages, self.nf, self.nf, self.cached, self.path,
                           self.accepted, self.next, self.ws, self.ws.numel(), stream)
        return self

    def check(self, move=True):
        torch.cuda.synchronize()
        path, acc, nxt, cached, free, n_free, planes = TO.tree_commit(
            self.parent, self.token, self.choice, self.q_start, self.kv_len, self.page, self.planes if move else [], self.table, self.free,
            self.n_free, self.n_pages, self.cached0, self.T)
        got = self.path.cpu().numpy()
        np.testing.assert_array_equal(got[:self.T], path)
        assert (got[self.T:] == -7).all()
        for g, w in ((self.accepted, acc), (self.next, nxt), (self.cached, cached), (self.d["free"], free)):
            np.testing.assert_array_equal(g.cpu().numpy(), w)
        assert int(self.nf.item()) == n_free
        for g, w in zip(self.dp, planes if move else self.planes):
            np.testing.assert_array_equal(g.cpu().numpy(), w)
        np.testing.assert_array_equal(self.d["table"].cpu().numpy(), self.table)
        return self.abi.csa2_status_fetch(self.ws)


@pytest.mark.parametrize("cached,nodes,page,shape", [
    ([0], [1], 8, "chain"), ([7, 0, 16, 15], [9, 1, 3, 0], 8, "random"), ([100, 3], [64, 1], 16, "random"), ([30, 31, 32, 33], [20, 20, 20, 20], 8, "star"),
    ([5], [1024], 8, "random"), ([600], [700], 200, "chain"), ([9, 50], [40, 33], 64, "roots"), ([0, 0], [0, 0], 8, "chain")])
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("vocab", [1, 3])
def test_commit(abi, cached, nodes, page, shape, fmt, vocab):
    """With one token everything is accepted that can be (of a chain all of it, nothing moves)."""
    c = Commit(abi, np.random.default_rng(len(nodes) + page + vocab), cached, nodes, page, fmt, shape, vocab).upload()
    assert c.call().check()[0] == abi.OK


def test_commit_long_paths_that_move(abi):
    """Paths of a few hundred nodes with a sibling before each: rows move by growing distances, over more than one batch,
    into rows that were sources before."""
    c = Commit(abi, np.random.default_rng(3), [13, 200], [801, 401], 8, "fp4")
    for a, n in ((0, 801), (801, 400)):
        for i in range(1, n):
            c.parent[a + i] = 0 if i < 3 else (i - 1) // 2 * 2  # node 2k + 2 continues 2k; 2k + 1 is its sibling
    c.token[:], c.choice[:] = 5, 5
    c.token[1::2] = 6
    c.parent[2] = 0
    c.token[801:1202] = 5
    c.token[802:1202:2] = 6
    assert c.upload().call().check()[0] == abi.OK
    assert int(c.accepted[0]) == 401


def test_commit_many_requests(abi):
    rng = np.random.default_rng(4)
    nodes = rng.integers(0, 12, 500)
    c = Commit(abi, rng, rng.integers(0, 60, 500), nodes, 8, "fp8", vocab=2).upload()
    assert c.call().check()[0] == abi.OK


def test_commit_without_rows_and_with_another_bound(abi):
    c = Commit(abi, np.random.default_rng(5), [20, 9], [30, 7], 8, "fp4").upload()
    assert c.call(move=False, max_q=900).check(move=False)[0] == abi.OK


def test_commit_records_what_is_bad(abi):
    rng = np.random.default_rng(6)
    # no first node of parent -1: nothing accepted, all the step's pages go back
    c = Commit(abi, rng, [20, 9], [30, 7], 8, "fp4", vocab=1)
    c.parent[0] = 0
    c.upload().call()
    torch.cuda.synchronize()
    assert c.accepted.tolist()[0] == 0 and c.cached.tolist()[0] == 20 and c.next.tolist()[0] == -1 and c.accepted.tolist()[1] > 0
    assert abi.csa2_status_fetch(c.ws)[0] == abi.ERR_DEVICE_BOUNDS
    # bad lengths and token bounds: the request keeps nothing, its length stays
    for what in ("short", "long", "bound", "order"):
        c = Commit(abi, rng, [20, 9, 4], [30, 7, 3], 8, "fp8", vocab=1)
        max_q = c.max_q
        if what == "short":
            c.kv_len[1] = 6
        elif what == "long":
            c.kv_len[1] = c.max_pages * 8 + 1
        elif what == "bound":
            max_q = 7
        else:
            c.q_start[2] = 60
        c.upload().call(max_q=max_q)
        torch.cuda.synchronize()
        bad = 0 if what == "bound" else 1
        assert int(c.accepted[bad]) == 0 and int(c.next[bad]) == -1 and int(c.cached[bad]) == int(c.cached0[bad])
        good = 1 - bad
        if what != "order":
            assert int(c.accepted[good]) > 0 and int(c.accepted[2]) > 0
        assert abi.csa2_status_fetch(c.ws)[0] == abi.ERR_DEVICE_BOUNDS
    # pages outside the cache: not moved, not given back
    c = Commit(abi, rng, [20], [30], 8, "fp8", vocab=3)
    c.choice[:] = 77
    c.table[0, 5] = c.n_pages
    c.upload().call()
    torch.cuda.synchronize()
    assert int(c.nf.item()) == c.n_free + 3 and c.d["free"].cpu().numpy()[c.n_free:c.n_free + 3].tolist() == c.table[0, [6, 4, 3]].tolist()
    assert abi.csa2_status_fetch(c.ws)[0] == abi.ERR_DEVICE_BOUNDS
    # a free list without room
    c = Commit(abi, rng, [20], [30], 8, "fp8", vocab=3)
    c.choice[:] = 77
    c.n_free = c.n_pages - 1
    c.upload().call()
    torch.cuda.synchronize()
    assert int(c.nf.item()) == c.n_free and (c.d["free"].cpu().numpy() == c.free).all()
    assert abi.csa2_status_fetch(c.ws)[0] == abi.ERR_DEVICE_BOUNDS


def test_commit_undoes_the_plan(abi):
    """What the plan took and the commit gives back stands on the free list as before."""
    rng = np.random.default_rng(7)
    n_pages, page = 40, 8
    cached, added = np.array([5, 16, 0], np.int32), np.array([30, 9, 17], np.int32)
    table = np.full((3, 8), -1, np.int32)
    ids = rng.permutation(n_pages).astype(np.int32)
    table[0, 0], table[1, :2] = ids[0], ids[1:3]
    free = np.zeros(n_pages, np.int32)
    free[:37] = ids[3:]
    t, nf, fr = dev(table), dev(np.array([37], np.int32)), dev(free)
    qs, kl = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    sl, po, ws = torch.zeros(56, dtype=torch.int64, device="cuda"), torch.zeros(56, dtype=torch.int64, device="cuda"), fresh_ws(abi, 256)
    c_in = dev(cached)
    abi.csa2_page_plan(c_in, dev(added), 3, page, t, 8, fr, n_pages, nf, nf, qs, kl, sl, po, 56, ws, 256)
    parent = np.concatenate([np.arange(-1, n - 1) for n in added]).astype(np.int32)
    i64 = lambda v: torch.full((56,), v, dtype=torch.int64, device="cuda")  # noqa: E731
    path, acc, nxt = torch.zeros(56, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    abi.csa2_tree_commit(dev(parent), i64(1), i64(2), qs, kl, 3, 56, 30, abi.FMT_FP8, None, None, 0, t, 8, page, fr, n_pages, nf, nf, c_in, path,
                         acc, nxt, ws, 256)
    torch.cuda.synchronize()
    assert acc.tolist() == [1, 1, 1] and c_in.tolist() == [6, 17, 1] and int(nf.item()) == 35
    # requests 1 and 2 keep one new page each (entries 17 and 1); every other one stands where it stood
    kept = {int(t[1, 2]), int(t[2, 0])}
    assert [int(x) for x in free[:37] if int(x) not in kept] == fr.cpu().numpy()[:35].tolist()
    assert abi.csa2_status_fetch(ws)[0] == abi.OK


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_rows_behind_four_gigabytes(abi, fmt):
    """Latents go to, are attended to in and move within pages whose bytes lie beyond 32 bits."""
    page, width = 16, 256 if fmt == "fp4" else 512
    n_pages = (9 << 29) // (width * page)
    n_rows = n_pages * page
    rng = np.random.default_rng(19)
    n, H = 40, 8
    small = Heads(abi, rng, n, H, fmt, turn=False)
    codes = torch.empty((n_rows, width), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n_rows, 32), dtype=torch.uint8, device="cuda") if fmt == "fp4" else None
    table = np.array([[n_pages - 1, n_pages // 2, n_pages - 3]], np.int32)
    p = np.arange(n)
    rows = dev(table[0, p // page].astype(np.int64) * page + p % page)
    f = abi.FMT_FP4 if fmt == "fp4" else abi.FMT_FP8
    abi.csa2_head_norm_rope(None, 0, 0, None, None, small.lat, small.l_stride, small.lw, n, 1e-6, None, None, 0, f, rows, n_rows, codes, scales,
                            small.ws, small.ws.numel())
    want_c, want_s = torch.zeros((n, width), dtype=torch.uint8, device="cuda"), torch.zeros((n, 32), dtype=torch.uint8, device="cuda")
    abi.csa2_head_norm_rope(None, 0, 0, None, None, small.lat, small.l_stride, small.lw, n, 1e-6, None, None, 0, f, None, n, want_c,
                            want_s if fmt == "fp4" else None, small.ws, small.ws.numel())
    assert torch.equal(codes[rows], want_c) and (scales is None or torch.equal(scales[rows], want_s))
    # 24 nodes on 16 entries, as in a cache of three pages
    parent = trees(rng, [24])
    s = dict(q=bf16(rng.standard_normal((24, H, D))), q_start=starts([24]), kv_len=np.array([n], np.int32), codes=np.zeros((48, width), np.uint8),
             scales=np.zeros((48, 32), np.uint8) if fmt == "fp4" else None, table=np.array([[0, 1, 2]], np.int32), page=page, fmt=fmt, T=24, H=H,
             max_q=24, max_kv=n)
    s["codes"][:n] = want_c.cpu().numpy()
    if fmt == "fp4":
        s["scales"][:n] = want_s.cpu().numpy()
    t = Tree(abi, s, parent).call()
    assert t.check()[0] == abi.OK
    near = t.out.clone()
    t.codes, t.scales, t.table = codes, scales, dev(table)
    t.call()
    torch.cuda.synchronize()
    assert torch.equal(near, t.out)
    tok, i32 = torch.zeros(24, dtype=torch.int64, device="cuda"), lambda v, m: torch.full((m,), v, dtype=torch.int32, device="cuda")  # noqa: E731
    free, nf, path, acc, cached, nxt = i32(0, n_pages), i32(0, 1), i32(0, 24), i32(0, 1), i32(0, 1), torch.zeros(1, dtype=torch.int64, device="cuda")
    abi.csa2_tree_commit(t.par, tok, tok, t.q_start, t.kv_len, 1, 24, 24, f, codes, scales, n_rows, t.table, 3, page, free, n_pages, nf, nf, cached,
                         path, acc, nxt, t.ws, t.ws.numel())
    torch.cuda.synchronize()
    k = int(acc[0])
    assert k > 1 and int(cached[0]) == 16 + k
    src = 16 + path[:k].long()
    assert (src != torch.arange(16, 16 + k, device="cuda")).any()
    assert torch.equal(codes[rows[16:16 + k]], want_c[src]) and (scales is None or torch.equal(scales[rows[16:16 + k]], want_s[src]))
    assert torch.equal(codes[rows[:16]], want_c[:16]) and abi.csa2_status_fetch(t.ws)[0] == abi.OK


@pytest.mark.parametrize("cached,nodes", [([30, 9], [5, 3]), ([1200, 300, 40], [8, 2, 5]), ([700], [90]), ([3300, 100], [70, 66])])
def test_attention_without_lse(abi, cached, nodes):
    s = attn_inputs(np.random.default_rng(20), np.asarray(cached) + nodes, nodes, 64, 16, "fp4")
    t = Tree(abi, s, trees(np.random.default_rng(1), nodes)).call()
    assert t.check()[0] == abi.OK
    out, t.lse = t.out.clone(), None
    t.out.fill_(7.0)
    t.call()
    torch.cuda.synchronize()
    assert torch.equal(out, t.out)


# --------------------------------------------------------- steps together
def tree_layer(abi, fmt, window, norms, seed=0, theta=10000.0):
    from csa2_sparse_attention_gb300 import paged
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    cache = paged.PagedLatents(3, 96, 60, 16, 20, heads=8, fmt=fmt, window=window, rope_theta=theta)
    hidden = 256
    kw = dict(q_norm=(1 + 0.2 * r(D)).to(torch.bfloat16).cuda(), latent_norm=(1 + 0.2 * r(D)).to(torch.bfloat16).cuda()) if norms else {}
    layer = paged.PagedLayer(cache, hidden, (1 + 0.1 * r(hidden)).to(torch.bfloat16).cuda(),
                             (r(8 * D, hidden) / 16).to(torch.bfloat16).cuda(), (r(D, hidden) / 16).to(torch.bfloat16).cuda(), turn=True, **kw)
    return paged, g, cache, layer


@pytest.mark.parametrize("fmt,window,norms", [("fp4", 0, True), ("fp4", 40, False), ("fp8", 0, True), ("fp8", 24, True)])
def test_steps_of_trees(abi, fmt, window, norms):
    """Prompts, then steps of drafted trees: every stage against its 64-bit form on what the stage before left, and over all
    steps the cache's entries against the accepted tokens' latents, turned by their places."""
    paged, g, cache, layer = tree_layer(abi, abi.FMT_FP4 if fmt == "fp4" else abi.FMT_FP8, window, norms)
    rng = np.random.default_rng(1)
    hidden, H, page, V = 256, 8, 16, 50
    pick = paged.TokenLogprobs(96, top=3)
    entries = [[], [], []]  # per request the latents that its entries have to be, before rounding
    cached = np.zeros(3, np.int32)
    for step in range(6):
        nodes = np.array([[40, 9, 17], [12, 0, 33], [7, 20, 1], [30, 30, 30], [1, 1, 1], [5, 64, 9]][step], np.int32)
        n = int(nodes.sum())
        parent = trees(rng, nodes, "chain" if step == 0 else "random")
        token = rng.integers(0, 4, n)
        par, tok = dev(parent), dev(token.astype(np.int64))
        cache.added.copy_(torch.from_numpy(nodes))
        layer.residual.zero_()
        x = torch.randn(n, hidden, generator=g).to(torch.bfloat16).cuda()
        free0, n_free0, cached0 = cache.free.cpu().numpy(), int(cache.n_free.item()), cached.copy()
        table0 = cache.table.cpu().numpy()
        out, lse = layer.step(x, n, int(nodes.max()), int((cached + nodes).max()), parent=par)
        torch.cuda.synchronize()
        want = PO.page_plan(cached, nodes, page, table0, free0, n_free0, cache.n_pages, cache.max_tokens)
        table, q_start, kv_len = want[0], want[1], want[2]
        np.testing.assert_array_equal(cache.table.cpu().numpy(), table)
        words = -(-int(nodes.max()) // 32)
        pos, mask = TO.tree_plan(parent, q_start, kv_len, window, words, np.zeros(n, np.int64), np.zeros((n, words), np.int32))
        np.testing.assert_array_equal(cache.pos.cpu().numpy()[:n], pos)
        np.testing.assert_array_equal(cache.mask.cpu().numpy()[:n * words].reshape(n, words), mask)
        # latents and queries as the layer made them
        lat = f64(layer.latents[:n])
        z = TO.head_norm(lat, f64(layer.latent_norm) if norms else None, layer.eps)
        z = TO.turned(z, pos) if cache.rope is not None else z
        cc, cs = cache.codes.cpu().numpy(), None if cache.scales is None else cache.scales.cpu().numpy()
        slots = want[3][:n]
        if fmt == "fp4":
            c, s = O.quantize_fp4(z)
            np.testing.assert_array_equal(cs[slots], s)
            np.testing.assert_array_equal(O.e2m1_decode(O.unpack_codes(cc[slots])), O.e2m1_decode(c))
        else:
            np.testing.assert_array_equal(O.e4m3_decode(cc[slots]), O.e4m3_decode(O.e4m3_encode(z)))
        s = dict(q=layer.q[:n].cpu(), q_start=q_start, kv_len=kv_len, codes=cc, scales=cs, table=table, page=page, T=n, H=H,
                 max_kv=int(kv_len.max()), max_q=int(nodes.max()))
        t = Tree.__new__(Tree)
        t.abi, t.s, t.window, t.parent, t.q, t.out, t.lse, t.ws = abi, s, window, parent, layer.q[:n], out, lse, cache.ws_attn
        assert t.check()[0] == abi.OK
        # the model's choices, from logits that like some of the drafted tokens
        lg = torch.randn(n, V, generator=g).cuda()
        lg[:, :4] += 3
        choice = pick(lg)[3][:, 0].long().contiguous()
        np.testing.assert_array_equal(choice.cpu().numpy(), lg.argmax(1).cpu().numpy())
        path, acc, nxt = cache.commit(par, tok, choice, n, int(nodes.max()))
        torch.cuda.synchronize()
        wp, wa, wn, wc, wf, wnf, _ = TO.tree_commit(parent, token, choice.cpu().numpy(), q_start, kv_len, page, [], table, free0.copy(),
                                                    want[5], cache.n_pages, cached0, n)
        np.testing.assert_array_equal(path.cpu().numpy(), wp)
        for a, b in ((acc, wa), (nxt, wn), (cache.cached, wc), (cache.free, wf), (cache.n_free, [wnf])):
            np.testing.assert_array_equal(a.cpu().numpy(), b)
        cached = wc.astype(np.int32)
        for r in range(3):
            entries[r] += [z[q_start[r] + j] for j in wp[q_start[r]:q_start[r] + wa[r]]]
            p = np.arange(len(entries[r]))
            assert len(p) == cached[r]
            if not len(p):
                continue
            rows = table[r, p // page].astype(np.int64) * page + p % page
            got = PO.latent_rows(cache.codes.cpu().numpy()[rows], None if cs is None else cache.scales.cpu().numpy()[rows])
            e = np.stack(entries[r])
            w = O.dequantize_fp4(*O.quantize_fp4(e)) if fmt == "fp4" else O.e4m3_decode(O.e4m3_encode(e))
            np.testing.assert_array_equal(got, w)
    for name, st in cache.status().items():
        assert st[0] == abi.OK, (name, st)
    assert pick.status()[0] == abi.OK
    # every page is either a request's or free
    held = [int(i) for r in range(3) for i in cache.table.cpu().numpy()[r, :-(-int(cached[r]) // page)]]
    left = cache.free.cpu().numpy()[:int(cache.n_free.item())].tolist()
    assert sorted(held + left) == list(range(cache.n_pages))


def test_captured_tree_step_is_the_eager_one(abi):
    """Plan, tree, heads, attention, choices and commit in one graph, replayed over growing lengths on another stream, against
    eager steps of a second cache: the same bytes."""
    got = []
    for captured in (False, True):
        paged, g, cache, layer = tree_layer(abi, abi.FMT_FP4, 0, True, seed=5)
        pick = paged.TokenLogprobs(30, top=1)
        nodes = np.array([10, 8, 12])
        n = 30
        par = dev(trees(np.random.default_rng(2), nodes))
        tok = dev(np.random.default_rng(3).integers(0, 3, n))
        cache.added.copy_(torch.from_numpy(nodes.astype(np.int32)))
        x, lg = torch.zeros(n, 256, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, 40, device="cuda")
        seen = []

        def step(stream):
            out, lse = layer.step(x, n, 12, 200, stream=stream, parent=par)
            with torch.cuda.stream(stream):
                choice = pick(lg, stream=stream)[3][:, 0].long()
            path, acc, nxt = cache.commit(par, tok, choice, n, 12, stream=stream)
            return out, lse, path, acc, nxt

        st = torch.cuda.Stream()
        graph, kept = None, None
        for k in range(4):
            torch.cuda.synchronize()
            x.copy_(torch.randn(n, 256, generator=g).to(torch.bfloat16))
            lg.copy_(torch.randn(n, 40, generator=g))
            lg[:, :3] += 2
            layer.residual.zero_()
            torch.cuda.synchronize()
            if captured and k == 1:
                state = [t.clone() for t in (cache.cached, cache.n_free, cache.free, cache.table, cache.codes, cache.scales)]
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=st):
                    kept = step(torch.cuda.current_stream())
                for t, v in zip((cache.cached, cache.n_free, cache.free, cache.table, cache.codes, cache.scales), state):
                    t.copy_(v)
                torch.cuda.synchronize()
            if graph is not None:
                with torch.cuda.stream(st):
                    graph.replay()
                res = kept
            else:
                res = step(st)
            torch.cuda.synchronize()
            seen.append([t.cpu().clone() for t in res] + [cache.codes.cpu().clone(), cache.cached.cpu().clone(), cache.free.cpu().clone()])
        got.append(seen)
        assert all(v[0] == abi.OK for v in cache.status().values())
    for a, b in zip(*got):
        for u, v in zip(a, b):
            assert torch.equal(u, v)


def test_refused_tree_step_leaves_the_cache_as_it_was(abi):
    """A plan without pages: nothing is appended or accepted, lengths and pages stay, and the next step runs."""
    paged, g, cache, layer = tree_layer(abi, abi.FMT_FP4, 0, True)
    par, tok = dev(trees(None, [30, 30, 30], "chain")), torch.zeros(90, dtype=torch.int64, device="cuda")
    x = torch.randn(90, 256, generator=g).to(torch.bfloat16).cuda()

    def step():
        layer.residual.zero_()
        layer.step(x, 90, 30, 320, parent=par)
        cache.commit(par, tok, tok, 90, 30)
        torch.cuda.synchronize()

    cache.added.copy_(torch.tensor([30, 30, 30], dtype=torch.int32))
    step()
    assert cache.cached.tolist() == [30, 30, 30]
    before = [t.clone() for t in (cache.cached, cache.n_free, cache.free, cache.codes, cache.table)]
    keep = int(cache.n_free.item())
    cache.n_free.fill_(1)
    step()
    assert cache.status()["plan"][0] == abi.ERR_DEVICE_BOUNDS and cache.accepted.tolist() == [0, 0, 0] and int(cache.n_free.item()) == 1
    cache.n_free.fill_(keep)
    for a, b in zip((cache.cached, cache.n_free, cache.free, cache.codes, cache.table), before):
        assert torch.equal(a, b)
    step()
    assert cache.cached.tolist() == [60, 60, 60]


def test_padded_tree_step(abi):
    """Tokens behind the planned ones: their rows of outputs and queries stay as they were, nothing is recorded."""
    paged, g, cache, layer = tree_layer(abi, abi.FMT_FP4, 0, True)
    nodes = [5, 0, 7]
    par = dev(np.concatenate([trees(np.random.default_rng(0), nodes), np.full(8, 3, np.int32)]))
    tok = torch.zeros(20, dtype=torch.int64, device="cuda")
    cache.added.copy_(torch.tensor(nodes, dtype=torch.int32))
    cache.out.fill_(7)
    cache.lse.fill_(7)
    x = torch.randn(20, 256, generator=g).to(torch.bfloat16).cuda()
    out, lse = layer.step(x, 20, 7, 50, parent=par)
    path, acc, nxt = cache.commit(par, tok, tok, 20, 7)
    torch.cuda.synchronize()
    assert (out[12:] == 7).all() and (lse[12:] == 7).all() and (out[:12] != 7).any() and (cache.pos[12:20] == -1).all()
    assert acc.tolist()[1] == 0 and cache.cached.tolist()[1] == 0
    for name, st in cache.status().items():
        assert st[0] == abi.OK, (name, st)


def test_layer_with_turned_queries_goes_by_distances(abi):
    """The layer's own rotation: the same prompt at other places gives the same outputs (within roundings of FP4 keys: the
    logits are compared by their log-sum-exp over a cache that does not round, E4M3 without rotation, and by queries)."""
    paged, g, cache, layer = tree_layer(abi, abi.FMT_FP4, 0, True)
    cache.added.copy_(torch.tensor([20, 20, 0], dtype=torch.int32))
    x = torch.randn(20, 256, generator=g).to(torch.bfloat16)
    layer.step(torch.cat((x, x)).cuda(), 40, 20, 20)
    torch.cuda.synchronize()
    assert torch.equal(layer.q[:20], layer.q[20:40])
    base = f64(layer.q[:20])
    w = f64(layer.q_norm)
    # undoing the rotation by the positions gives rows of the weights' norm
    back = TO.turned(base, -np.arange(20))
    rms = np.sqrt(((back / w) ** 2).mean(-1))
    assert np.abs(rms - 1).max() < 2.0 ** -7


def test_one_layer_turns_once(abi):
    """A layer that turns its queries takes no function for it; without norms or turn nothing changes."""
    paged, g, cache, layer = tree_layer(abi, abi.FMT_FP4, 0, True)
    x = torch.zeros(3, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="turns its queries itself"):
        layer.step(x, 3, 1, 20, rotate=lambda q, p: None)


def test_tree_calls_on_two_streams(abi):
    """Calls of two caches at once on two streams, each with workspaces of its own."""
    rng = np.random.default_rng(20)
    s = [attn_inputs(rng, np.array([900, 300]) + n, n, 64, 16, "fp4") for n in ([12, 3], [66, 70])]
    t = [Tree(abi, x, trees(rng, np.diff(x["q_start"]))) for x in s]
    p = [Logp(abi, logits(rng, 9, 30011), picks(rng, 9, 30011, 1), 7) for _ in range(2)]
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(2):
            t[i].call(st[i])
            p[i].call(st[i])
    for i in range(2):
        assert t[i].check()[0] == abi.OK and p[i].check()[0] == abi.OK
