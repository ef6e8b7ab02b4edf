"""Refusals of the paged-step calls: every bad argument returns before any
launch (the pointers are never valid), and empty calls do nothing.  The
64-bit forms are pinned by hand-worked values."""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO


@pytest.fixture(scope="module")
def abi():
    from csa2_sparse_attention_gb300 import build
    build.build()
    from csa2_sparse_attention_gb300 import abi as A
    return A


F = 1 << 20  # never dereferenced


def args(defaults, **kw):
    d = dict(defaults)
    d.update(kw)
    return [d[k] for k in defaults]


PLAN = dict(cached=F, added=F + 64, n_req=4, page=16, table=F, max_pages=8, free=F, n_pages=32, n_free=F, n_free_out=F,
            q_start=F, kv_len=F + 128, slots=F, pos=F, max_new=10, ws=F, ws_bytes=256, stream=None)
ATTN = dict(q=F, n_tokens=4, heads=64, q_start=F, kv_len=F, n_req=2, max_q=2, max_kv=100, fmt=0, codes=F, scales=F, n_rows=128,
            table=F, max_pages=8, page=16, window=0, sm_scale=0.04, out=F, lse=F, ws=F, ws_bytes=1 << 40, stream=None)
NORM = dict(x=F, x_stride=512, residual=F, residual_out=F, weight=F, n=4, dim=512, eps=1e-6, group=0, codes=F, scales=F, y=None,
            stream=None)
MATVEC = dict(x=F, fmt=0, x_scales=None, x_stride=256, n=2, k=256, codes=F, scales=F, n_out=8, alpha=1.0, out=F, out_dtype=0, ws=F,
              ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(page=0), "U"), (dict(page=12), "U"), (dict(page=65544), "U"), (dict(n_req=-1), "I"), (dict(cached=None), "I"),
    (dict(cached=F + 4), "I"), (dict(kv_len=F), "I"), (dict(kv_len=F + 64), "I"), (dict(table=None), "I"), (dict(free=None), "I"),
    (dict(n_free=None), "I"), (dict(n_free_out=None), "I"), (dict(q_start=None), "I"), (dict(slots=None), "I"),
    (dict(pos=F + 8), "I"), (dict(max_new=-1), "I"), (dict(max_new=1 << 31), "I"), (dict(max_pages=-1), "I"),
    (dict(n_pages=1 << 31), "I"), (dict(ws=None), "W"), (dict(ws_bytes=255), "W"), (dict(ws=F + 8), "W")])
def test_page_plan_refusals(abi, kw, status):
    c0 = abi.csa2_launch_count()
    assert abi.lib.csa2_page_plan(*args(PLAN, **kw)) == {"U": 2, "I": 1, "W": 6}[status]
    assert abi.csa2_launch_count() == c0


@pytest.mark.parametrize("kw,status", [
    (dict(heads=0), "U"), (dict(heads=129), "U"), (dict(page=4), "U"), (dict(page=20), "U"), (dict(fmt=2), "U"),
    (dict(scales=None), "I"), (dict(fmt=1), "I"), (dict(q=None), "I"), (dict(q=F + 2), "I"), (dict(q_start=None), "I"),
    (dict(kv_len=F + 4), "I"), (dict(codes=None), "I"), (dict(table=None), "I"), (dict(out=None), "I"), (dict(lse=F + 4), "I"),
    (dict(window=-1), "I"), (dict(sm_scale=0.0), "I"), (dict(sm_scale=float("nan")), "I"), (dict(sm_scale=float("inf")), "I"),
    (dict(n_tokens=-1), "I"), (dict(n_req=-1), "I"), (dict(max_q=-1), "I"), (dict(max_kv=-1), "I"), (dict(n_rows=-1), "I"),
    (dict(max_pages=1 << 31), "I"), (dict(n_tokens=(1 << 22) + 1), "U"), (dict(max_kv=(1 << 30) + 1), "U"),
    (dict(n_req=(1 << 20) + 1), "U"), (dict(ws=None), "W"), (dict(ws_bytes=255), "W")])
def test_paged_attn_refusals(abi, kw, status):
    c0 = abi.csa2_launch_count()
    assert abi.lib.csa2_paged_attn(*args(ATTN, **kw)) == {"U": 2, "I": 1, "W": 6}[status]
    assert abi.csa2_launch_count() == c0


def test_paged_attn_workspace(abi):
    ws = abi.csa2_paged_attn_workspace_bytes
    assert ws(0, 64, 0, 0, 0, 0) >= abi.STATUS_BYTES
    for bad in ((-1, 64, 1, 1, 1, 0), (1, 0, 1, 1, 1, 0), (1, 129, 1, 1, 1, 0), (1, 64, -1, 1, 1, 0), (1, 64, 1, -1, 1, 0),
                (1, 64, 1, 1, -1, 0), (1, 64, 1, 1, 1, -1)):
        assert ws(*bad) == 0, bad


@pytest.mark.parametrize("kw,status", [
    (dict(dim=0), "I"), (dict(dim=12), "U"), (dict(dim=16392, x_stride=16392), "U"), (dict(group=64), "U"),
    (dict(group=128, dim=520, x_stride=520), "U"), (dict(x_stride=504), "I"), (dict(x_stride=516), "I"), (dict(residual=None), "I"),
    (dict(residual_out=None), "I"), (dict(x=None), "I"), (dict(weight=None), "I"), (dict(codes=None), "I"), (dict(scales=None), "I"),
    (dict(y=F + 2), "I"), (dict(codes=F + 8), "I"), (dict(eps=-1.0), "I"), (dict(eps=float("nan")), "I"), (dict(n=-1), "I")])
def test_rmsnorm_refusals(abi, kw, status):
    c0 = abi.csa2_launch_count()
    assert abi.lib.csa2_rmsnorm_fp8(*args(NORM, **kw)) == {"U": 2, "I": 1}[status]
    assert abi.csa2_launch_count() == c0


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=2), "U"), (dict(k=64, x_stride=64), "U"), (dict(k=200, x_stride=208), "U"), (dict(k=65664, x_stride=65664), "U"),
    (dict(n_out=0), "U"), (dict(n_out=-1), "I"), (dict(n=-1), "I"), (dict(x_stride=240), "I"), (dict(x_stride=264), "I"),
    (dict(x_scales=F), "I"), (dict(fmt=1), "I"), (dict(x=None), "I"), (dict(codes=F + 4), "I"), (dict(scales=None), "I"),
    (dict(out=None), "I"), (dict(out_dtype=3), "I"), (dict(alpha=float("inf")), "I"), (dict(alpha=float("nan")), "I"),
    (dict(ws=None), "W"), (dict(ws_bytes=0), "W")])
def test_matvec_refusals(abi, kw, status):
    c0 = abi.csa2_launch_count()
    assert abi.lib.csa2_fp4_matvec(*args(MATVEC, **kw)) == {"U": 2, "I": 1, "W": 6}[status]
    assert abi.csa2_launch_count() == c0


def test_empty_calls_launch_nothing(abi):
    c0 = abi.csa2_launch_count()
    assert abi.lib.csa2_paged_attn(*args(ATTN, n_tokens=0)) == abi.OK
    assert abi.lib.csa2_paged_attn(*args(ATTN, n_req=0)) == abi.OK
    assert abi.lib.csa2_rmsnorm_fp8(*args(NORM, n=0)) == abi.OK
    assert abi.lib.csa2_fp4_matvec(*args(MATVEC, n=0)) == abi.OK
    assert abi.csa2_launch_count() == c0


def test_paged_attn_workspace_of_the_largest_bounds(abi):
    """No size overflows: a bound on a request's tokens above the call's own changes nothing."""
    size = abi.csa2_paged_attn_workspace_bytes
    assert size(40, 128, 3, 2 ** 31 - 1, 1 << 30, 0) == size(40, 128, 3, 40, 1 << 30, 0) >= 256
    assert size(1 << 22, 128, 1 << 20, 1 << 22, 1 << 30, 2 ** 31 - 1) >= 256
    assert size(4, 64, 2, 4, (1 << 30) + 1, 0) == 0


def test_cache_refusals(abi):
    """What does not fit the cache's buffers is refused before any call."""
    from csa2_sparse_attention_gb300 import paged
    c = paged.PagedLatents(2, 8, 4, 16, 2, heads=4, fmt=abi.FMT_FP8, device="cpu")
    bf = torch.bfloat16
    c0 = abi.csa2_launch_count()
    for bad in (lambda: c.append(torch.zeros(9, 512, dtype=bf), 9), lambda: c.append(torch.zeros(4, 512, dtype=bf), 5),
                lambda: c.append(torch.zeros(8, 512), 8), lambda: c.append(torch.zeros(8, 256, dtype=bf), 8),
                lambda: c.append(torch.zeros(512, 8, dtype=bf).t(), 8), lambda: c.append(torch.zeros(8, 512, dtype=bf), -1),
                lambda: c.attend(torch.zeros(9, 4, 512, dtype=bf), 9, 1, 1), lambda: c.attend(torch.zeros(8, 5, 512, dtype=bf), 8, 1, 1),
                lambda: c.workspace(8, 1, (1 << 31) - 1), lambda: paged.fp4_weight(torch.zeros(4, 200, dtype=bf)),
                lambda: paged.fp4_weight(torch.zeros(4, 256))):
        with pytest.raises(ValueError):
            bad()
    assert abi.csa2_launch_count() == c0


# ------------------------------------------------- the 64-bit forms by hand
def test_plan_form_by_hand():
    table = np.array([[4, -1, -1], [2, 6, -1]], np.int32)
    free = np.array([0, 1, 3, 5, 7, 0, 0, 0], np.int32)
    t, qs, kl, slots, pos, left, ok = PO.page_plan([7, 16], [3, 1], 8, table, free, 5, 8, 6)
    assert ok and t.tolist() == [[4, 7, -1], [2, 6, 5]] and left == 3
    assert qs.tolist() == [0, 3, 4] and kl.tolist() == [10, 17]
    assert slots.tolist() == [39, 56, 57, 40, -1, -1] and pos.tolist() == [7, 8, 9, 16, -1, -1]


@pytest.mark.parametrize("window", [0, 3])
def test_attention_form_is_torch_attention(window):
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 120, (40, 512)).astype(np.uint8)
    table = np.array([[3, 0, 4]], np.int32)
    q = rng.standard_normal((4, 2, 512)).astype(np.float32)
    out, lse, _ = PO.paged_attention(q, [0, 4], [20], codes, None, table, 8, window, 0.04)
    rows = np.r_[24:32, 0:8, 32:36]
    c = torch.from_numpy(codes[rows]).view(torch.float8_e4m3fn).double()
    t = torch.arange(16, 20)[:, None]
    p = torch.arange(20)[None]
    keep = (p <= t) & ((p > t - window) if window else True)
    want = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q).double().permute(1, 0, 2)[None], c[None, None],
                                                            c[None, None], attn_mask=keep, scale=0.04)
    np.testing.assert_allclose(out, want[0].permute(1, 0, 2).numpy(), rtol=1e-12, atol=1e-12)


def test_norm_and_product_forms_by_hand():
    assert np.allclose(PO.rmsnorm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 0.0), [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]])
    codes = np.full((1, 8), 0x21, np.uint8)  # 0.5, 1.0 in turn
    got, reach = PO.matvec(np.arange(16.0)[None], np.array([2.0], np.float32), codes, np.array([[0x40]], np.uint8), 0.5)
    assert got[0, 0] == 0.5 * 2 * 2 * (0.5 * 56 + 64) and reach[0, 0] == got[0, 0]


# ------------------------------------------------------------- the sources
def test_no_kernel_loads_by_multicast():
    """Ranks of several GPUs load the same library: no copy into shared memory reaches more than its own block."""
    import glob
    import os
    import re
    root = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "csa2_sparse_attention_gb300", "csrc")
    files = glob.glob(os.path.join(root, "*.cu*"))
    assert len(files) > 10
    for f in files:
        assert not re.search("multi" + "cast", open(f).read()), f


@pytest.mark.parametrize("kw", [dict(n_req=0), dict(max_tokens=0), dict(n_pages=0), dict(max_pages=0), dict(page_size=12),
                                dict(page_size=0), dict(page_size=65544), dict(heads=0), dict(heads=129), dict(fmt=2), dict(window=-1),
                                dict(sm_scale=0.0), dict(sm_scale=1e-50), dict(sm_scale=float("nan")), dict(sm_scale=float("inf"))])
def test_cache_that_no_step_can_use(abi, kw):
    """Refused when it is made, not in the middle of its first step."""
    from csa2_sparse_attention_gb300 import paged
    good = dict(n_req=2, max_tokens=8, n_pages=4, page_size=16, max_pages=2, heads=4, fmt=abi.FMT_FP8, device="cpu")
    paged.PagedLatents(**good)
    with pytest.raises(ValueError):
        paged.PagedLatents(**{**good, **kw})


def test_rows_on_another_device_are_refused(abi):
    """A pointer of another device's memory never reaches a kernel."""
    from csa2_sparse_attention_gb300 import paged
    c = paged.PagedLatents(2, 8, 4, 16, 2, heads=4, fmt=abi.FMT_FP8, device="cpu")
    rows = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16, device="meta")  # noqa: E731
    c0 = abi.csa2_launch_count()
    with pytest.raises(ValueError, match="latents: on meta"):
        c.append(rows(8, 512), 8)
    with pytest.raises(ValueError, match="q: on meta"):
        c.attend(rows(8, 4, 512), 8, 1, 1)
    assert abi.csa2_launch_count() == c0


@pytest.mark.parametrize("kw", [dict(hidden=200), dict(hidden=16512), dict(tokens=65537), dict(eps=-1.0), dict(eps=float("nan")),
                                dict(eps=float("inf"))])
def test_layer_that_no_step_can_use(abi, kw):
    """Sizes that the norm or the products do not run are refused when the layer is made."""
    from csa2_sparse_attention_gb300 import paged
    use = {**dict(hidden=256, tokens=4, eps=1e-6), **kw}
    c = paged.PagedLatents(1, 4, 1, 8, 1, heads=1, fmt=abi.FMT_FP8, device="cpu")
    c.max_tokens = use["tokens"]
    w = lambda *shape: torch.zeros(1, dtype=torch.bfloat16).expand(*shape)  # noqa: E731
    with pytest.raises(ValueError, match="channels for steps"):
        paged.PagedLayer(c, use["hidden"], w(use["hidden"]), w(512, use["hidden"]), w(512, use["hidden"]), use["eps"])


def test_a_cache_without_rotation(abi):
    """rope_theta None has no table, and what is appended is given no positions."""
    from csa2_sparse_attention_gb300 import paged
    c = paged.PagedLatents(2, 8, 4, 16, 2, heads=4, fmt=abi.FMT_FP4, rope_theta=None, device="cpu")
    assert c.rope is None and c.scales is not None


def test_turned_queries_go_by_distances():
    """The rotation of queries and keys alike leaves logits that a shift of all positions does not change."""
    from oracle import csa2_oracle as O
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((5, 512)), rng.standard_normal((9, 512))
    at = lambda t, p, shift: O.rope(q, t + shift) @ O.rope(k, p + shift).T  # noqa: E731
    t, p = np.arange(4, 9), np.arange(9)
    # angles up to 2^17 in 64 bits: off by 2^-35, of 512 products of size 10 at most
    np.testing.assert_allclose(at(t, p, 0), at(t, p, 100000), rtol=0, atol=512 * 10 * 2.0 ** -35)
    assert np.abs(q @ O.rope(k, p).T - q @ O.rope(k, p + 1).T).max() > 1  # (with keys alone turned it does)


@pytest.mark.parametrize("out", [F, F + 16, F + 4 * 64 * 1024 - 16, F - 16, F - 4 * 64 * 1024 + 16])
def test_attention_into_its_queries_is_refused(abi, out):
    """Blocks read queries after others have written outputs."""
    c0 = abi.csa2_launch_count()
    assert abi.lib.csa2_paged_attn(*args(ATTN, out=out)) == abi.ERR_INVALID_ARG
    assert abi.csa2_launch_count() == c0


@pytest.mark.parametrize("kw", [dict(out=F), dict(out=F + 2 * 256 * 2 - 16), dict(out=F + 2 * 300 * 2, x_stride=352),
                                dict(out=F - 16), dict(out=F - 2 * 8 * 4 + 16, out_dtype=1),
                                dict(out=F + 2 * 256 - 16, fmt=1, x_scales=4 * F)])
def test_products_into_their_rows_are_refused(abi, kw):
    c0 = abi.csa2_launch_count()
    assert abi.lib.csa2_fp4_matvec(*args(MATVEC, **kw)) == abi.ERR_INVALID_ARG
    assert abi.csa2_launch_count() == c0
