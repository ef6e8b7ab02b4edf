"""Refusals of the calls of a step of trees beyond those of test_tree_cpu.py: no launch, no pointer that is valid."""
import pytest
import torch

from tests.test_tree_cpu import COMMIT, abi, refused  # noqa: F401

FAR = 1 << 40  # never dereferenced


# 4 tokens x 64 heads: 262144 bytes of outputs, 1024 of log-sum-exps; 128 rows of 256 and 32 bytes; every buffer on its own
ATTN = dict(q=FAR, n_tokens=4, heads=64, q_start=2 * FAR, kv_len=3 * FAR, n_req=2, max_q=2, max_kv=100, pos=4 * FAR, mask=5 * FAR, words=1,
            fmt=0, codes=6 * FAR, scales=7 * FAR, n_rows=128, table=8 * FAR, max_pages=8, page=16, window=0, sm_scale=0.04, out=9 * FAR,
            lse=10 * FAR, ws=11 * FAR, ws_bytes=1 << 39, stream=None)


@pytest.mark.parametrize("kw", [
    dict(lse=9 * FAR), dict(lse=9 * FAR + 262128), dict(lse=9 * FAR - 1008), dict(out=10 * FAR + 1008), dict(lse=FAR + 262128),
    dict(lse=2 * FAR), dict(lse=3 * FAR - 1008), dict(lse=4 * FAR + 16), dict(lse=5 * FAR), dict(lse=6 * FAR + 128 * 256 - 16),
    dict(lse=7 * FAR + 128 * 32 - 16), dict(lse=8 * FAR + 48), dict(out=2 * FAR - 262128), dict(out=3 * FAR), dict(out=4 * FAR + 16),
    dict(out=5 * FAR - 16), dict(out=6 * FAR + 128 * 256 - 16), dict(out=6 * FAR + 128 * 512 - 16, fmt=1, scales=None), dict(out=7 * FAR - 262128),
    dict(out=8 * FAR + 48)])
def test_attention_outputs_over_inputs_are_refused(abi, kw):
    refused(abi, "csa2_tree_attn", ATTN, kw, "I")


@pytest.mark.parametrize("name", ["n_free", "n_free_out"])
@pytest.mark.parametrize("by", [1, 2, 3])
def test_commit_counts_that_no_load_can_reach_are_refused(abi, name, by):
    refused(abi, "csa2_tree_commit", COMMIT, {name: 9 * FAR + by}, "I")


PAGES = dict(cached=FAR, added=2 * FAR, n_req=2, page=16, table=3 * FAR, max_pages=4, free=4 * FAR, n_pages=8, n_free=5 * FAR, n_free_out=5 * FAR,
             q_start=6 * FAR, kv_len=7 * FAR, slots=8 * FAR, pos=9 * FAR, max_new=6, ws=10 * FAR, ws_bytes=256, stream=None)


@pytest.mark.parametrize("name", ["n_free", "n_free_out", "q_start", "kv_len"])
@pytest.mark.parametrize("by", [1, 2, 3])
def test_page_plan_numbers_that_no_load_can_reach_are_refused(abi, name, by):
    refused(abi, "csa2_page_plan", PAGES, {name: 11 * FAR + by}, "I")


def test_views_off_a_boundary_are_refused_before_a_step(abi):
    """Nodes' values and weights that the calls would refuse in the middle of a step."""
    from csa2_sparse_attention_gb300 import paged
    c = paged.PagedLatents(2, 8, 4, 16, 2, heads=1, fmt=abi.FMT_FP8, device="cpu")
    bf = torch.bfloat16
    par, tok = torch.zeros(12, dtype=torch.int32), torch.zeros(12, dtype=torch.int64)
    w = lambda *shape: torch.zeros(shape, dtype=bf)  # noqa: E731
    c0 = abi.csa2_launch_count()
    for bad in (lambda: c.tree(par[1:], 8, 4), lambda: c.tree(par[3:], 8, 4), lambda: c.commit(par[2:], tok, tok, 8, 4),
                lambda: c.commit(par, tok[1:], tok, 8, 4), lambda: c.commit(par, tok, tok[1:], 8, 4),
                lambda: paged.PagedLayer(c, 256, w(256), w(512, 256), w(512, 256), q_norm=w(520)[3:515]),
                lambda: paged.PagedLayer(c, 256, w(256), w(512, 256), w(512, 256), latent_norm=w(520)[4:516])):
        with pytest.raises(ValueError, match="not 16-byte aligned"):
            bad()
    assert abi.csa2_launch_count() == c0
