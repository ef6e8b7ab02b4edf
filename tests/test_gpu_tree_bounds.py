"""Calls of a step of trees at the ends of what they document: requests whose bounds do not hold, requests without keys,
steps without tokens, the smallest and largest values; the forms and bounds are those of test_gpu_tree.py."""
import numpy as np
import pytest
import torch

from oracle import tree_oracle as TO
from tests.test_gpu_tree import Commit, abi  # noqa: F401

pytestmark = pytest.mark.gpu


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
