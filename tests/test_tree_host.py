"""Calls over drafted tokens that are refused before anything is launched.  No GPU needed."""
import numpy as np
import pytest

import paged_kv_cache_196_gb300 as pk


def status(fn, *args, **kw):
    with pytest.raises(pk.KVError) as e:
        fn(*args, **kw)
    return e.value.status


def test_no_pool():
    assert status(pk.kv_tree_workspace_size, None, 1, 4, 4, 4) == -1
    assert status(pk.paged_tree_attention, None, None, None, 0, 0, None, None, 0, None, 0, 1, 1.0, None, pk.KV_F32,
                  stream=0) == -1
    assert status(pk.kv_verify_tree, None, None, None, pk.KV_F32, 10, None, 0, 0, None, None, None, None, 0, 0, None, None,
                  None, stream=0) == -1
    z = np.zeros(4, np.int32)
    assert status(pk.kv_keep_path, [], z, 1, z, 1, z, z, 1, z, 1, z, stream=0) == -1
    assert status(pk.kv_keep_path, [None], z, 1, z, 1, z, z, 1, z, 1, z, stream=0) == -1
    assert status(pk.kv_keep_path, [None, None], z, 1, z, 1, z, z, 1, z, 1, z, stream=0) == -1


def test_sizes():
    assert status(pk.kv_verify_tree, None, None, None, pk.KV_F32, 0, None, 0, 0, None, None, None, None, 0, 0, None, None,
                  None, stream=0) == -1
    assert pk.lib().kv_tree_workspace_size(None, 1, 4, 4, 4, None) == -1


def test_reference_of_the_walk():
    """The tests' own walk against cases worked out by hand."""
    from _tree import verify_reference
    p = np.array([[0.5, 0.25, 0.25], [0.0, 1.0, 0.0], [0.2, 0.3, 0.5]])
    q = np.array([[0.25, 0.5, 0.25], [1.0, 0.0, 0.0], [0.2, 0.3, 0.5]])
    # node 1 (token 1): 0.6 * 0.5 = 0.3 >= 0.25: rejected; what is left is token 0 alone
    got = verify_reference(p, q, [0, 2], [-1, 0], [0, 1], [0, 0.6], [0.9], 2, 3)
    assert [x.tolist() for x in got] == [[0], [[-1, -1]], [[0, -1, -1]]]
    # 0.4 * 0.5 < 0.25: accepted; the row after node 1 is all token 1
    got = verify_reference(p, q, [0, 2], [-1, 0], [0, 1], [0, 0.4], [0.9], 2, 3)
    assert [x.tolist() for x in got] == [[1], [[1, -1]], [[1, 1, -1]]]
    # chosen drafts: 0.3 >= 0.25 rejects token 1, token 2 then has a third of what is left
    got = verify_reference(p, None, [0, 3], [-1, 0, 0], [0, 1, 2], [0, 0.3, 0.32], [0.0], 2, 3)
    assert [x.tolist() for x in got] == [[1], [[2, -1]], [[2, 0, -1]]]
    got = verify_reference(p, None, [0, 3], [-1, 0, 0], [0, 1, 2], [0, 0.3, 0.34], [0.99], 2, 3)
    assert [x.tolist() for x in got] == [[0], [[-1, -1]], [[0, -1, -1]]]
