"""The 4-bit store at the places where a code or a scale is decided: every border
between two codes under every scale and every border between two scales, with the
fp32 numbers next to them, against 64 bits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_196_gb300 as pk
from _gpu import require_cuda
from _i4 import E4M3, f64, stored

pytestmark = pytest.mark.gpu


def steps(x, n):
    """The fp32 number n places from x."""
    x = np.float32(x)
    for _ in range(abs(n)):
        x = np.nextafter(x, np.float32(np.inf if n > 0 else -np.inf))
    return x


def store_and_read(rows, g):
    """rows [n][16] fp32 as groups of a 4-bit pool's K and V with scale g."""
    rows = np.concatenate([rows, np.zeros((-len(rows) % 8, 16), np.float32)]).reshape(-1, 1, 128)
    n = len(rows)
    pool = pk.kv_pool_create(-(-n // 16), 16, 1, 128, pk.KV_I4)
    pk.kv_pool_set_i4_scales(pool, g, g)
    x = torch.from_numpy(rows).cuda()
    slots = torch.arange(n, dtype=torch.int64, device="cuda")
    pk.kv_append_rope(pool, x, x, pk.KV_F32, slots, n)
    k, v = torch.empty_like(x), torch.empty_like(x)
    pk.kv_read_tokens(pool, slots, n, k, v, pk.KV_F32)
    assert pk.kv_get_device_error(pool) == 0
    pk.kv_pool_destroy(pool)
    return rows, f64(k), f64(v)


@pytest.mark.parametrize("g", [1.0, 2.0 ** -7])
def test_every_border_between_codes(g):
    require_cuda()
    rows = []
    for s in E4M3[1:]:
        at = [sign * steps((k + 0.5) * s, d) for k in range(7) for d in (-2, -1, 0, 1, 2) for sign in (1, -1)]
        for i in range(0, len(at), 14):  # 7 s makes s the group's scale
            rows.append([7 * s, *at[i:i + 14], -7 * s])
    rows = np.array(rows, np.float32) * np.float32(g)
    rows, k, v = store_and_read(rows, g)
    want = stored(rows.astype(np.float64), g)
    np.testing.assert_array_equal(k, want)
    np.testing.assert_array_equal(v, want)
    # the scales were the ones meant: the largest element is kept as 7 s
    assert np.array_equal(np.abs(k).reshape(-1, 16).max(1)[:5 * len(E4M3[1:])], np.repeat(7 * E4M3[1:] * g, 5))


def test_every_border_between_scales():
    require_cuda()
    rows = []
    borders = np.concatenate([(E4M3[1:] + E4M3[:-1]) / 2, E4M3[1:]])
    for b in borders:
        for d in (-3, -2, -1, 0, 1, 2, 3):
            m = steps(7 * b, d)
            rows.append([m, -m / 2, m / 3, 0] * 4)
    rows, k, v = store_and_read(np.array(rows, np.float32), 1.0)
    want = stored(rows.astype(np.float64))
    np.testing.assert_array_equal(k, want)
    np.testing.assert_array_equal(v, want)
