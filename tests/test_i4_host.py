"""Host logic of the 4-bit pools' calls and of their tests' reference. No GPU."""
import numpy as np
import pytest
import torch

import paged_kv_cache_196_gb300 as pk
from _i4 import E4M3, e4m3_round, stored


def test_null_pools_are_refused():
    for f, a in ((pk.kv_append_rope, (None, None, None, pk.KV_BF16, None, 0)),
                 (pk.kv_read_tokens, (None, None, 0, None, None, pk.KV_F32)),
                 (pk.kv_pool_set_i4_scales, (None, 1.0, 1.0)),
                 (pk.paged_decode_attention_i4, (None, None, pk.KV_BF16, None, 0, None, 0, 1, 1.0, None, pk.KV_F32)),
                 (pk.kv_prefill_i4_workspace_size, (None, 1, 1, 1, 1)),
                 (pk.paged_prefill_attention_i4, (None, None, pk.KV_BF16, None, 0, 0, None, 0, None, 0, 1, 1.0, None, pk.KV_F32))):
        with pytest.raises(pk.KVError) as e:
            k = {} if f in (pk.kv_pool_set_i4_scales, pk.kv_prefill_i4_workspace_size) else {"stream": 0}
            f(*a, **k)
        assert e.value.status == -1


def test_plan_bounds():
    for lens in ([1], [0, 0], [100] * 64, [196608] * 8, list(range(1, 4000, 37))):
        width = max(1, -(-max(lens) // 16))
        s = pk.kv_decode_plan_i4(lens, 4, width)
        pb, ms = pk.kv_decode_split_plan(len(lens), 4, width, s)
        assert s >= 1 and 1 <= ms <= 65535 and pb * ms >= width
    assert pk.kv_decode_plan_i4([], 4, 10) == 1
    with pytest.raises(pk.KVError):
        pk.kv_decode_plan_i4([5], 0, 10)


def test_reference_scales_are_those_of_the_type():
    """The tests' e4m3 rounding against the type's own, and its ties."""
    assert len(E4M3) == 127 and E4M3[-1] == 448
    x = np.concatenate([E4M3, (E4M3[1:] + E4M3[:-1]) / 2, np.random.default_rng(0).uniform(0, 448, 4000),
                        np.random.default_rng(1).uniform(0, 2.0 ** -6, 4000)])
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(e4m3_round(x.astype(np.float32).astype(np.float64)), want)
    assert e4m3_round(np.array([1e9]))[0] == 448


def test_stored_values_fit_sixteen_bits():
    """Every code times every scale, a 256th of it and the kernels' constants are
    exact in fp16 (and the values in bf16); a scale's byte shifted by 7 is its 256th."""
    assert np.array_equal((np.arange(127, dtype=np.uint16) << 7).view(np.float16).astype(np.float64), E4M3 / 256)
    assert np.isnan(np.array([0xff << 7], np.uint16).view(np.float16))[0]
    c = np.arange(-8, 8)[:, None] * E4M3[None]
    for x in (c, c / 256, 72 * E4M3 / 256, 1032 * E4M3 / 256, E4M3 / 256):
        assert np.array_equal(x.astype(np.float16).astype(np.float64), x)
    t = torch.from_numpy(c)
    assert torch.equal(t.to(torch.bfloat16).double(), t)


def test_stored_reference():
    x = np.zeros((1, 16))
    assert np.array_equal(stored(x), x)
    x[0, :4] = [7, 3.5, 0.5, -1.5]          # scale 1: ties to even
    assert stored(x)[0, :4].tolist() == [7, 4, 0, -2]
    x[0, 0] = 1e6
    assert stored(x)[0, 0] == 3136
    x[0, 1] = np.nan
    assert np.isnan(stored(x)).all()
