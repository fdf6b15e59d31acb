"""Tensor maps are made under the calling thread's context, and leave it as it is."""
import ctypes
import threading
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import paged_kv_cache_196_gb300 as pk
from _gpu import require_cuda
from _tree import TreeCase

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    require_cuda()


def test_a_context_of_the_threads_own_stays():
    torch.zeros(1, device="cuda")
    cuda = ctypes.CDLL("libcuda.so.1")

    def current():
        c = ctypes.c_void_p()
        assert cuda.cuCtxGetCurrent(ctypes.byref(c)) == 0
        return c.value

    def work():
        dev, ctx = ctypes.c_int(), ctypes.c_void_p()
        assert cuda.cuDeviceGet(ctypes.byref(dev), torch.cuda.current_device()) == 0
        assert cuda.cuCtxCreate_v2(ctypes.byref(ctx), 0, dev) == 0
        try:
            assert current() == ctx.value
            # (reserving makes the maps of the request's region; nothing is launched)
            c = pk.kv_contig_create(1, 64, 1, 128, pk.KV_BF16)
            try:
                pk.kv_contig_reserve(c, 0)
                return current() == ctx.value
            finally:
                pk.kv_contig_destroy(c)
        finally:
            assert cuda.cuCtxDestroy_v2(ctx) == 0

    with ThreadPoolExecutor(1) as pool:
        assert pool.submit(work).result()


def test_a_thread_without_a_context_gets_one():
    c = pk.kv_contig_create(1, 64, 1, 128, pk.KV_BF16)
    try:
        with ThreadPoolExecutor(1) as pool:
            pool.submit(pk.kv_contig_reserve, c, 0).result()
    finally:
        pk.kv_contig_destroy(c)


@pytest.mark.parametrize("seed", range(4))
def test_first_prefills_of_two_host_threads(seed):
    """They make what the pool keeps for its calls (its tensor maps) together."""
    case = TreeCase("bf16", 128, 2, 4, [700, 20], [9, 3], kind="chain", seed=seed)
    try:
        a = [case.args("f32") for _ in range(2)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        start = threading.Barrier(2)

        def one(i):
            start.wait(timeout=30)
            x = a[i]
            pk.paged_prefill_attention(case.pool, x["q"], x["cu"], x["total"], 9, x["tables"], case.width, x["lens"], 2,
                                       case.hq, case.scale, x["out"], pk.KV_F32, x["lse"], stream=streams[i])
        with ThreadPoolExecutor(2) as pool:
            list(pool.map(one, range(2)))
        torch.cuda.synchronize()
        assert pk.kv_get_device_error(case.pool) == 0
        out, lse, _, _ = case.reference()
        for x in a:
            got = x["out"].double().cpu().numpy()[:case.total]
            # (the prefill weighs in bf16 once: 2^-8 of the largest value)
            assert (abs(got - out) <= 2.0 ** -7 * abs(case.v[0].double()).max().item()).all()
        assert torch.equal(a[0]["out"], a[1]["out"])
    finally:
        case.close()
