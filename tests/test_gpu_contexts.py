"""Tensor maps are made under the calling thread's context, and leave it as it is."""
import ctypes
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import paged_kv_cache_196_gb300 as pk
from _gpu import require_cuda

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
