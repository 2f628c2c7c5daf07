"""The workspace of moe_orthogonalize may begin at any multiple of 16 bytes, as every operator's may.  The
kernels read and write rows of A and B 32 bytes at a time, so the call rounds the beginning up to 1024 bytes,
and the size that it asks for has room for that."""

import ctypes

import pytest

from expert_routed_ffn_gb300 import build as moe_build
from expert_routed_ffn_gb300 import capi

QUINTIC = (3.4445, -4.7750, 2.0315)
FROM = 1024  # where the parts begin, from the beginning rounded up to it


def _room(n):
    return -(-n // FROM) * FROM


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return capi.load()


def _need(lib, E, N, K):
    need = ctypes.c_size_t()
    assert lib.moe_orthogonalize_workspace(E, N, K, ctypes.byref(need)) == capi.MOE_OK
    return need.value


@pytest.mark.parametrize("E,N,K", [(1, 64, 64), (2, 64, 128), (3, 72, 136), (32, 1408, 2048), (1, 8, 16384)])
def test_size_has_room_for_a_beginning_at_16_bytes(lib, E, N, K):
    # X twice and its low half [E, N, K], A and B [E, m, m] with rows padded to 16, all fp16; a factor of each
    # matrix and at least one fp64 sum of each
    m = min(N, K)
    parts = 3 * _room(2 * E * N * K) + 2 * _room(2 * E * m * (-(-m // 16) * 16)) + _room(4 * E) + _room(8 * E)
    assert _need(lib, E, N, K) >= parts + FROM - 16


def test_less_than_that_is_refused(lib):
    need = _need(lib, 1, 64, 64)
    table = (ctypes.c_float * 15)(*QUINTIC * 5)
    for start in (1 << 24, (1 << 24) + 16, (1 << 24) + 1008):
        # never dereferenced: the size is refused first
        status = lib.moe_orthogonalize(ctypes.c_void_p(1 << 26), 1, 1, 64, 64, table, 5, 1e-7, 1.0, ctypes.c_void_p(1 << 27),
                                       ctypes.c_void_p(start), need - 1, None)
        assert status == capi.MOE_ERR_INVALID_ARG and str(need) in lib.moe_last_error().decode()


@pytest.mark.gpu
@pytest.mark.parametrize("E,N,K", [(1, 64, 64), (2, 200, 136), (3, 136, 264)])
def test_any_beginning_gives_the_same(lib, E, N, K):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(71)
    G = torch.randn(E, N, K, generator=gen, device="cuda")
    want = capi.orthogonalize(G)
    need = _need(lib, E, N, K)
    pool = torch.empty(need + 4096, dtype=torch.uint8, device="cuda")
    table = (ctypes.c_float * 15)(*QUINTIC * 5)
    assert pool.data_ptr() % 512 == 0
    for start in (0, 16, 32, 48, 496, 1008, 1024, 2032):
        pool.fill_(0x5A)
        out = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda")
        status = lib.moe_orthogonalize(G.data_ptr(), capi.MOE_DTYPE_F32, E, N, K, table, 5, 1e-7, 1.0, out.data_ptr(),
                                       pool.data_ptr() + start, need, torch.cuda.current_stream().cuda_stream)
        assert status == capi.MOE_OK
        assert torch.equal(out, want), start
        assert bool((pool[:start] == 0x5A).all()) and bool((pool[start + need:] == 0x5A).all()), start
    assert capi.operators_status() == capi.MOE_OK
