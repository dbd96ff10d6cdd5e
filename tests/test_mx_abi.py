"""MXFP4 and routing entry points without a GPU: the argument checks of the C ABI
(every refusal comes before a device is touched) and of the Python layer."""
import ctypes

import pytest
import torch

import dequant_gemv_nf4_amd as nf4

EINVAL, EALIGN, ERANGE = -1, -2, -3
P = ctypes.c_void_p(0x100000)      # fake, 16-byte aligned; never dereferenced on these paths
ODD = ctypes.c_void_p(0x100001)
TWO = ctypes.c_void_p(0x100002)
NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    return nf4._lib._load()


BAD_SHAPES = [(0, 32, EINVAL), (-1, 32, EINVAL), (4, 0, EINVAL), (4, 48, EINVAL), (4, -32, EINVAL),
              (4, 32768 + 32, ERANGE), (1 << 31, 32, ERANGE), (1 << 17, 32768, ERANGE),
              (1 << 62, 1 << 40, ERANGE)]


@pytest.mark.parametrize("N,K,expect", BAD_SHAPES)
def test_matrix_shapes(lib, N, K, expect):
    assert lib.nf4_mx_pack(P, 0, N, K, P, P, NULL, NULL) == expect
    assert lib.nf4_mx_unpack(P, P, N, K, P, 1, NULL) == expect
    assert lib.nf4_mx_gemm(P, P, N, K, P, 4, P, 0, NULL) == expect
    assert lib.nf4_mx_gemm_packed(P, P, N, K, P, P, 4, P, 0, NULL) == expect
    assert lib.nf4_mx_gemm_grouped(P, P, 2, N, K, P, P, 4, P, 0, NULL) == expect
    assert lib.nf4_mx_gemm_grouped_grad(P, P, 2, N, K, P, P, 4, P, 0, NULL) == expect


def _calls(lib):
    """(name, call, pointer arguments with the alignment each needs; 0: may be null)."""
    return [
        ("pack", lambda a, b, c, d: lib.nf4_mx_pack(a, 1, 4, 64, b, c, d, NULL), (16, 4, 1, 0)),
        ("unpack", lambda a, b, c: lib.nf4_mx_unpack(a, b, 4, 64, c, 0, NULL), (4, 1, 16)),
        ("gemm", lambda a, b, c, d: lib.nf4_mx_gemm(a, b, 4, 64, c, 3, d, 0, NULL),
         (16, 1, 16, 16)),
        ("packed", lambda a, b, c, d, e: lib.nf4_mx_gemm_packed(a, b, 4, 64, c, d, 3, e, 0, NULL),
         (16, 1, 16, 1, 16)),
        ("grouped", lambda a, b, c, d, e: lib.nf4_mx_gemm_grouped(a, b, 2, 8, 64, c, d, 3, e, 0,
                                                                  NULL), (16, 1, 16, 4, 16)),
        ("grad", lambda a, b, c, d, e: lib.nf4_mx_gemm_grouped_grad(a, b, 2, 8, 64, c, d, 3, e, 0,
                                                                    NULL), (16, 1, 16, 4, 16)),
        ("sort", lambda a, b, c, d, e: lib.nf4_moe_sort(a, 3, 2, 4, b, c, d, e, NULL),
         (8, 4, 4, 4, 0)),
        ("gather", lambda a, b, c: lib.nf4_moe_gather(a, 0, b, 3, 2, 8, c, NULL), (4, 4, 4)),
        ("combine", lambda a, b, c, d: lib.nf4_moe_combine(a, 0, b, c, 3, 2, 8, d, NULL),
         (4, 4, 0, 4)),
        ("combine_grad", lambda a, b, c, d, e, f: lib.nf4_moe_combine_grad(
            a, b, 0, c, d, 3, 2, 8, e, f, NULL), (4, 4, 4, 4, 4, 4)),
    ]


def test_null_and_misaligned_pointers(lib):
    for name, call, need in _calls(lib):
        for i, a in enumerate(need):
            args = [P] * len(need)
            args[i] = NULL
            if a:
                assert call(*args) == EINVAL, (name, i)
            args[i] = ODD
            if a != 1:
                assert call(*args) == EALIGN, (name, i)
            if a > 2:
                args[i] = TWO
                assert call(*args) == EALIGN, (name, i)


@pytest.mark.parametrize("dtype", [-1, 2, 7])
def test_unknown_dtypes(lib, dtype):
    assert lib.nf4_mx_pack(P, dtype, 4, 64, P, P, NULL, NULL) == EINVAL
    assert lib.nf4_mx_unpack(P, P, 4, 64, P, dtype, NULL) == EINVAL
    assert lib.nf4_mx_gemm(P, P, 4, 64, P, 3, P, dtype, NULL) == EINVAL
    assert lib.nf4_mx_gemm_packed(P, P, 4, 64, P, P, 3, P, dtype, NULL) == EINVAL
    assert lib.nf4_mx_gemm_grouped(P, P, 2, 8, 64, P, P, 3, P, dtype, NULL) == EINVAL
    assert lib.nf4_mx_gemm_grouped_grad(P, P, 2, 8, 64, P, P, 3, P, dtype, NULL) == EINVAL
    assert lib.nf4_moe_gather(P, dtype, P, 3, 2, 8, P, NULL) == EINVAL
    assert lib.nf4_moe_combine(P, dtype, P, P, 3, 2, 8, P, NULL) == EINVAL
    assert lib.nf4_moe_combine_grad(P, P, dtype, P, P, 3, 2, 8, P, P, NULL) == EINVAL


@pytest.mark.parametrize("M", [0, -1, 1 << 26, 1 << 60])
def test_rows_of_a_product(lib, M):
    assert lib.nf4_mx_gemm(P, P, 4, 64, P, M, P, 0, NULL) == ERANGE
    assert lib.nf4_mx_gemm_packed(P, P, 4, 64, P, P, M, P, 0, NULL) == ERANGE


def test_experts_and_rows(lib):
    for f in (lib.nf4_mx_gemm_grouped, lib.nf4_mx_gemm_grouped_grad):
        assert f(P, P, 0, 8, 64, P, P, 3, P, 0, NULL) == EINVAL
        assert f(P, P, 513, 8, 64, P, P, 3, P, 0, NULL) == ERANGE
        assert f(P, P, 2, 8, 64, P, P, -1, P, 0, NULL) == EINVAL
        assert f(P, P, 2, 8, 64, P, P, 1 << 26, P, 0, NULL) == ERANGE
    assert lib.nf4_mx_gemm_grouped_grad(P, P, 2, 12, 64, P, P, 3, P, 0, NULL) == EINVAL
    assert lib.nf4_mx_gemm_grouped_grad(P, P, 2, (1 << 23) + 8, 32, P, P, 3, P, 0, NULL) == ERANGE


@pytest.mark.parametrize("T,topk,expect", [(-1, 2, EINVAL), (4, 0, EINVAL), (4, 513, ERANGE),
                                           (1 << 24, 1, ERANGE), ((1 << 24) - 1, 65, ERANGE),
                                           (1 << 62, 4, ERANGE)])
def test_slots(lib, T, topk, expect):
    assert lib.nf4_moe_sort(P, T, topk, 4, P, P, P, NULL, NULL) == expect
    assert lib.nf4_moe_gather(P, 0, P, T, topk, 8, P, NULL) == expect
    assert lib.nf4_moe_combine(P, 0, P, P, T, topk, 8, P, NULL) == expect
    assert lib.nf4_moe_combine_grad(P, P, 0, P, P, T, topk, 8, P, P, NULL) == expect


def test_sort_experts_and_row_widths(lib):
    assert lib.nf4_moe_sort(P, 3, 2, 0, P, P, P, NULL, NULL) == EINVAL
    assert lib.nf4_moe_sort(P, 3, 2, 513, P, P, P, NULL, NULL) == ERANGE
    for H, expect in ((0, EINVAL), (-4, EINVAL), ((1 << 20) + 1, ERANGE)):
        assert lib.nf4_moe_gather(P, 0, P, 3, 2, H, P, NULL) == expect
        assert lib.nf4_moe_combine(P, 0, P, P, 3, 2, H, P, NULL) == expect
        assert lib.nf4_moe_combine_grad(P, P, 0, P, P, 3, 2, H, P, P, NULL) == expect


def test_python_refuses_host_tensors_and_wrong_types():
    codes = torch.zeros((4, 32), dtype=torch.uint8)
    scales = torch.zeros((4, 2), dtype=torch.uint8)
    X = torch.zeros((3, 64), dtype=torch.bfloat16)
    place = torch.zeros((3, 2), dtype=torch.int32)
    for call in (lambda: nf4.mx_pack(X), lambda: nf4.mx_unpack(codes, scales),
                 lambda: nf4.mx_gemm(codes, scales, X),
                 lambda: nf4.mx_gemm_packed(codes, scales, codes, scales),
                 lambda: nf4.mx_gemm_grouped(codes[None], scales[None], X, place[0]),
                 lambda: nf4.mx_gemm_grouped_grad(codes[None], scales[None], X, place[0]),
                 lambda: nf4.moe_sort(place.long(), 4), lambda: nf4.moe_gather(X, place),
                 lambda: nf4.moe_combine(X, place), lambda: nf4.moe_combine_grad(X, X, place, X)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(TypeError, match="torch.Tensor"):
        nf4.nf4_mx_pack([1.0], codes, scales)
