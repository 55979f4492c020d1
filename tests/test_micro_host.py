"""Block-scaled FP4 and the quantising row stages without a GPU: the oracle
against hand-made values and brute force, the sizes and refusals of the C ABI,
and the refusals of the Python entry points."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import micro_oracle as MO
from oracle import sp24_oracle as O
from structured_sparse_fp8_b200 import _lib
from structured_sparse_fp8_b200 import build as B
import structured_sparse_fp8_b200 as sp


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _lib.load()


# ------------------------------------------------------------------ oracle
def test_nvfp4_hand_example():
    # row amax 6 * 448: R / 2688 = 1, so the block scales stand alone
    x = np.zeros((1, 32))
    x[0, 0], x[0, 1], x[0, 2] = 2688.0, 1344.0, -672.0     # block 0: sf = 448 -> 6, 3, -1.5
    x[0, 16:20] = [3.0, -1.0, 0.25, 0.125]                 # block 1: sf = 448 * 3 / 2688 = 0.5
    codes, byts, rs = MO.quantize(x, "nvfp4")
    assert rs[0] == 1.0
    assert O.e4m3_decode(byts)[0].tolist() == [448.0, 0.5]
    assert O.e2m1_decode(codes)[0, :4].tolist() == [6.0, 3.0, -1.5, 0.0]
    assert O.e2m1_decode(codes)[0, 16:20].tolist() == [6.0, -2.0, 0.5, 0.0]  # 0.125 / 0.5 is a tie: to even


def test_mxfp4_hand_example():
    x = np.zeros((1, 64))
    x[0, :6] = [7.0, 5.0, 3.5, -0.25, 0.75, 2.5]           # floor(log2 7) = 2: scale 1
    x[0, 32:34] = [0.375, -0.1875]                         # floor(log2 0.375) = -2: scale 2^-4
    codes, byts, rs = MO.quantize(x, "mxfp4")
    assert rs is None and byts[0].tolist() == [127, 123]
    assert O.e2m1_decode(codes)[0, :6].tolist() == [6.0, 4.0, 4.0, -0.0, 1.0, 2.0]
    assert O.e2m1_decode(codes)[0, 32:34].tolist() == [6.0, -3.0]


def test_e2m1_codes_agree_with_the_nearest_value_search():
    v = np.concatenate([np.arange(-8, 8, 1 / 64), [5.0, -5.0, 0.25, -0.25, 1e30, 0.0, -0.0]])
    assert np.array_equal(MO.e2m1_codes(v), O.e2m1_encode(v.astype(np.float32)))


@pytest.mark.parametrize("rows,n", [(1, 1), (1, 5), (127, 4), (128, 3), (300, 9)])
def test_tile_order_is_a_permutation(rows, n):
    off = MO.tile_offsets(rows, n)
    assert len(np.unique(off)) == rows * n and off.max() < MO.tile_bytes(rows, n)
    s = np.random.default_rng(rows).integers(1, 255, (rows, n)).astype(np.uint8)
    t = MO.to_tiles(s)
    assert np.array_equal(MO.from_tiles(t, rows, n), s) and int((t != 0).sum()) == rows * n
    # spelled out for one place: row 37 of band 1, block 6
    if rows > 165 and n > 6:
        assert t[(1 * ((n + 3) // 4) + 1) * 512 + 5 * 16 + 1 * 4 + 2] == s[165, 6]


def test_zero_and_tiny_rows():
    x = np.zeros((3, 32))
    x[1] = 2.0 ** -130                 # a subnormal row: below the floor, all codes 0
    x[2, 0] = 2688.0 * 2.0 ** -100     # exactly the floor
    codes, byts, rs = MO.quantize(x, "nvfp4")
    assert rs.tolist() == [1.0, 2.0 ** -100, 2.0 ** -100]
    assert not codes[:2].any() and byts[0].tolist() == [0, 0]
    assert O.e2m1_decode(codes)[2, 0] == 6.0 and O.e4m3_decode(byts)[2, 0] == 448.0


# ------------------------------------------------------------------ C ABI
FAKE = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)


def test_block_scale_sizes(lib):
    for fmt, name in ((0, "nvfp4"), (1, "mxfp4")):
        for rows, cols in ((1, 32), (128, 64), (129, 4096), (1000, 4160)):
            want = MO.tile_bytes(rows, cols // MO.BLOCK[name])
            assert lib.fp4_block_scales_size(rows, cols, fmt) == want == sp.fp4_block_scales_size(rows, cols, name)
    assert lib.fp4_block_scales_size(0, 32, 0) == 0
    assert lib.fp4_block_scales_size(1, 32, 2) == 0
    assert lib.fp4_block_scales_size(1, 48, 1) == 0


def test_quantize_refusals(lib):
    f = lib.fp4_quantize_microscaled
    assert f(FAKE, 4, 64, 2, FAKE, FAKE, FAKE, None, None) == _lib.SP24_ERR_DTYPE
    assert f(FAKE, 4, 64, -1, FAKE, FAKE, FAKE, None, None) == _lib.SP24_ERR_DTYPE
    for bad in ((None, FAKE, FAKE, FAKE), (FAKE, None, FAKE, FAKE), (FAKE, FAKE, None, FAKE), (FAKE, FAKE, FAKE, None)):
        assert f(bad[0], 4, 64, 0, bad[1], bad[2], bad[3], None, None) == _lib.SP24_ERR_NULL
    for rows, cols in ((0, 64), (-1, 64), (4, 0), (4, 48), (4, 16), ((1 << 31) - 127, 64), (4, 1 << 31)):
        assert f(FAKE, rows, cols, 0, FAKE, FAKE, FAKE, None, None) == _lib.SP24_ERR_SHAPE
    for bad in ((ODD, FAKE, FAKE, FAKE), (FAKE, ODD, FAKE, FAKE), (FAKE, FAKE, ODD, FAKE), (FAKE, FAKE, FAKE, ODD)):
        assert f(bad[0], 4, 64, 0, bad[1], bad[2], bad[3], None, None) == _lib.SP24_ERR_ALIGN
    u = lib.fp4_unpack_e4m3
    assert u(None, 4, 64, FAKE, None) == _lib.SP24_ERR_NULL
    assert u(FAKE, 4, 48, FAKE, None) == _lib.SP24_ERR_SHAPE
    assert u(FAKE, 0, 64, FAKE, None) == _lib.SP24_ERR_SHAPE
    assert u(FAKE, 4, 64, ODD, None) == _lib.SP24_ERR_ALIGN


def test_norm_and_gate_refusals(lib):
    EPS = ctypes.byref(ctypes.c_float(0.1))
    n8, n4 = lib.fp8_rmsnorm_quantize_pertoken, lib.fp4_rmsnorm_quantize_microscaled
    g8, g4 = lib.fp8_silu_mul_quantize_pertoken, lib.fp4_silu_mul_quantize_microscaled
    assert n8(None, None, FAKE, EPS, 4, 64, None, FAKE, FAKE, None, None) == _lib.SP24_ERR_NULL
    assert n8(FAKE, None, None, EPS, 4, 64, None, FAKE, FAKE, None, None) == _lib.SP24_ERR_NULL
    assert n8(FAKE, FAKE, FAKE, EPS, 4, 64, None, FAKE, FAKE, None, None) == _lib.SP24_ERR_NULL  # no residual_out
    assert n8(FAKE, None, FAKE, EPS, 4, 64, FAKE, FAKE, FAKE, None, None) == _lib.SP24_ERR_NULL  # no residual
    assert n8(FAKE, None, FAKE, EPS, 4, 64, None, FAKE, None, None, None) == _lib.SP24_ERR_NULL
    assert n8(FAKE, None, FAKE, None, 4, 64, None, FAKE, FAKE, None, None) == _lib.SP24_ERR_NULL
    assert n4(FAKE, None, FAKE, None, 4, 64, 0, None, FAKE, FAKE, FAKE, None, None) == _lib.SP24_ERR_NULL
    for eps in (-1e-6, float("nan"), float("inf")):
        assert n8(FAKE, None, FAKE, ctypes.byref(ctypes.c_float(eps)), 4, 64, None, FAKE, FAKE, None, None) == _lib.SP24_ERR_SHAPE
    assert n8(FAKE, None, FAKE, EPS, 4, 40, None, FAKE, FAKE, None, None) == _lib.SP24_ERR_SHAPE
    assert n8(FAKE, None, FAKE, EPS, 0, 64, None, FAKE, FAKE, None, None) == _lib.SP24_ERR_SHAPE
    assert n8(FAKE, ODD, FAKE, EPS, 4, 64, FAKE, FAKE, FAKE, None, None) == _lib.SP24_ERR_ALIGN
    assert n8(FAKE, FAKE, FAKE, EPS, 4, 64, ODD, FAKE, FAKE, None, None) == _lib.SP24_ERR_ALIGN
    assert n8(FAKE, None, ODD, EPS, 4, 64, None, FAKE, FAKE, None, None) == _lib.SP24_ERR_ALIGN
    assert n4(FAKE, None, FAKE, EPS, 4, 64, 7, None, FAKE, FAKE, FAKE, None, None) == _lib.SP24_ERR_DTYPE
    assert n4(FAKE, None, FAKE, EPS, 4, 64, -1, None, FAKE, FAKE, FAKE, None, None) == _lib.SP24_ERR_DTYPE
    assert n4(FAKE, None, FAKE, EPS, 4, 64, 0, None, FAKE, None, FAKE, None, None) == _lib.SP24_ERR_NULL
    assert n4(FAKE, None, FAKE, EPS, 4, 48, 0, None, FAKE, FAKE, FAKE, None, None) == _lib.SP24_ERR_SHAPE
    assert g8(FAKE, 4, 24, FAKE, FAKE, None, None) == _lib.SP24_ERR_SHAPE
    assert g8(FAKE, 4, 32, None, FAKE, None, None) == _lib.SP24_ERR_NULL
    assert g8(ODD, 4, 32, FAKE, FAKE, None, None) == _lib.SP24_ERR_ALIGN
    assert g4(FAKE, 4, 48, 1, FAKE, FAKE, None, None, None) == _lib.SP24_ERR_SHAPE
    assert g4(FAKE, 4, 64, 0, FAKE, FAKE, None, None, None) == _lib.SP24_ERR_NULL
    assert g4(FAKE, 4, 64, -1, FAKE, FAKE, FAKE, None, None) == _lib.SP24_ERR_DTYPE


def test_gemm_refusals(lib):
    g = lib.fp4_gemm_microscaled

    def call(xq=FAKE, xb=FAKE, xs=FAKE, wq=FAKE, wb=FAKE, ws=FAKE, fmt=0, y=FAKE, m=4, n=64, k=64):
        return g(xq, xb, xs, 1, wq, wb, ws, 1, fmt, y, m, n, k, None, None)

    assert call(fmt=2) == call(fmt=-1) == _lib.SP24_ERR_DTYPE
    for a in ("xq", "xb", "wq", "wb", "y"):
        assert call(**{a: None}) == _lib.SP24_ERR_NULL
        assert call(**{a: ODD}) == _lib.SP24_ERR_ALIGN
    for a in ("xs", "ws"):
        assert call(**{a: ODD}) == _lib.SP24_ERR_ALIGN
    for bad in (dict(m=0), dict(m=(1 << 31) - 1), dict(n=0), dict(n=(1 << 31) - 8), dict(n=12), dict(n=-8), dict(k=0), dict(k=32), dict(k=96), dict(k=-64)):
        assert call(**bad) == _lib.SP24_ERR_SHAPE


def test_gemm_refuses_sums_whose_stages_pass_an_int(lib):
    g = lib.fp4_gemm_microscaled
    for k in (1 << 31) - 64, (1 << 31) - 128, (1 << 31) - 192:
        assert g(FAKE, FAKE, FAKE, 1, FAKE, FAKE, FAKE, 1, 0, FAKE, 1, 8, k, None, None) == _lib.SP24_ERR_SHAPE
    # the longest sum passes the checks of shapes (and is refused for its alignment here)
    assert g(ODD, FAKE, FAKE, 1, FAKE, FAKE, FAKE, 1, 0, FAKE, 1, 8, (1 << 31) - 256, None, None) == _lib.SP24_ERR_ALIGN


DEVICE_STATE = r"""
#include "micro_kernels.h"
#include <cstdio>
static int current = 0, attributes = 0;
extern "C" cudaError_t cudaGetDevice(int *dev) { *dev = current; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void *, enum cudaFuncAttribute, int) { ++attributes; return cudaSuccess; }
static void kernel(int) {}
int main() {
  static sp24::DeviceNumbers<2> numbers;
  int asked = 0, n = 0;
  bool fails = true;
  auto ask = [&](int *v) { ++asked; *v = 10 * current + (current == 2 ? -20 : 3); return fails ? cudaErrorUnknown : cudaSuccess; };
  // a failure is reported, and not kept
  bool ok = numbers.get(0, &n, ask) == cudaErrorUnknown && asked == 1;
  fails = false;
  for (int i = 0; i < 3; ++i) ok &= numbers.get(0, &n, ask) == cudaSuccess && n == 3 && asked == 2;
  // another number and another device are asked for on their own
  ok &= numbers.get(1, &n, ask) == cudaSuccess && asked == 3;
  current = 1;
  ok &= numbers.get(0, &n, ask) == cudaSuccess && n == 13 && asked == 4;
  current = 2;  // a device that has none: known too
  for (int i = 0; i < 2; ++i) ok &= numbers.get(0, &n, ask) == cudaSuccess && n == 0 && asked == 5;
  current = 0;
  ok &= numbers.get(0, &n, ask) == cudaSuccess && n == 3 && asked == 5;
  // the allowance of shared memory, likewise once a device
  static std::atomic<uint64_t> ready{0};
  for (int d : {0, 1, 0, 1}) {
    current = d;
    ok &= sp24::allow_shared(kernel, 65536u, ready) == cudaSuccess;
  }
  ok &= attributes == 2;
  std::puts(ok ? "ok" : "wrong");
}
"""


def test_what_a_device_is_asked_is_kept_for_each_device(tmp_path):
    """Against fakes of the CUDA calls: a failed question is asked again, and
    one device's answer is not another's."""
    src = tmp_path / "state.cpp"
    src.write_text(DEVICE_STATE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(B.nvcc_path())), "include")
    subprocess.run(["g++", "-std=c++17", "-I", B.CSRC, "-I", B.INCLUDE, "-I", cuda, str(src), "-o", str(tmp_path / "state")],
                   check=True, capture_output=True, timeout=120)
    assert subprocess.run([str(tmp_path / "state")], capture_output=True, text=True, timeout=60).stdout == "ok\n"


# ------------------------------------------------------------------ Python
def test_python_refuses_cpu_tensors_and_unknown_formats(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    q = torch.zeros(4, 32, dtype=torch.uint8)
    s = torch.zeros(512, dtype=torch.uint8)
    for call in (lambda: sp.fp4_quantize_microscaled(x), lambda: sp.fp4_unpack_e4m3(q),
                 lambda: sp.fp8_rmsnorm_quantize_pertoken(x, w, 1e-5),
                 lambda: sp.fp4_rmsnorm_quantize_microscaled(x, w, 1e-5), lambda: sp.fp8_silu_mul_quantize_pertoken(x),
                 lambda: sp.fp4_silu_mul_quantize_microscaled(x),
                 lambda: sp.fp4_gemm_microscaled(q, s, None, q, s, None)):
        with pytest.raises(sp.Sp24Error):
            call()
    with pytest.raises(sp.Sp24Error, match="format"):
        sp.fp4_block_scales_size(4, 64, "fp4")
