"""MXFP4 on the CPU: the oracle's pins, the sizes, and every refusal of the entry points
(all of them return during argument validation, so no pointer is dereferenced)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle as O
import post_weight_quantization_gq_amd as gq
from post_weight_quantization_gq_amd import binding as B

FAKE = ctypes.c_void_p(0x10000)      # aligned, never dereferenced (validation fails first)
FAKE_ODD = ctypes.c_void_p(0x10008)  # 8-byte aligned only


def test_oracle_grid_ties_and_saturation():
    """One block whose maximum 6 gives the scale 1: ties go to the even index, values over 5
    (up to the block's maximum below 8) to 6, signs are kept."""
    x = np.zeros((1, 32))
    x[0, :14] = [6.0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, 7.9, -0.2, -0.75, -6.0]
    want = [6.0, 0.0, 0.5, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 6.0, 0.0, -1.0, -6.0]
    Q, S = O.mx_quantize(x)
    assert Q.shape == (1, 64) and S.shape == (1, 4)
    assert S.tolist() == [[127, 127, 127, 127]]
    v = O.mx_values(Q, S, 32)
    np.testing.assert_array_equal(v[0, :14], want)
    assert np.signbit(v[0, 11])
    assert Q[0, 0] == 7 and Q[0, 4] == (7 << 4 | 6)      # 6.0 | 0.25, and 5.0 | 5.1


def test_oracle_scales():
    x = np.zeros((6, 40))
    x[1, 0], x[2, 0], x[3, 0], x[4, 0], x[5, 35] = 2.0 ** 127 * 1.99, 2.0 ** -126, 1e-45, np.inf, np.nan
    Q, S = O.mx_quantize(x)
    assert S[:, 0].tolist() == [0, 252, 0, 0, 255, 0]
    assert S[:, 1].tolist() == [0, 0, 0, 0, 0, 255]
    assert (S[:, 2:] == 127).all() and (Q[:, 20:] == 0).all()
    v = O.mx_values(Q, S, 40)
    assert v[1, 0] == 6 * 2.0 ** 125 and v[2, 0] == 2.0 ** -126 and v[3, 0] == 0.0
    assert np.isnan(v[4, :32]).all() and (v[4, 32:] == 0).all() and np.isnan(v[5, 32:]).all()


def test_oracle_rounds_within_half_a_step():
    """Away from saturation a value is off by at most a quarter of its magnitude's binade: half
    a step of a one-bit mantissa, 2^-2 relative to normal values, 0.25 units below 1."""
    x = np.random.default_rng(0).standard_normal((64, 96))
    v = O.mx_values(*O.mx_quantize(x), 96)
    unit = np.repeat(2.0 ** np.floor(np.log2(np.abs(x.reshape(64, 3, 32)).max(2))) / 4, 32, axis=1)
    u = np.abs(x) / unit
    ok = u <= 6.0
    assert np.all(np.abs(v - x)[ok] <= np.maximum(0.25 * unit, 0.25 * np.abs(x))[ok])
    np.testing.assert_array_equal(np.abs(v)[~ok], 6.0 * unit[~ok])


def test_sizes():
    assert [gq.mxfp4_row_bytes(d) for d in (1, 128, 129, 4096)] == [64, 64, 128, 2048]
    assert [gq.mxfp4_row_scales(d) for d in (1, 128, 129, 4096)] == [4, 4, 8, 128]
    for d in (0, -1, (1 << 20) + 1):
        assert gq.mxfp4_row_bytes(d) == 0 and gq.mxfp4_row_scales(d) == 0
    # bad sizes need nothing; float32 activations need their planes
    assert gq.mxfp4_gemm_workspace_size(0, 4096, 4096) == 0
    assert gq.mxfp4_gemm_workspace_size(8, 0, 4096) == 0
    assert gq.mxfp4_gemm_mx_workspace_size(8, 4096, 1 << 21) == 0
    assert gq.mxfp4_gemm_dx_workspace_size(8, 4096, 4096, 0) == 0


def test_workspaces_over_the_sizes():
    """Every size has a plan (the host's arithmetic alone), small ones and float32 ones too."""
    for n in (1, 2, 15, 16, 17, 33, 64, 65, 129, 1000, 100000):
        for d_in in (1, 31, 128, 129, 1000, 1 << 20):
            for d_out in (1, 16, 1000, 70000):
                for experts in (1, 3, 4096):
                    for dt in (gq.GQ_BF16, gq.GQ_F32):
                        a = gq.mxfp4_gemm_workspace_size(n, d_in, d_out, experts, dt)
                        b = gq.mxfp4_gemm_dx_workspace_size(n, d_in, d_out, experts, dt)
                        assert a % 256 == 0 and b % 256 == 0
                        if dt == gq.GQ_F32:          # three planes of two bytes
                            assert a >= 6 * n * d_in and b >= 6 * n * d_out
                    assert gq.mxfp4_gemm_mx_workspace_size(n, d_in, d_out, experts) % 256 == 0


def _err():
    return gq.library().gq_last_error().decode()


def test_quantize_argument_errors():
    lib = gq.library()
    for fn in (lambda **k: lib.mxfp4_quantize(k.get("x", FAKE), k.get("dt", 1), k.get("rows", 4),
                                              k.get("d", 64), k.get("Q", FAKE), k.get("S", FAKE), None),
               lambda **k: lib.mxfp4_dequantize(k.get("Q", FAKE), k.get("S", FAKE), k.get("rows", 4),
                                                k.get("d", 64), k.get("x", FAKE), k.get("dt", 1), None)):
        assert fn(x=None) == B.GQ_EINVAL and "null" in _err()
        assert fn(S=None) == B.GQ_EINVAL
        assert fn(dt=2) == B.GQ_EDTYPE
        assert fn(rows=-1) == B.GQ_ESHAPE
        assert fn(d=0) == B.GQ_ESHAPE
        assert fn(d=(1 << 20) + 1) == B.GQ_ENOTIMPL
        assert fn(rows=1 << 40) == B.GQ_ENOTIMPL
        assert fn(Q=FAKE_ODD) == B.GQ_EINVAL and "aligned" in _err()
        assert fn(S=ctypes.c_void_p(0x10002)) == B.GQ_EINVAL
        assert fn(x=ctypes.c_void_p(0x10001)) == B.GQ_EINVAL
        assert fn() == B.GQ_EINVAL and "overlap" in _err()         # all one address
        assert fn(rows=0, x=None, Q=None, S=None) == B.GQ_OK


@pytest.mark.parametrize("name", ["mxfp4_gemm", "mxfp4_gemm_mx", "mxfp4_gemm_dx"])
def test_product_argument_errors(name):
    lib = gq.library()

    def call(x=FAKE, xs=FAKE, dt=1, n=8, k=256, Q=FAKE, S=FAKE, m=128, experts=1, offsets=None,
             y=FAKE, ydt=1, ws=None, wsb=0):
        first = (x, xs) if name == "mxfp4_gemm_mx" else (x, dt)
        return getattr(lib, name)(*first, n, k, Q, S, m, experts, offsets, y, ydt, ws, wsb, None)

    assert call(x=None) == B.GQ_EINVAL and "null" in _err()
    assert call(Q=None) == B.GQ_EINVAL
    assert call(S=None) == B.GQ_EINVAL
    assert call(y=None) == B.GQ_EINVAL
    if name == "mxfp4_gemm_mx":
        assert call(xs=None) == B.GQ_EINVAL
        assert call(xs=ctypes.c_void_p(0x10002)) == B.GQ_EINVAL
    else:
        assert call(dt=3) == B.GQ_EDTYPE
        assert call(x=ctypes.c_void_p(0x10002), dt=0, k=33) == B.GQ_EINVAL
    assert call(ydt=-1) == B.GQ_EDTYPE
    assert call(n=-1) == B.GQ_ESHAPE
    assert call(k=0) == B.GQ_ESHAPE
    assert call(m=0) == B.GQ_ESHAPE
    assert call(n=1 << 31) == B.GQ_ENOTIMPL
    assert call(k=(1 << 20) + 1) == B.GQ_ENOTIMPL
    assert call(m=(1 << 20) + 1) == B.GQ_ENOTIMPL
    assert call(experts=0) == B.GQ_EINVAL and "experts" in _err()
    assert call(experts=4097, offsets=FAKE) == B.GQ_ENOTIMPL
    assert call(experts=2) == B.GQ_EINVAL and "offsets" in _err()
    assert call(experts=2, offsets=ctypes.c_void_p(0x10004)) == B.GQ_EINVAL
    assert call(x=FAKE_ODD) == B.GQ_EINVAL and "aligned" in _err()
    assert call(Q=FAKE_ODD) == B.GQ_EINVAL
    assert call(S=ctypes.c_void_p(0x10002)) == B.GQ_EINVAL
    assert call(y=ctypes.c_void_p(0x10001)) == B.GQ_EINVAL
    assert call(y=ctypes.c_void_p(0x10002), ydt=0) == B.GQ_EINVAL
    assert call(ws=FAKE_ODD, wsb=1 << 30) == B.GQ_EINVAL and "ws" in _err()
    # the output on the inputs (every pointer here is the same address)
    assert call() == B.GQ_EINVAL and "overlap" in _err()
    far = [ctypes.c_void_p(i << 32) for i in range(1, 6)]
    assert call(x=far[0], xs=far[1], Q=far[2], S=far[3], y=far[0]) == B.GQ_EINVAL and "overlap" in _err()
    assert call(x=far[0], xs=far[1], Q=far[2], S=far[3], y=ctypes.c_void_p((3 << 32) + 256)) == B.GQ_EINVAL
    assert call(x=far[0], xs=far[1], Q=far[2], S=far[3], y=far[4], experts=1, offsets=far[4]) == B.GQ_EINVAL
    if name != "mxfp4_gemm_mx":                       # float32: a workspace, here too small, then on x
        assert call(x=far[0], dt=0, Q=far[2], S=far[3], y=far[4], ws=far[1], wsb=16) == B.GQ_EINVAL
        assert "too small" in _err()
        assert call(x=far[0], dt=0, Q=far[2], S=far[3], y=far[4], ws=far[0], wsb=1 << 30) == B.GQ_EINVAL
        assert "overlap" in _err()
    assert call(n=0, x=None, Q=None, S=None, y=None) == B.GQ_OK
    # no rows and bad sizes: still refused
    assert call(n=0, k=0) == B.GQ_ESHAPE


def test_binding_refusals():
    """Shapes, dtypes and devices are checked before any launch: these CPU tensors never reach
    a kernel."""
    u8 = torch.uint8
    x = torch.zeros(5, 200, dtype=torch.bfloat16)
    Q, S = torch.zeros(64, 128, dtype=u8), torch.zeros(64, 8, dtype=u8)
    XQ, XS = torch.zeros(5, 128, dtype=u8), torch.zeros(5, 8, dtype=u8)
    off = torch.zeros(3, dtype=torch.int64)

    def status(fn, *a, **k):
        with pytest.raises(B.GQError) as ei:
            fn(*a, **k)
        return ei.value.status

    assert status(gq.mxfp4_quantize, torch.zeros(4, 0)) == B.GQ_ESHAPE
    assert status(gq.mxfp4_quantize, torch.zeros(())) == B.GQ_ESHAPE
    assert status(gq.mxfp4_quantize, x, Q=Q) == B.GQ_ESHAPE
    assert status(gq.mxfp4_quantize, x) == B.GQ_EINVAL                   # host tensor
    assert status(gq.mxfp4_dequantize, XQ, XS, 300) == B.GQ_ESHAPE
    assert status(gq.mxfp4_gemm, x[0], Q, S) == B.GQ_ESHAPE
    assert status(gq.mxfp4_gemm, x[:, :100], Q, S) == B.GQ_ESHAPE
    assert status(gq.mxfp4_gemm, x, Q, S[:, :4]) == B.GQ_ESHAPE
    assert status(gq.mxfp4_gemm, x, Q, S, offsets=off) == B.GQ_ESHAPE    # one weight
    assert status(gq.mxfp4_gemm, x, Q[None], S[None]) == B.GQ_ESHAPE     # several, no offsets
    assert status(gq.mxfp4_gemm_mx, XQ[0], XS[0], Q, S, 200) == B.GQ_ESHAPE
    assert status(gq.mxfp4_gemm_mx, XQ, XS, Q, S, 128) == B.GQ_ESHAPE
    assert status(gq.mxfp4_gemm_dx, x, Q, S, 100) == B.GQ_ESHAPE
    assert status(gq.mxfp4_gemm, x, Q, S) == B.GQ_EINVAL                 # host tensors
