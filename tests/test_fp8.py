"""8-bit rows and products and the gated feed-forward block on the CPU: the oracle's pins, the sizes
and every refusal (all of them return during argument validation: no pointer is dereferenced)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle as O
import post_weight_quantization_gq_amd as gq
from post_weight_quantization_gq_amd import binding as B
from _product_kernels import CASES, U8, kernel, types

FP8 = torch.float8_e4m3fn
FAR = [ctypes.c_void_p(i << 52) for i in range(1, 17)]      # apart, aligned, never dereferenced


def off(p, by):
    return ctypes.c_void_p(p.value + by)


def err():
    return gq.library().gq_last_error().decode()


# ---- the oracle -------------------------------------------------------------------------

def test_oracle_grid_is_the_types():
    """All 256 codes, by torch's reading of them; values and ties by its conversion."""
    every = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    ref = every.view(FP8).to(torch.float64).numpy()
    from oracle.fp8_oracle import _codes
    np.testing.assert_array_equal(O.code_values(every.numpy()), ref)
    g = O.FP8_GRID
    mid = (g[1:] + g[:-1]) / 2                 # every border between two codes, and beside it
    u = np.concatenate([g, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)])
    u = np.concatenate([u, -u])
    np.testing.assert_array_equal(_codes(u), torch.from_numpy(u).float().to(FP8).view(torch.uint8).numpy())


def test_oracle_scales():
    x = np.zeros((7, 130))
    x[0, 0], x[1, 5], x[2, 5], x[3, 0], x[4, 129] = 448.0, np.nextafter(448.0, 1000.0), 224.0, 2.0 ** -130, np.nan
    x[5, 0] = float(np.finfo(np.float32).max)
    Q, S = O.fp8_quantize(x)
    assert Q.shape == (7, 256) and S.shape == (7, 4)
    assert S[:, 0].tolist() == [127, 128, 126, 0, 0, 247, 0] and S[4, 1] == 255
    assert (S[:, 2:] == 127).all()
    assert Q[0, 0] == 126 and Q[2, 5] == 126
    v = O.fp8_values(Q, S, 130)
    assert v[0, 0] == 448.0 and v[2, 5] == 224.0 and v[5, 0] == 2.0 ** 128
    assert np.isnan(v[4, 128:]).all() and (v[4, :128] == 0).all()
    W = np.ones((129, 130))
    W[128, 129] = 1000.0
    Q, S = O.fp8_quantize_weight(W)
    assert Q.shape == (129, 256) and S.tolist() == [[119, 119], [119, 129]]
    assert O.fp8_weight_values(Q, S, 130)[128, 129] == 1024.0 and (Q[:, 130:] == 0).all()


def test_oracle_rounds_within_half_a_step():
    """Off by at most half a step: 2^-4 of a normal value, 2^-10 units below 2^-6 of them."""
    x = np.random.default_rng(0).standard_normal((64, 256)) * np.exp(2 * np.random.default_rng(1).standard_normal((64, 256)))
    Q, S = O.fp8_quantize(x)
    unit = np.repeat(np.ldexp(1.0, S[:, :2].astype(int) - 127), 128, axis=1)
    assert np.all(np.abs(O.fp8_values(Q, S, 256) - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * unit))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_oracle_activation_slopes_against_differences(act):
    z = np.linspace(-8, 8, 401)
    h = 1e-4
    diff = (O.ffn_act(z + h, act)[0] - O.ffn_act(z - h, act)[0]) / (2 * h)
    # |third derivative| < 4 throughout: the difference is off by at most 4 h^2 / 6, and by
    # rounding of values below 8 over 2 h
    assert np.max(np.abs(diff - O.ffn_act(z, act)[1])) <= 4 * h * h / 6 + 8 * 2.0 ** -50 / h
    t = torch.from_numpy(z)
    ref = {"silu": torch.nn.functional.silu(t), "gelu": torch.nn.functional.gelu(t),
           "gelu_tanh": torch.nn.functional.gelu(t, approximate="tanh")}[act].numpy()
    np.testing.assert_allclose(O.ffn_act(z, act)[0], ref, rtol=1e-12, atol=1e-14)


# ---- sizes ------------------------------------------------------------------------------

def test_sizes():
    assert [gq.fp8_row_bytes(d) for d in (1, 128, 129, 4096)] == [128, 128, 256, 4096]
    assert [gq.fp8_row_scales(d) for d in (1, 128, 512, 513, 4096)] == [4, 4, 4, 8, 32]
    for d in (0, -1, (1 << 20) + 1):
        assert gq.fp8_row_bytes(d) == 0 and gq.fp8_row_scales(d) == 0
    for size in (gq.fp8_gemm_workspace_size, gq.fp8_gemm_dx_workspace_size, gq.fp8_ffn_gate_workspace_size,
                 gq.fp8_ffn_gate_packed_workspace_size, gq.ffn_gate_workspace_size, gq.ffn_gate_dx_workspace_size):
        assert size(0, 4096, 4096) == 0 and size(8, 0, 4096) == 0 and size(8, 4096, 1 << 21) == 0
        assert size(8, 4096, 4096, 0) == 0 and size(1 << 31, 8, 8) == 0


def test_workspaces_over_the_sizes():
    """Every size has a plan (the host's arithmetic alone)."""
    for n in (1, 2, 15, 16, 17, 33, 64, 65, 129, 1000, 100000):
        for d_in in (1, 31, 128, 129, 1000, 1 << 20):
            for d_out in (1, 16, 1000, 70000):
                for experts in (1, 3, 4096):
                    for scales in (torch.uint8, torch.float32):
                        for size in (gq.fp8_gemm_workspace_size, gq.fp8_gemm_dx_workspace_size,
                                     gq.fp8_ffn_gate_workspace_size, gq.fp8_ffn_gate_packed_workspace_size):
                            assert size(n, d_in, d_out, experts, scales) % 256 == 0
                    for size in (gq.ffn_gate_workspace_size, gq.ffn_gate_dx_workspace_size, gq.ffn_gate_dw_workspace_size):
                        assert size(n, d_in, d_out, experts) % 256 == 0


# ---- refusals of the C entry points ------------------------------------------------------

def test_row_argument_errors():
    lib = gq.library()
    x0, q0, s0 = FAR[:3]
    for fn in (lambda x=x0, dt=1, rows=4, d=64, Q=q0, S=s0, sdt=0: lib.fp8_quantize(x, dt, rows, d, Q, S, sdt, None),
               lambda x=x0, dt=1, rows=4, d=64, Q=q0, S=s0, sdt=0: lib.fp8_dequantize(Q, S, sdt, rows, d, x, dt, None)):
        assert fn(x=None) == B.GQ_EINVAL and "null" in err()
        assert fn(Q=None) == B.GQ_EINVAL and fn(S=None) == B.GQ_EINVAL
        assert fn(dt=2) == B.GQ_EDTYPE and fn(sdt=2) == B.GQ_EDTYPE and fn(sdt=-1) == B.GQ_EDTYPE
        assert fn(rows=-1) == B.GQ_ESHAPE and fn(d=0) == B.GQ_ESHAPE
        assert fn(d=(1 << 20) + 1) == B.GQ_ENOTIMPL and fn(rows=1 << 40) == B.GQ_ENOTIMPL
        assert fn(Q=off(q0, 8)) == B.GQ_EINVAL and "aligned" in err()
        assert fn(S=off(s0, 2)) == B.GQ_EINVAL and fn(x=off(x0, 1)) == B.GQ_EINVAL
        assert fn(x=off(x0, 2), dt=0) == B.GQ_EINVAL
        assert fn(Q=x0) == B.GQ_EINVAL and "overlap" in err()
        assert fn(S=off(x0, 4)) == B.GQ_EINVAL and fn(S=off(q0, 508)) == B.GQ_EINVAL
        assert fn(rows=0, x=None, Q=None, S=None) == B.GQ_OK
    for fn in (lambda x=x0, dt=1, E=2, o=4, d=64, Q=q0, S=s0, sdt=0: lib.fp8_quantize_weight(x, dt, E, o, d, Q, S, sdt, None),
               lambda x=x0, dt=1, E=2, o=4, d=64, Q=q0, S=s0, sdt=0: lib.fp8_dequantize_weight(Q, S, sdt, E, o, d, x, dt, None)):
        assert fn(x=None) == B.GQ_EINVAL and fn(Q=None) == B.GQ_EINVAL and fn(S=None) == B.GQ_EINVAL
        assert fn(E=0) == B.GQ_EINVAL and fn(E=4097) == B.GQ_ENOTIMPL
        assert fn(o=0) == B.GQ_ESHAPE and fn(d=0) == B.GQ_ESHAPE
        assert fn(o=(1 << 20) + 1) == B.GQ_ENOTIMPL and fn(d=(1 << 20) + 1) == B.GQ_ENOTIMPL
        assert fn(o=1 << 20, d=1 << 20, E=2) == B.GQ_ENOTIMPL
        assert fn(dt=7) == B.GQ_EDTYPE and fn(sdt=2) == B.GQ_EDTYPE
        assert fn(Q=off(q0, 8)) == B.GQ_EINVAL and fn(S=off(s0, 2), sdt=1) == B.GQ_EINVAL
        assert fn(Q=x0) == B.GQ_EINVAL and "overlap" in err()


def _calls():
    """name -> a call of it with every argument by name; all have n, k (d_in), m (d_out or d_ff)."""
    lib = gq.library()
    a, aS, w, wS, u, uS, y, y2, o, wsp = FAR[:10]

    def gemm(n=8, k=256, m=128, a=a, aS=aS, w=w, wS=wS, y=y, ydt=1, sdt=0, experts=1, offsets=None, ws=None, wsb=0):
        return lib.fp8_gemm(a, aS, n, k, w, wS, sdt, m, experts, offsets, y, ydt, ws, wsb, None)

    def dx(n=8, k=256, m=128, a=a, aS=aS, w=w, wS=wS, y=y, ydt=1, sdt=0, experts=1, offsets=None, ws=None, wsb=0):
        return lib.fp8_gemm_dx(a, aS, n, m, w, wS, sdt, k, experts, offsets, y, ydt, ws, wsb, None)

    def gate8(n=8, k=256, m=128, a=a, aS=aS, w=w, wS=wS, u=u, uS=uS, y=y, ydt=1, sdt=0, act=0, experts=1, offsets=None, ws=None, wsb=0):
        return lib.fp8_ffn_gate(a, aS, n, k, w, wS, u, uS, sdt, m, act, experts, offsets, y, ydt, ws, wsb, None)

    def packed(n=8, k=256, m=128, a=a, aS=aS, w=w, wS=wS, u=u, uS=uS, y=y, y2=y2, sdt=0, act=0, experts=1, offsets=None, ws=None, wsb=0):
        return lib.fp8_ffn_gate_packed(a, aS, n, k, w, wS, u, uS, sdt, m, act, experts, offsets, y, y2, ws, wsb, None)

    def gate(n=8, k=256, m=128, a=a, w=w, u=u, y=y, ydt=1, zg=None, zu=None, act=0, experts=1, offsets=None, ws=None, wsb=0):
        return lib.ffn_gate(a, n, k, w, u, m, act, experts, offsets, y, ydt, zg, zu, ws, wsb, None)

    def gate_dx(n=8, k=256, m=128, a=a, a2=aS, w=w, u=u, y=y, ydt=1, experts=1, offsets=None, ws=None, wsb=0):
        return lib.ffn_gate_dx(a, a2, n, m, w, u, k, experts, offsets, y, ydt, ws, wsb, None)

    def gate_dw(n=8, k=256, m=128, a=a, a2=aS, w=w, y=y, y2=y2, ydt=1, experts=1, offsets=None, ws=None, wsb=0):
        return lib.ffn_gate_dw(a, a2, n, m, w, k, experts, offsets, y, y2, ydt, ws, wsb, None)

    return dict(gemm=gemm, dx=dx, gate8=gate8, packed=packed, gate=gate, gate_dx=gate_dx, gate_dw=gate_dw)


@pytest.mark.parametrize("name", ["gemm", "dx", "gate8", "packed", "gate", "gate_dx", "gate_dw"])
def test_product_argument_errors(name):
    call = _calls()[name]
    takes = call.__code__.co_varnames[:call.__code__.co_argcount]
    pointers = [p for p in ("a", "aS", "a2", "w", "wS", "u", "uS", "y") if p in takes]
    for p in pointers:
        if (name, p) != ("gate_dw", "y"):                  # either weight's gradient can be left out
            assert call(**{p: None}) == B.GQ_EINVAL and "null" in err(), p
        if p not in ("wS", "uS"):                          # (bytes)
            assert call(**{p: off(FAR[12], 1)}) == B.GQ_EINVAL and "aligned" in err(), p
    if "y2" in takes:
        assert call(y=None, y2=None) == B.GQ_EINVAL
    if "ydt" in takes:
        assert call(ydt=2) == B.GQ_EDTYPE and call(ydt=-1) == B.GQ_EDTYPE
        assert call(y=off(FAR[6], 1)) == B.GQ_EINVAL and call(y=off(FAR[6], 2), ydt=0) == B.GQ_EINVAL
    if "sdt" in takes:
        assert call(sdt=2) == B.GQ_EDTYPE and call(sdt=-1) == B.GQ_EDTYPE
        assert call(aS=off(FAR[1], 2)) == B.GQ_EINVAL and "aligned" in err()
        assert call(wS=off(FAR[3], 2), sdt=1) == B.GQ_EINVAL and "aligned" in err()
    if "act" in takes:
        assert call(act=3) == B.GQ_EINVAL and "activation" in err()
        assert call(act=-1) == B.GQ_EINVAL
    if "zg" in takes:
        assert call(zg=FAR[10]) == B.GQ_EINVAL and "both" in err()
        assert call(zg=FAR[10], zu=off(FAR[11], 2)) == B.GQ_EINVAL
        assert call(zg=FAR[10], zu=off(FAR[10], 4 * 8 * 128 - 4)) == B.GQ_EINVAL and "overlap" in err()
    assert call(n=-1) == B.GQ_ESHAPE and call(k=0) == B.GQ_ESHAPE and call(m=0) == B.GQ_ESHAPE
    assert call(n=1 << 31) == B.GQ_ENOTIMPL
    assert call(k=(1 << 20) + 1) == B.GQ_ENOTIMPL and call(m=(1 << 20) + 1) == B.GQ_ENOTIMPL
    assert call(experts=0) == B.GQ_EINVAL and "experts" in err()
    assert call(experts=4097, offsets=FAR[8]) == B.GQ_ENOTIMPL
    assert call(experts=2) == B.GQ_EINVAL and "offsets" in err()
    assert call(experts=2, offsets=off(FAR[8], 4)) == B.GQ_EINVAL and "aligned" in err()
    assert call(a=off(FAR[0], 8)) == B.GQ_EINVAL and "aligned" in err()
    assert call(w=off(FAR[2], 8)) == B.GQ_EINVAL and "aligned" in err()
    assert call(ws=off(FAR[9], 8), wsb=1 << 30) == B.GQ_EINVAL and "ws" in err()
    assert call(y=FAR[0]) == B.GQ_EINVAL and "overlap" in err()
    assert call(y=off(FAR[2], 256)) == B.GQ_EINVAL and "overlap" in err()
    assert call(offsets=FAR[6]) == B.GQ_EINVAL and "overlap" in err()
    if name != "gate_dw":                                  # (no rows: gradients of zero)
        assert call(n=0, a=None, w=None, y=None) == B.GQ_OK
    assert call(n=0, k=0) == B.GQ_ESHAPE


def test_dz_argument_errors():
    lib = gq.library()

    def call(dh=FAR[0], dt=1, zg=FAR[1], zu=FAR[2], count=64, act=0, a=FAR[3], b=FAR[4]):
        return lib.ffn_gate_dz(dh, dt, zg, zu, count, act, a, b, None)

    for p in ("dh", "zg", "zu", "a", "b"):
        assert call(**{p: None}) == B.GQ_EINVAL and "null" in err()
    assert call(dt=5) == B.GQ_EDTYPE and call(count=-1) == B.GQ_ESHAPE and call(count=(1 << 34) + 1) == B.GQ_ENOTIMPL
    assert call(act=3) == B.GQ_EINVAL and call(act=-1) == B.GQ_EINVAL
    assert call(dh=off(FAR[0], 1)) == B.GQ_EINVAL and call(zg=off(FAR[1], 2)) == B.GQ_EINVAL
    assert call(b=off(FAR[4], 1)) == B.GQ_EINVAL
    assert call(a=FAR[4]) == B.GQ_EINVAL and "overlap" in err()
    assert call(a=off(FAR[1], 4)) == B.GQ_EINVAL and call(b=FAR[0]) == B.GQ_EINVAL
    assert call(count=0, dh=None, zg=None, zu=None, a=None, b=None) == B.GQ_OK


def test_backward_argument_errors():
    lib = gq.library()
    names = "dh x G U zg zu dx dG dU".split()

    def call(dt=1, n=8, k=256, m=128, act=0, experts=1, offsets=None, dxt=1, dwt=1, ws=None, wsb=0, **p):
        p = {name: p.get(name, FAR[i]) for i, name in enumerate(names)}
        return lib.ffn_gate_backward(p["dh"], dt, p["x"], n, k, p["G"], p["U"], m, act, experts, offsets, p["zg"], p["zu"],
                                     p["dx"], dxt, p["dG"], p["dU"], dwt, ws, wsb, None)

    for p in names[:6]:
        assert call(**{p: None}) == B.GQ_EINVAL and "null" in err(), p
    none = dict(dx=None, dG=None, dU=None)
    assert call(**none) == B.GQ_EINVAL and "nothing" in err()
    assert call(**none, n=0) == B.GQ_EINVAL
    # what an output does not need can be left out: these get as far as the overlap of what is there
    assert call(dx=None, G=None, U=None, dU=FAR[0]) == B.GQ_EINVAL and "overlap" in err()
    assert call(dG=None, dU=None, x=None, dx=FAR[0]) == B.GQ_EINVAL and "overlap" in err()
    assert call(dt=2) == B.GQ_EDTYPE and call(dxt=2) == B.GQ_EDTYPE and call(dwt=-1) == B.GQ_EDTYPE
    assert call(act=3) == B.GQ_EINVAL and call(act=-1) == B.GQ_EINVAL
    assert call(n=-1) == B.GQ_ESHAPE and call(k=0) == B.GQ_ESHAPE and call(m=0) == B.GQ_ESHAPE
    assert call(n=1 << 31) == B.GQ_ENOTIMPL and call(k=(1 << 20) + 1) == B.GQ_ENOTIMPL and call(m=(1 << 20) + 1) == B.GQ_ENOTIMPL
    assert call(experts=0) == B.GQ_EINVAL and call(experts=2) == B.GQ_EINVAL and "offsets" in err()
    assert call(experts=4097, offsets=FAR[10]) == B.GQ_ENOTIMPL
    assert call(offsets=off(FAR[10], 4)) == B.GQ_EINVAL
    assert call(dh=off(FAR[0], 1)) == B.GQ_EINVAL and call(dh=off(FAR[0], 2), dt=0) == B.GQ_EINVAL
    for p in ("x", "G", "U"):
        assert call(**{p: off(FAR[12], 8)}) == B.GQ_EINVAL and "aligned" in err()
        assert call(**{p: off(FAR[12], 8)}, k=257, dx=FAR[0]) == B.GQ_EINVAL and "overlap" in err()
    assert call(zg=off(FAR[4], 2)) == B.GQ_EINVAL and call(dx=off(FAR[6], 1)) == B.GQ_EINVAL
    assert call(dU=off(FAR[8], 2), dwt=0) == B.GQ_EINVAL and call(ws=off(FAR[10], 8), wsb=1 << 30) == B.GQ_EINVAL
    for a in ("dx", "dG", "dU"):
        for b in names:
            if a != b:
                assert call(**{a: FAR[names.index(b)]}) == B.GQ_EINVAL and "overlap" in err(), (a, b)
    assert call(n=0, dG=None, dU=None) == B.GQ_OK
    need = gq.ffn_gate_backward_workspace_size(8, 256, 128)
    assert need >= 2 * 8 * 128 * 2 and gq.ffn_gate_backward_workspace_size(8, 256, 129) >= 2 * 8 * 136 * 2
    assert call(ws=FAR[10], wsb=need - 1) == B.GQ_EINVAL and "workspace" in err()
    assert gq.ffn_gate_backward_workspace_size(0, 256, 128) >= 0 and gq.ffn_gate_backward_workspace_size(8, 0, 128) == 0


# ---- refusals of the binding --------------------------------------------------------------

def status(fn, *a, **k):
    with pytest.raises(B.GQError) as e:
        fn(*a, **k)
    return e.value.status


def test_binding_refusals():
    """Shapes, dtypes and devices are checked before any launch: these CPU tensors never reach
    a kernel."""
    u8, bf = torch.uint8, torch.bfloat16
    x = torch.zeros(5, 200, dtype=bf)
    XQ, XS = torch.zeros(5, 256, dtype=u8).view(FP8), torch.zeros(5, 4, dtype=u8)
    Q, S = torch.zeros(64, 256, dtype=u8).view(FP8), torch.zeros(1, 2, dtype=u8)
    GQ = torch.zeros(5, 128, dtype=u8).view(FP8)
    at = torch.zeros(3, dtype=torch.int64)
    assert status(gq.fp8_quantize, torch.zeros(4, 0)) == B.GQ_ESHAPE
    assert status(gq.fp8_quantize, torch.zeros(())) == B.GQ_ESHAPE
    assert status(gq.fp8_quantize, x, Q=Q) == B.GQ_ESHAPE
    assert status(gq.fp8_quantize, x, scales=bf) == B.GQ_EDTYPE
    assert status(gq.fp8_quantize, x, S=XS, scales=torch.float32) == B.GQ_EDTYPE
    assert status(gq.fp8_quantize, x) == B.GQ_EINVAL                     # host tensor
    assert status(gq.fp8_quantize_weight, x[0]) == B.GQ_ESHAPE
    assert status(gq.fp8_quantize_weight, x, S=XS) == B.GQ_ESHAPE
    assert status(gq.fp8_quantize_weight, x) == B.GQ_EINVAL
    assert status(gq.fp8_dequantize, XQ, XS, 300) == B.GQ_ESHAPE
    assert status(gq.fp8_dequantize, XQ, XS, 200, dtype=u8) == B.GQ_EDTYPE
    assert status(gq.fp8_dequantize, XQ, XS, 200) == B.GQ_EINVAL
    assert status(gq.fp8_dequantize_weight, Q, XS, 200) == B.GQ_ESHAPE
    assert status(gq.fp8_dequantize_weight, Q, S, 200) == B.GQ_EINVAL
    assert status(gq.fp8_gemm, XQ[0], XS[0], Q, S, 200) == B.GQ_ESHAPE
    assert status(gq.fp8_gemm, XQ, XS, Q, S, 300) == B.GQ_ESHAPE
    assert status(gq.fp8_gemm, XQ, XS, Q, S, 200) == B.GQ_EINVAL         # host tensors
    assert status(gq.fp8_gemm_dx, XQ, XS, Q, S, 200) == B.GQ_ESHAPE      # 64 outputs: rows of 128
    assert status(gq.fp8_gemm_dx, GQ, XS, Q, S, 200, offsets=at) == B.GQ_ESHAPE
    assert status(gq.fp8_gemm_dx, GQ, XS, Q, S, 200) == B.GQ_EINVAL
    assert status(gq.fp8_ffn_gate, XQ, XS, Q, S, Q, S, 200, act="relu") == B.GQ_EINVAL
    assert status(gq.fp8_ffn_gate, XQ, XS, Q, S, Q, S, 200) == B.GQ_EINVAL
    G = torch.zeros(64, 200, dtype=bf)
    assert status(gq.ffn_gate, x, G, G, act="tanh") == B.GQ_EINVAL
    assert status(gq.ffn_gate, x[0], G, G) == B.GQ_ESHAPE
    assert status(gq.ffn_gate, x, G[0], G) == B.GQ_ESHAPE
    assert status(gq.ffn_gate, x, G, G[:32]) == B.GQ_ESHAPE
    assert status(gq.ffn_gate, x, G, G, offsets=at) == B.GQ_ESHAPE
    assert status(gq.ffn_gate, x, G, G) == B.GQ_EINVAL
    leaf = x.clone().requires_grad_()
    assert status(gq.ffn_gate, leaf, G, G, save=True) == B.GQ_EINVAL
    assert status(gq.ffn_gate, leaf, G, G, y=torch.zeros(5, 64)) == B.GQ_EINVAL
    assert status(gq.ffn_gate, leaf, G, G) == B.GQ_EINVAL
    z = torch.zeros(5, 64)
    assert status(gq.ffn_gate_dz, z, z[:4], z) == B.GQ_ESHAPE
    assert status(gq.ffn_gate_dz, z, z, z) == B.GQ_EINVAL
    assert status(gq.ffn_gate_dx, z[0], z, G, G) == B.GQ_ESHAPE
    assert status(gq.ffn_gate_dx, z, z[:4], G, G) == B.GQ_ESHAPE
    assert status(gq.ffn_gate_dw, z, z, x, experts=2) == B.GQ_EINVAL
    assert status(gq.ffn_gate_dw, z, z, x) == B.GQ_EINVAL


def test_stages_of_the_library_and_the_binding():
    lib = gq.library()
    assert len(B.PRODUCT_STAGES) == B.PRODUCT_STAGE_COUNT
    assert lib.gq_timing_read_product(None, None) == B.GQ_EINVAL
    ms, n = (ctypes.c_double * 4)(*[5.0] * 4), (ctypes.c_int64 * 4)(*[7] * 4)
    assert lib.gq_timing_read_product(ms, n) == B.GQ_OK and list(ms) == [0.0] * 4 and list(n) == [0] * 4
    assert math.isclose(sum(ms), 0.0)


# ---- how products are done --------------------------------------------------------------

def test_the_kernels_cases_reach_every_kernel():
    """Whatever a sweep over rows, widths, experts and types can choose is run by a case of the kernels' tests."""
    rows = (1, 2, 8, 16, 17, 32, 33, 64, 100, 129, 200, 257, 333, 512, 700, 1024, 1500, 2048, 4096, 8192, 20000)
    widths = (32, 64, 200, 512, 640, 1000, 1100, 2048, 4096, 5000, 8192, 11008, 28672, 100000)
    missing = {}
    for op in B.PRODUCTS:
        for t in types(op):
            covered = {kernel(op, *c, *t) for c in CASES[op]}
            for n in rows:
                for d_in in widths:
                    for d_out in widths:
                        for experts in (None, 2, 8, 64, 300):
                            if (experts or 1) * d_in * d_out > 1 << 37:          # weights past a card's memory
                                continue
                            k = kernel(op, n, d_in, d_out, experts, *t)
                            if k not in covered:
                                missing.setdefault(k, (n, d_in, d_out, experts))
    assert not missing


@pytest.mark.parametrize("op", B.PRODUCTS)
def test_parts_and_workspaces_stay_small(op):
    """A split contraction's float32 parts: no more than a few hundred tiles' of 256 x 256."""
    size = getattr(gq, op + "_workspace_size")
    for n in (1, 16, 100, 1000, 4096, 65536):
        for d_in in (128, 4096, 28672):
            for d_out in (128, 4096, 28672):
                for experts in (1, 8, 256):
                    extra = () if op.startswith("ffn") else (U8,) if op.endswith("packed") else (U8, gq.GQ_F32)
                    p = gq.product_plan(op, n, d_in, d_out, experts, dtype=gq.GQ_F32)
                    assert 1 <= p["split"] <= 16
                    outputs = n * d_out * (1 + ("gate" in op)) * 4
                    if p["split"] > 1:
                        assert size(n, d_in, d_out, experts, *extra) <= 16 * 512 * 256 * 256 * 4
                    elif not op.endswith("packed"):
                        assert size(n, d_in, d_out, experts, *extra) == 0, (n, d_in, d_out, experts)
                    else:
                        assert size(n, d_in, d_out, experts, *extra) <= outputs + 256


@pytest.mark.parametrize("op,n,d_in,d_out,experts", [
    ("fp8_gemm", (1 << 31) - 1, 8, 1, 1), ("fp8_gemm", 4096, 128, 1 << 19, 4096), ("fp8_gemm_dx", (1 << 31) - 1, 1, 8, 1),
    ("fp8_ffn_gate", 4096, 128, 1 << 19, 4096), ("ffn_gate", 1 << 30, 8, 1 << 10, 1), ("ffn_gate_dx", 1 << 30, 1 << 10, 8, 1),
    ("ffn_gate_dw", 1, 1 << 19, 1 << 19, 64)])
def test_more_tiles_than_a_launch_takes(op, n, d_in, d_out, experts):
    """Refused by the sizes, and the largest sizes that are not have a plan."""
    with pytest.raises(gq.GQError) as e:
        gq.product_plan(op, n, d_in, d_out, experts)
        gq.product_plan(op, (1 << 31) - (1 << 21) - 1, d_in, d_out, experts)
    assert e.value.status == B.GQ_ENOTIMPL


def test_plan_refusals():
    lib = gq.library()
    plan = (ctypes.c_int32 * 6)()

    def status(op=0, s=0, dt=1, n=8, d_in=128, d_out=128, experts=1, plan=plan):
        return lib.gq_product_plan(op, s, dt, n, d_in, d_out, experts, plan)

    assert status() == B.GQ_OK and list(plan) == [0, 1, 16, 16, 4, 1]
    assert status(dt=0) == B.GQ_OK and list(plan)[:2] == [1, 1]
    assert status(op=-1) == B.GQ_EINVAL and status(op=7) == B.GQ_EINVAL and status(plan=None) == B.GQ_EINVAL
    assert status(s=2) == B.GQ_EDTYPE and status(op=4, s=2) == B.GQ_OK
    assert status(dt=2) == B.GQ_EDTYPE and status(op=3, dt=2) == B.GQ_OK
    assert status(n=0) == B.GQ_ESHAPE and status(d_in=0) == B.GQ_ESHAPE and status(d_out=-1) == B.GQ_ESHAPE
    assert status(n=1 << 31) == B.GQ_ENOTIMPL and status(d_in=(1 << 20) + 1) == B.GQ_ENOTIMPL
    assert status(experts=0) == B.GQ_EINVAL and status(experts=4097) == B.GQ_ENOTIMPL
    with pytest.raises(ValueError):
        gq.product_plan("gemv", 8, 128, 128)
    with pytest.raises(gq.GQError):
        gq.product_plan("fp8_gemm", 8, 0, 128)
