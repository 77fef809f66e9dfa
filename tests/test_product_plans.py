"""How 8-bit products and those of the gated feed-forward block are planned, from their sizes alone."""
import ctypes

import pytest

import post_weight_quantization_gq_amd as gq
from post_weight_quantization_gq_amd import binding as B


@pytest.mark.parametrize("op", ["fp8_gemm", "fp8_ffn_gate", "fp8_ffn_gate_packed", "ffn_gate"])
def test_every_part_of_a_streamed_contraction_has_a_line(op):
    """A line is 128 bytes of a weight's row; the waves of all parts take equal runs of them, the last ones what is left."""
    split = set()
    for n in (1, 8, 16):
        for d_in in [*range(1100, 34000, 100), *range(2048, 33000, 128), 65536, 100000, 131072]:
            lines = -(-d_in // (64 if op == "ffn_gate" else 128))
            for d_out in (1, 130, 256, 512, 1000, 2048, 4100):
                for experts in (1, 4):
                    p = gq.product_plan(op, n, d_in, d_out, experts, dtype=gq.GQ_F32)
                    if p["streamed"]:
                        run = -(-lines // (p["waves"] * p["split"]))
                        assert (p["split"] - 1) * p["waves"] * run < lines, (n, d_in, d_out, experts)
                        split.add(p["split"])
    assert len(split) > 4 and max(split) <= 16


@pytest.mark.parametrize("op", ["gemm", "gemm_mx"])
def test_every_part_of_a_streamed_mxfp4_contraction_has_a_piece(op):
    """A piece is 512 values of a row, 256 where the activations are three planes."""
    split = set()
    for n in (1, 8, 16):
        for d_in in [*range(1100, 34000, 100), *range(2048, 33000, 128), 65536, 100000]:
            for d_out in (1, 130, 256, 512, 1000, 2048, 4100):
                for dtype in (gq.GQ_F32, gq.GQ_BF16):
                    p = gq.mxfp4_plan(op, n, d_in, d_out, dtype=dtype)
                    if p["streamed"]:
                        pieces = -(-d_in // (256 if p["planes"] == 3 else 512))
                        run = -(-pieces // (p["waves"] * p["split"]))
                        assert (p["split"] - 1) * p["waves"] * run < pieces or p["split"] == 1, (n, d_in, d_out, dtype)
                        split.add(p["split"])
    assert len(split) > 3


BLOCKS = {8: (1 << 23) - 8, 4: (1 << 24) - 8}              # of 64 lanes a wave, in eights: fewer than 2^32 lanes


def _most(rows, cols, waves, experts=1):
    """The most rows that tiles of `rows` rows in `cols` columns of them take (an expert's last tile can be part-empty)."""
    return (BLOCKS[waves] // cols - (experts if experts > 1 else 0)) * rows


LIMITS = [                                                 # op, d_in, d_out, experts, float32 output, the most rows
    ("fp8_gemm", 8, 1, 1, False, _most(128, 1, 4)), ("fp8_gemm_dx", 1, 8, 1, False, _most(256, 1, 8)),
    ("fp8_gemm_dx", 1, 8, 64, False, _most(256, 1, 8, 64)), ("fp8_gemm_dx", 1, 8, 64, True, _most(128, 1, 8, 64)),
    ("fp8_ffn_gate", 8, 1 << 10, 1, False, _most(256, 8, 8)), ("fp8_ffn_gate", 8, 1 << 10, 1, True, _most(128, 8, 8)),
    ("fp8_ffn_gate_packed", 8, 1 << 10, 1, True, _most(128, 8, 8)),
    ("ffn_gate", 8, 1 << 10, 1, False, _most(256, 8, 8)), ("ffn_gate", 8, 1 << 10, 64, True, _most(256, 8, 8, 64)),
    ("ffn_gate_dx", 1 << 10, 8, 1, False, _most(256, 4, 8)),
    # eight rows an expert on average are streamed; by tiles they would be too many
    ("fp8_gemm", 128, 1 << 19, 4096, False, 8 * 4096), ("fp8_ffn_gate", 128, 1 << 19, 4096, True, 8 * 4096)]


def _far(i):
    return ctypes.c_void_p(i << 56)                        # apart, aligned, never dereferenced


def _call(op, n, d_in, d_out, experts, dtype):
    """Status and message of a call whose output lies on its rows, which is refused after every check of the sizes: it never
    gets as far as a launch."""
    lib = gq.library()
    at, none = (_far(9) if experts > 1 else None), (None, 0, None)
    a, w, u, y = (_far(1), _far(2)), (_far(3), _far(4)), (_far(5), _far(6)), _far(1)
    if op == "fp8_gemm":
        status = lib.fp8_gemm(*a, n, d_in, *w, 0, d_out, experts, at, y, dtype, *none)
    elif op == "fp8_gemm_dx":
        status = lib.fp8_gemm_dx(*a, n, d_out, *w, 0, d_in, experts, at, y, dtype, *none)
    elif op == "fp8_ffn_gate":
        status = lib.fp8_ffn_gate(*a, n, d_in, *w, *u, 0, d_out, 0, experts, at, y, dtype, *none)
    elif op == "fp8_ffn_gate_packed":
        status = lib.fp8_ffn_gate_packed(*a, n, d_in, *w, *u, 0, d_out, 0, experts, at, y, _far(7), *none)
    elif op == "ffn_gate":
        status = lib.ffn_gate(a[0], n, d_in, w[0], u[0], d_out, 0, experts, at, y, dtype, None, None, *none)
    elif op == "ffn_gate_dx":
        status = lib.ffn_gate_dx(*a, n, d_out, w[0], u[0], d_in, experts, at, y, dtype, *none)
    else:
        status = lib.ffn_gate_dw(*a, n, d_out, w[0], d_in, experts, at, y, _far(8), dtype, *none)
    return status, lib.gq_last_error().decode()


def _taken(op, n, d_in, d_out, experts, dtype):
    plan = gq.product_plan(op, n, d_in, d_out, experts, dtype=dtype)
    status, message = _call(op, n, d_in, d_out, experts, dtype)
    assert status == B.GQ_EINVAL and "overlap" in message, message
    return plan


def _refused(op, n, d_in, d_out, experts, dtype):
    with pytest.raises(gq.GQError) as e:
        gq.product_plan(op, n, d_in, d_out, experts, dtype=dtype)
    assert e.value.status == B.GQ_ENOTIMPL and "tiles" in e.value.message
    status, message = _call(op, n, d_in, d_out, experts, dtype)
    assert status == B.GQ_ENOTIMPL and "tiles" in message, message


@pytest.mark.parametrize("op,d_in,d_out,experts,f32,most", LIMITS)
def test_the_most_tiles_of_a_launch(op, d_in, d_out, experts, f32, most):
    """The largest number of rows has a plan and passes the checks of the call; one more is refused by both."""
    dtype = gq.GQ_F32 if f32 else gq.GQ_BF16
    assert 0 < most < 1 << 31
    _taken(op, most, d_in, d_out, experts, dtype)
    _refused(op, most + 1, d_in, d_out, experts, dtype)


def test_the_most_tiles_of_weights_gradients():
    """2^21 tiles of 256 x 256 each, of both weights: one expert's fit a launch, two experts' do not."""
    for n in (1, 4096):
        assert _taken("ffn_gate_dw", n, 1 << 18, 1 << 19, 1, gq.GQ_BF16)["rows"] == 256
        _refused("ffn_gate_dw", n, 1 << 18, 1 << 19, 2, gq.GQ_BF16)


@pytest.mark.parametrize("op", ["fp8_gemm", "fp8_gemm_dx", "fp8_ffn_gate", "fp8_ffn_gate_packed", "ffn_gate", "ffn_gate_dx"])
def test_rows_of_a_narrow_layer(op):
    """Near 2^31 where tiles have 256 rows, near 2^30 where float32 sums of 8-bit codes take 128."""
    for dtype in (gq.GQ_F32, gq.GQ_BF16):
        wide = op.startswith("fp8") and (dtype == gq.GQ_F32 or op.endswith("packed"))
        _taken(op, (1 << (30 if wide else 31)) - (1 << 21) - 1, 8, 8, 1, dtype)
