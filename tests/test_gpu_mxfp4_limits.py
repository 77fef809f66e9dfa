"""GPU tests of the MXFP4 rows and products at sizes that one launch's limits do not hold."""
import numpy as np
import pytest
import torch

import oracle as O
import post_weight_quantization_gq_amd as gq

from test_gpu_mxfp4 import BF, F32, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
def test_more_rows_than_a_launch_has_lanes(device, dtype):
    """Rows of one value, each padded to 16 pieces of 8: 2^28 of them are 2^32 pieces, more than a
    launch can have lanes.  Packed and read back, every part of them equals a call on that part
    alone, and the last rows are the oracle's."""
    rows, part = (1 << 28) + 37, 1 << 25
    gen = torch.Generator(device=device)
    gen.manual_seed(5)
    x = torch.randn((rows, 1), generator=gen, device=device, dtype=dtype)
    Q = torch.full((rows, 64), 0xEE, dtype=torch.uint8, device=device)
    S = torch.full((rows, 4), 0xEE, dtype=torch.uint8, device=device)
    gq.mxfp4_quantize(x, Q=Q, S=S)
    y = gq.mxfp4_dequantize(Q, S, 1, dtype=dtype, y=torch.full_like(x, 99.0))
    for r in range(0, rows, part):
        q, s = gq.mxfp4_quantize(x[r:r + part])
        assert torch.equal(q, Q[r:r + part]) and torch.equal(s, S[r:r + part]), r
        assert torch.equal(gq.mxfp4_dequantize(q, s, 1, dtype=dtype), y[r:r + part]), r
    Qr, Sr = O.mx_quantize(f64(x[-100:]))
    np.testing.assert_array_equal(Q[-100:].cpu().numpy(), Qr)
    np.testing.assert_array_equal(S[-100:].cpu().numpy(), Sr)
    np.testing.assert_array_equal(f64(y[-100:]), O.mx_values(Qr, Sr, 1))
