"""MXFP4 products of few rows an expert, as the library plans them by their mean, under routings
that are far from it."""
import pytest
import torch

import post_weight_quantization_gq_amd as gq

from test_gpu_mxfp4_kernels import BF, F32, _Call, _ids, _selecting_weight

# op, activations, rows, d_in, d_out, experts: streamed, their contraction whole and split
STREAMED = [("gemm", "bf16", 1024, 1100, 130, 64), ("gemm", "bf16", 64, 8192, 48, 4),
            ("gemm", "bf16", 2000, 520, 120, 130), ("gemm", "f32", 500, 520, 250, 64),
            ("gemm", "f32", 60, 4096, 130, 5), ("gemm_mx", "mx", 1024, 2100, 130, 64),
            ("gemm_mx", "mx", 64, 8200, 48, 4), ("gemm_mx", "mx", 2000, 520, 120, 130)]


def _routings(n, E):
    """Rows of each expert: all to one (the first, the last), two halves, one row more than a group
    of 16 or two, and a ramp."""
    one = [0] * E
    yield [n] + one[1:]
    yield one[1:] + [n]
    yield [0, n // 2 - 1] + one[3:] + [n // 2 - 1]
    yield [33, n - 33 - 17] + one[3:] + [17]
    yield [n * 2 * e // (E * (E + 1)) for e in range(E)]


def test_the_cases_are_streamed():
    plans = [gq.mxfp4_plan(op, n, d_in, d_out, E, gq.GQ_F32 if dtype == "f32" else gq.GQ_BF16)
             for op, dtype, n, d_in, d_out, E in STREAMED]
    assert all(p["streamed"] for p in plans)
    split = {(c[0], c[1]) for c, p in zip(STREAMED, plans) if p["split"] > 1}
    whole = {(c[0], c[1]) for c, p in zip(STREAMED, plans) if p["split"] == 1}
    assert split == whole == {("gemm", "bf16"), ("gemm", "f32"), ("gemm_mx", "mx")}
    for c in STREAMED:
        for counts in _routings(c[2], c[5]):
            assert len(counts) == c[5] and sum(counts) <= c[2] and min(counts) >= 0


@pytest.mark.gpu
@pytest.mark.parametrize("case", STREAMED, ids=_ids)
def test_exact_however_the_rows_are_spread(device, case):
    """One nonzero weight an output: equal bits for every routing, rows of no expert left alone."""
    n, E = case[2], case[5]
    c = _Call(case, device, exact=True)
    Q, S, index, value = _selecting_weight(c.gen, c.op, c.E, c.d_out, c.d_in, device)
    for counts in _routings(n, E):
        first = (n - sum(counts)) // 2
        c.at = [first + sum(counts[:e]) for e in range(E + 1)]
        c.off = torch.tensor(c.at, device=device)
        for out in (F32, BF):
            y = c.run(Q, S, out)
            for e, r in c.parts():
                want = c.a[r][:, index[e]] * value[e]
                assert torch.equal(y[r], want.to(F32).to(out)), (counts[:3], e)


@pytest.mark.gpu
@pytest.mark.parametrize("op", ["gemm", "gemm_mx"])
def test_one_expert_with_all_rows_takes_no_multiple(device, op):
    """3040 rows over 190 experts: all of them one expert's takes about as long as 16 each (measured:
    63 us against 52), where rows taken in turn by one block a weight took 37 times as long."""
    E, n, d_in, d_out = 190, 3040, 8192, 128
    Q, S = gq.mxfp4_quantize(torch.randn(E, d_out, d_in, device=device))
    x = torch.randn(n, d_in, device=device, dtype=BF)
    y = torch.zeros(n, d_out, device=device, dtype=BF)
    XQ, XS = gq.mxfp4_quantize(x)

    def us(off):
        best = float("inf")
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(10):
                if op == "gemm":
                    gq.mxfp4_gemm(x, Q, S, offsets=off, y=y)
                else:
                    gq.mxfp4_gemm_mx(XQ, XS, Q, S, d_in, offsets=off, y=y)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b) * 100)
        return best

    even = us(torch.arange(0, n + 1, 16, device=device))
    one = us(torch.tensor([0] * (E // 2) + [n] * (E - E // 2 + 1), device=device))
    print("evenly", even, "us, all to one expert", one, "us")
    assert one <= 4 * even
