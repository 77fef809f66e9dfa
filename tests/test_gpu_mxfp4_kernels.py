"""GPU tests of every kernel, tile and split of the MXFP4 products (the sizes of _mx_cases).

Selection.  Each output has one nonzero weight, a power of two, so it is one activation times it:
exact in float32, however the terms are ordered or split (float32 activations are the sum of three
bfloat16 planes of 8 bits each, and so is every partial sum), and rounded once to bfloat16.  The
outputs have to be equal: a plane, a stage, a scale or a block lost, stale or in the wrong place
shows as such, which a bound over sums of thousands of terms would not see.

Dense.  Random codes under random scales against float64, by the bound of the other MXFP4 tests:
T terms, products exact, every float32 addition off by at most 2^-23 of a partial sum that is at
most A = sum |a w|: |y - y64| <= (T + 8) 2^-23 A, T = K, or 3 K for three planes (whose sizes sum
to at most (1 + 2^-7) |a|, within the slack of truncation), and half a step of a bfloat16 output.
"""
import numpy as np
import pytest
import torch

import post_weight_quantization_gq_amd as gq

from _mx_cases import CASES

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
VALUES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def _ids(c):
    return "-".join(str(v) for v in c)


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _power(e):
    """2^e in float64, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _decode(Q, S, d):
    """float64 values [..][d]."""
    codes = torch.stack((Q & 15, Q >> 4), dim=-1).flatten(-2).long()
    v = VALUES.to(Q.device)[codes & 7] * (1 - 2 * (codes >> 3))
    return (v.unflatten(-1, (S.shape[-1], 32)) * _power(S.long() - 127).unsqueeze(-1)).flatten(-2)[..., :d]


def _scales(gen, shape, d, device, low=-8, high=9):
    """Scale bytes of rows of d values, 127 past their last block."""
    groups = -(-d // 128)
    S = torch.randint(127 + low, 127 + high, (*shape, 4 * groups), generator=gen, device=device).to(torch.uint8)
    S[..., -(-d // 32):] = 127
    return S


def _codes(gen, shape, d, device):
    """Random codes of rows of d values, 0 past their end."""
    codes = torch.randint(0, 16, (*shape, 128 * -(-d // 128)), generator=gen, device=device).to(torch.uint8)
    codes[..., d:] = 0
    return codes


def _selecting_weight(gen, op, E, d_out, d_in, device):
    """Packed weights in which each output (a row, for the gradient a column) has one nonzero, a
    power of two: (Q, S, index [E][outputs] of the contraction, value [E][outputs] float64)."""
    codes = torch.zeros((E, d_out, 128 * -(-d_in // 128)), dtype=torch.uint8, device=device)
    S = _scales(gen, (E, d_out), d_in, device)
    K, m = (d_out, d_in) if op == "gemm_dx" else (d_in, d_out)
    # spread evenly over the contraction, from a random start, in a random order
    at = (torch.arange(m, device=device) * K // m + torch.randint(0, K, (E, 1), generator=gen, device=device)) % K
    at = at[:, torch.randperm(m, generator=gen, device=device)]
    pick = torch.tensor([1, 2, 4, 6], dtype=torch.uint8, device=device)        # 0.5, 1, 2, 4
    code = pick[torch.randint(0, 4, (E, m), generator=gen, device=device)]
    code += 8 * torch.randint(0, 2, (E, m), generator=gen, device=device).to(torch.uint8)
    e, o = torch.arange(E, device=device)[:, None], torch.arange(m, device=device)[None]
    row, col = (at, o.expand(E, m)) if op == "gemm_dx" else (o.expand(E, m), at)
    codes[e, row, col] = code
    value = VALUES.to(device)[(code & 7).long()] * (1 - 2 * (code >> 3).long())
    return _pack(codes), S, at, value * _power(S[e, row, col // 32].long() - 127)


def _offsets(gen_np, n, E):
    """Rows before the first expert, empty experts, one with many, rows behind the last."""
    lo, hi = min(2, n // 4), n - min(3, n // 4)
    p = np.exp(0.7 * gen_np.standard_normal(E))
    p[gen_np.random(E) < 0.2] = 0.0
    p[E // 2] += 1e-3
    return np.concatenate([[lo], lo + np.cumsum(gen_np.multinomial(hi - lo, p / p.sum()))])


class _Call:
    """Activations, offsets and the call of a case for given weights."""

    def __init__(self, case, device, exact):
        self.op, self.dtype, self.n, self.d_in, self.d_out, self.experts = case
        self.E = self.experts or 1
        seed = sum((i + 1) * v for i, v in enumerate((self.n, self.d_in, self.d_out, self.E))) + exact
        self.gen = torch.Generator(device=device)
        self.gen.manual_seed(seed)
        gen, n = self.gen, self.n
        self.K, self.m = (self.d_out, self.d_in) if self.op == "gemm_dx" else (self.d_in, self.d_out)
        self.at = [0, n]
        if self.experts:
            self.at = _offsets(np.random.default_rng(seed), n, self.E).tolist()
        self.off = torch.tensor(self.at, device=device) if self.experts else None
        if self.dtype == "mx":
            codes = _codes(gen, (n,), self.K, device)
            if exact:
                codes[..., :self.K] |= 1                                   # no zeros
            self.x = _pack(codes), _scales(gen, (n,), self.K, device)
            self.a = _decode(*self.x, self.K)
            return
        if exact:        # every bit of the mantissa in use
            bits = 24 if self.dtype == "f32" else 8
            x = torch.randint(1 << (bits - 1), 1 << bits, (n, self.K), generator=gen, device=device).double()
            x *= 1 - 2 * torch.randint(0, 2, (n, self.K), generator=gen, device=device)
            x *= _power(torch.randint(-40, 20, (n, self.K), generator=gen, device=device))
        else:
            x = torch.randn((n, self.K), generator=gen, device=device)
        self.x = x.to(F32 if self.dtype == "f32" else BF)
        self.a = self.x.double()

    def run(self, Q, S, out):
        y = torch.full((self.n, self.m), -77.0, dtype=out, device=Q.device)
        Q, S = (Q, S) if self.experts else (Q[0], S[0])
        if self.op == "gemm_mx":
            gq.mxfp4_gemm_mx(*self.x, Q, S, self.d_in, offsets=self.off, y=y)
        elif self.op == "gemm":
            gq.mxfp4_gemm(self.x, Q, S, offsets=self.off, y=y)
        else:
            gq.mxfp4_gemm_dx(self.x, Q, S, self.d_in, offsets=self.off, y=y)
        assert (y[:self.at[0]] == -77.0).all() and (y[self.at[-1]:] == -77.0).all()
        return y

    def parts(self):
        return [(e, slice(self.at[e], self.at[e + 1])) for e in range(self.E) if self.at[e + 1] > self.at[e]]


@pytest.mark.parametrize("case", CASES, ids=_ids)
def test_one_term_a_product_is_exact(device, case):
    c = _Call(case, device, exact=True)
    Q, S, index, value = _selecting_weight(c.gen, c.op, c.E, c.d_out, c.d_in, device)
    for out in (F32, BF):
        y = c.run(Q, S, out)
        for e, r in c.parts():
            want = c.a[r][:, index[e]] * value[e]
            assert torch.equal(want.to(F32).double(), want)              # one float32 value
            assert torch.equal(y[r], want.to(F32).to(out)), (out, e)


@pytest.mark.parametrize("case", CASES, ids=_ids)
def test_dense_against_float64(device, case):
    c = _Call(case, device, exact=False)
    codes = _codes(c.gen, (c.E, c.d_out), c.d_in, device)
    Q, S = _pack(codes), _scales(c.gen, (c.E, c.d_out), c.d_in, device, low=-4, high=5)
    del codes
    terms = c.K * (3 if c.dtype == "f32" else 1)
    for out in (F32, BF):
        y, worst = c.run(Q, S, out), 0.0
        for e, r in c.parts():
            W = _decode(Q[e], S[e], c.d_in)
            W = W if c.op == "gemm_dx" else W.T.contiguous()
            ref = c.a[r] @ W
            limit = (terms + 8) * 2.0 ** -23 * (c.a[r].abs() @ W.abs())
            if out == BF:
                limit += 2.0 ** -8 * ref.abs() + 2.0 ** -134
            err = (y[r].double() - ref).abs()
            worst = max(worst, float((err / limit.clamp_min(1e-300)).max()))
        print(out, "worst error / bound", worst)
        assert worst <= 1.0
