"""GPU tests of every kernel, tile and split of the 8-bit products and the gated feed-forward block (the
sizes of _product_kernels).

The operands are small integers under scales of few bits, so that every product and every partial sum,
in whatever order and however split, is a multiple of one power of two and below 2^24 of it: exact in
float32.  The sums of a contraction have to be equal to float64's, and a bfloat16 output to their nearest: a
stage, a scale, a part or a block lost, stale or in the wrong place shows as such, which a bound over thousands of
rounded terms would not see.  (Matrix cores that add eight products by 14 bits of the largest, 16 here,
cut at 2^-9: below the unit.)  |x w| <= 4 and scales of at most 1.5 by 1.5 in units of 1/16: a sum
of K terms is below 144 K units, for K <= 100000 below 2^24.

Workspaces hold NaN beforehand, and what lies around them and the outputs stays as it was.
"""
import pytest
import torch

import post_weight_quantization_gq_amd as gq
from _product_cases import BF, EPS, F32, FP8, U8, act64, check, counts, generator, of, spans
from _product_kernels import CASES, types

pytestmark = pytest.mark.gpu


def integers(device, *shape, seed):
    return torch.randint(-2, 3, shape, generator=generator(device, seed), device=device)


def some_scales(device, shape, used, scales, down, seed):
    """Scales of few bits, 2^-down of them, and their values; 1 behind the `used` of a row."""
    i = torch.randint(0, 3 if scales == U8 else 4, shape, generator=generator(device, seed), device=device)
    if scales == U8:
        S = (126 - down + i).to(U8)
        S[..., used:] = 127
        return S, torch.exp2(S.double() - 127)
    S = torch.tensor([0.5, 0.75, 1.0, 1.5], device=device)[i] * 2.0 ** -down
    S[..., used:] = 1.0
    return S, S.double()


def packed_rows(device, n, d, scales, seed):
    blocks = -(-d // 128)
    codes = integers(device, n, 128 * blocks, seed=seed)
    codes[:, d:] = 0
    S, s = some_scales(device, (n, -(-blocks // 4) * 4), blocks, scales, 0, seed + 100)
    return codes.float().to(FP8), S, codes.double()[:, :d] * s.repeat_interleave(128, 1)[:, :d]


def packed_weight(device, E, d_out, d_in, scales, down, seed):
    blocks = -(-d_in // 128)
    codes = integers(device, *E, d_out, 128 * blocks, seed=seed)
    codes[..., d_in:] = 0
    S, s = some_scales(device, (*E, -(-d_out // 128), blocks), blocks, scales, down, seed + 100)
    s = s.repeat_interleave(128, -2)[..., :d_out, :].repeat_interleave(128, -1)[..., :d_in]
    return codes.float().to(FP8), S, codes.double()[..., :d_in] * s


class Guarded:
    """A buffer with values around it that have to stay."""

    def __init__(self, device, shape, dtype, fill):
        self.count = 1
        for s in shape:
            self.count *= s
        self.all = torch.full((self.count + 512,), 77, device=device, dtype=torch.float32).to(dtype)
        self.t = self.all[256:256 + self.count].view(shape)
        self.t.copy_(torch.full(shape, fill, device=device, dtype=torch.float32).to(dtype))

    def intact(self):
        around = torch.cat([self.all[:256], self.all[256 + self.count:]]).float()
        return bool((around == torch.tensor(77.0).to(self.all.dtype).float().item()).all())


def scratch(device, size):
    ws = Guarded(device, (size,), U8, 255)
    assert ws.t.data_ptr() % 256 == 0
    return ws


def equal(y, ref, at, out, what):
    """The rows of experts are their sums, rounded once; the others as they were."""
    want = ref.to(F32).to(out)
    live = slice(0, len(ref)) if at is None else slice(at[0], at[-1])
    assert torch.equal(ref.to(F32).double(), ref), "the oracle's sums are float32 numbers"
    assert torch.equal(y[live], want[live]), what
    assert bool((y[:live.start] == 7).all()) and bool((y[live.stop:] == 7).all())


def sums(x, W, at):
    z = torch.zeros(x.shape[0], W.shape[-2], dtype=torch.float64, device=x.device)
    for e, r in spans(x.shape[0], at):
        z[r] = x[r] @ of(W, e).T
    return z


def ids(c):
    return "-".join(str(v) for v in c)


def cases(*ops):
    return [pytest.param(op, *c, s, o, id=f"{op}-{ids(c)}-{'' if s is None else str(s)[6:]}-{str(o)[6:]}")
            for op in ops for c in CASES[op] for s, o in types(op)]


def down_by(k):
    """2^-down of weights whose products with rows of k are about 1."""
    return max(0, round(0.5 * torch.tensor(4.0 * k).log2().item()))


def routing(device, n, experts):
    at = counts(n, experts, seed=n) if experts else None
    return at, torch.tensor(at, device=device) if experts else None, (experts,) if experts else ()


@pytest.mark.parametrize("op,n,d_in,d_out,experts,scales,out", cases("fp8_gemm", "fp8_gemm_dx"))
def test_fp8_sums(device, op, n, d_in, d_out, experts, scales, out):
    at, offsets, E = routing(device, n, experts)
    back = op == "fp8_gemm_dx"
    k, m = (d_out, d_in) if back else (d_in, d_out)
    XQ, XS, x = packed_rows(device, n, k, scales, seed=1)
    Q, S, w = packed_weight(device, E, d_out, d_in, scales, down_by(k), seed=2)
    y = Guarded(device, (n, m), out, 7)
    size = gq.fp8_gemm_dx_workspace_size if back else gq.fp8_gemm_workspace_size
    ws = scratch(device, size(n, d_in, d_out, experts or 1, scales, gq.GQ_F32 if out == F32 else gq.GQ_BF16))
    (gq.fp8_gemm_dx if back else gq.fp8_gemm)(XQ, XS, Q, S, d_in, offsets=offsets, y=y.t, ws=ws.t)
    equal(y.t, sums(x, w.transpose(-1, -2) if back else w, at), at, out, op)
    assert y.intact() and ws.intact()


def check_h(h, zg, zu, act, at, out, what):
    """h of exact products: act rounds (_product_cases), and one product."""
    v = act64(zg, act)[0]
    live = slice(0, len(zg)) if at is None else slice(at[0], at[-1])
    ref, limit = v * zu, 33 * EPS * (1 + zg * zg) * (v * zu).abs() + (zg * zu).abs() * 2.0 ** -126 + 2.0 ** -140
    check(h[live], ref[live], limit[live], out, what)
    return ref, limit


@pytest.mark.parametrize("op,n,d_in,d_ff,experts,scales,out", cases("fp8_ffn_gate", "ffn_gate"))
def test_gate(device, op, n, d_in, d_ff, experts, scales, out):
    at, offsets, E = routing(device, n, experts)
    h = Guarded(device, (n, d_ff), out, 7)
    dt = gq.GQ_F32 if out == F32 else gq.GQ_BF16
    act = ("silu", "gelu", "gelu_tanh")[(n + d_in) % 3]
    if op == "ffn_gate":
        x = integers(device, n, d_in, seed=1).to(BF)
        g, u = (integers(device, *E, d_ff, d_in, seed=s).to(BF) * 2.0 ** -down_by(d_in) for s in (2, 3))
        ws = scratch(device, gq.ffn_gate_workspace_size(n, d_in, d_ff, experts or 1))
        got, zg, zu = gq.ffn_gate(x, g, u, act=act, offsets=offsets, y=h.t, save=True, ws=ws.t)
        x, g, u = x.double(), g.double(), u.double()
        want = sums(x, g, at), sums(x, u, at)
        live = slice(0, n) if at is None else slice(at[0], at[-1])
        assert torch.equal(zg[live].double(), want[0][live]) and torch.equal(zu[live].double(), want[1][live])
        saved = got.clone()
        assert torch.equal(gq.ffn_gate(x.to(BF), g.to(BF), u.to(BF), act=act, offsets=offsets, y=h.t, ws=ws.t), saved)
    else:
        XQ, XS, x = packed_rows(device, n, d_in, scales, seed=1)
        (G, GS, g), (U, US, u) = (packed_weight(device, E, d_ff, d_in, scales, down_by(d_in), seed=s) for s in (2, 3))
        ws = scratch(device, gq.fp8_ffn_gate_workspace_size(n, d_in, d_ff, experts or 1, scales, dt))
        gq.fp8_ffn_gate(XQ, XS, G, GS, U, US, d_in, act=act, offsets=offsets, y=h.t, ws=ws.t)
        want = sums(x, g, at), sums(x, u, at)
    check_h(h.t, *want, act, at, out, op)
    if at:
        assert bool((h.t[:at[0]] == 7).all()) and bool((h.t[at[-1]:] == 7).all())
    assert h.intact() and ws.intact()


@pytest.mark.parametrize("op,n,d_in,d_ff,experts,scales,out", cases("fp8_ffn_gate_packed"))
def test_packed_gate(device, op, n, d_in, d_ff, experts, scales, out):
    """Codes within half a step of h, scales the smallest powers of two that hold their block."""
    at, offsets, E = routing(device, n, experts)
    XQ, XS, x = packed_rows(device, n, d_in, scales, seed=1)
    (G, GS, g), (U, US, u) = (packed_weight(device, E, d_ff, d_in, scales, down_by(d_in), seed=s) for s in (2, 3))
    HQ = Guarded(device, (n, gq.fp8_row_bytes(d_ff)), U8, 7)
    HS = Guarded(device, (n, gq.fp8_row_scales(d_ff)), scales, 7)
    ws = scratch(device, gq.fp8_ffn_gate_packed_workspace_size(n, d_in, d_ff, experts or 1, scales))
    gq.fp8_ffn_gate(XQ, XS, G, GS, U, US, d_in, offsets=offsets, packed=True, HQ=HQ.t.view(FP8), HS=HS.t, ws=ws.t)
    zg, zu = sums(x, g, at), sums(x, u, at)
    live = slice(0, n) if at is None else slice(at[0], at[-1])
    ref = (act64(zg, "silu")[0] * zu)[live]
    off = (33 * EPS * (1 + zg[live] ** 2) * ref.abs()) + 2.0 ** -140
    q, s = HQ.t[live], HS.t[live]
    blocks = -(-d_ff // 128)
    unit = torch.exp2(s.double() - 127) if scales == U8 else s.double()
    got = q.view(FP8).double()[:, :d_ff] * unit.repeat_interleave(128, 1)[:, :d_ff]
    step = torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * unit.repeat_interleave(128, 1)[:, :d_ff])
    assert bool(((got - ref).abs() <= step + 2 * off).all())
    pad = (0, 128 * blocks - d_ff)
    top = torch.nn.functional.pad(ref.abs(), pad).view(len(ref), blocks, 128).amax(2)
    most = torch.nn.functional.pad(off, pad).view(len(ref), blocks, 128).amax(2)
    unit = unit[:, :blocks]
    assert bool((top <= 448 * unit + most).all()) and bool(((top > 224 * unit - most) | (top == 0)).all())
    assert not q[:, d_ff:].any() and bool((s[:, blocks:] == (127 if scales == U8 else 1)).all())
    for b in (HQ, HS):
        assert bool((b.t[:live.start] == 7).all()) and bool((b.t[live.stop:] == 7).all()) and b.intact()
    assert ws.intact()


@pytest.mark.parametrize("op,n,d_in,d_ff,experts,scales,out", cases("ffn_gate_dx"))
def test_dx(device, op, n, d_in, d_ff, experts, scales, out):
    at, offsets, E = routing(device, n, experts)
    a, b = (integers(device, n, d_ff, seed=s).to(BF) for s in (1, 2))
    g, u = (integers(device, *E, d_ff, d_in, seed=s).to(BF) for s in (3, 4))
    y = Guarded(device, (n, d_in), out, 7)
    ws = scratch(device, gq.ffn_gate_dx_workspace_size(n, d_in, d_ff, experts or 1))
    gq.ffn_gate_dx(a, b, g, u, offsets=offsets, y=y.t, ws=ws.t)
    ref = sums(a.double(), g.double().transpose(-1, -2), at) + sums(b.double(), u.double().transpose(-1, -2), at)
    equal(y.t, ref, at, out, op)
    assert y.intact() and ws.intact()


@pytest.mark.parametrize("op,n,d_in,d_ff,experts,scales,out", cases("ffn_gate_dw"))
def test_dw(device, op, n, d_in, d_ff, experts, scales, out):
    at, offsets, E = routing(device, n, experts)
    x = integers(device, n, d_in, seed=1).to(BF)
    a, b = (integers(device, n, d_ff, seed=s).to(BF) for s in (2, 3))
    got = [Guarded(device, (*E, d_ff, d_in), out, 7) for _ in range(2)]
    ws = scratch(device, gq.ffn_gate_dw_workspace_size(n, d_in, d_ff, experts or 1))
    gq.ffn_gate_dw(a, b, x, experts=experts, offsets=offsets, dG=got[0].t, dU=got[1].t, ws=ws.t)
    for d, z in zip(got, (a, b)):
        for e, r in spans(n, at):
            want = z[r].double().T @ x[r].double()
            assert torch.equal(of(d.t, e), want.to(F32).to(out)), e
        assert d.intact()
    assert ws.intact()


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("n,d_in,d_ff,experts", sorted(set(CASES["ffn_gate_dx"] + CASES["ffn_gate_dw"]), key=str))
def test_backward_is_its_parts(device, n, d_in, d_ff, experts, out):
    """One call for the whole pass: dz rounded to bfloat16, then both products, with odd d_ff too."""
    at, offsets, E = routing(device, n, experts)
    x = integers(device, n, d_in, seed=1).to(BF)
    g, u = (integers(device, *E, d_ff, d_in, seed=s).to(BF) * 2.0 ** -down_by(d_in) for s in (2, 3))
    dh = torch.randn(n, d_ff, generator=generator(device, 4), device=device).to(out)
    _, zg, zu = gq.ffn_gate(x, g, u, act="gelu", offsets=offsets, save=True)
    dzg, dzu = gq.ffn_gate_dz(dh, zg, zu, act="gelu")
    want = [gq.ffn_gate_dx(dzg, dzu, g, u, offsets=offsets, out_dtype=out),
            *gq.ffn_gate_dw(dzg, dzu, x, experts=experts, offsets=offsets, out_dtype=out)]
    ws = scratch(device, gq.ffn_gate_backward_workspace_size(n, d_in, d_ff, experts or 1))
    for which in ((True, True, True), (True, False, False), (False, True, False), (False, False, True)):
        given = [torch.zeros_like(w) if on else None for w, on in zip(want, which)]
        got = gq.ffn_gate_backward(dh, x, g, u, zg, zu, act="gelu", offsets=offsets, which=which, dx=given[0], dG=given[1],
                                   dU=given[2], ws=ws.t)
        for have, w, on in zip(got, want, which):
            assert (have is None) if not on else torch.equal(have, w)
    assert ws.intact()
