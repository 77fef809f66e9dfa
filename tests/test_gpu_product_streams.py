"""GPU tests of the 8-bit products and the gated feed-forward block as programs use them: captured and
replayed, on other streams, two at once, with skewed experts, the same tensor twice, past 32 bits."""
import pytest
import torch

import post_weight_quantization_gq_amd as gq
from _product_cases import BF, F32, FP8, U8, generator, normal
from test_gpu_product_kernels import integers, packed_rows, packed_weight, sums

pytestmark = pytest.mark.gpu

OPS = ["quantize", "gemm", "gemm32", "dx", "gate8", "packed", "gate", "backward"]


def program(device, op, n, d_in=1024, d_ff=640):
    """(a call of one operator from x into its outputs, the outputs, the shape of x, its workspace's size)."""
    w = [normal(device, d_ff, d_in, seed=s, dtype=BF, scale=d_in ** -0.5) for s in (1, 2)]
    q = [gq.fp8_quantize_weight(v) for v in w]
    out = F32 if op == "gemm32" else BF
    new = lambda *shape, dtype=BF: torch.zeros(shape, device=device, dtype=dtype)
    rows = lambda x, o, **k: gq.fp8_quantize(x, Q=o[0], S=o[1], **k)
    XQ = [new(n, gq.fp8_row_bytes(d_in), dtype=U8).view(FP8), new(n, gq.fp8_row_scales(d_in), dtype=U8)]
    if op == "quantize":
        return lambda x, ws=None, **k: rows(x, XQ, **k), XQ, (n, d_in), 0
    if op in ("gemm", "gemm32"):
        y = new(n, d_ff, dtype=out)
        return (lambda x, ws=None, **k: gq.fp8_gemm(*rows(x, XQ, **k), *q[0], d_in, y=y, ws=ws, **k), [y], (n, d_in),
                gq.fp8_gemm_workspace_size(n, d_in, d_ff, dtype=gq.GQ_F32 if out == F32 else gq.GQ_BF16))
    if op == "dx":
        GQ = [new(n, gq.fp8_row_bytes(d_ff), dtype=U8).view(FP8), new(n, gq.fp8_row_scales(d_ff), dtype=U8)]
        y = new(n, d_in)
        return (lambda x, ws=None, **k: gq.fp8_gemm_dx(*rows(x, GQ, **k), *q[0], d_in, y=y, ws=ws, **k), [y], (n, d_ff),
                gq.fp8_gemm_dx_workspace_size(n, d_in, d_ff))
    if op == "gate8":
        y = new(n, d_ff)
        return (lambda x, ws=None, **k: gq.fp8_ffn_gate(*rows(x, XQ, **k), *q[0], *q[1], d_in, y=y, ws=ws, **k), [y], (n, d_in),
                gq.fp8_ffn_gate_workspace_size(n, d_in, d_ff))
    if op == "packed":
        o = [new(n, gq.fp8_row_bytes(d_ff), dtype=U8).view(FP8), new(n, gq.fp8_row_scales(d_ff), dtype=U8)]
        return (lambda x, ws=None, **k: gq.fp8_ffn_gate(*rows(x, XQ, **k), *q[0], *q[1], d_in, packed=True, HQ=o[0], HS=o[1],
                                                        ws=ws, **k), o, (n, d_in),
                gq.fp8_ffn_gate_packed_workspace_size(n, d_in, d_ff))
    if op == "gate":
        y = new(n, d_ff)
        return (lambda x, ws=None, **k: gq.ffn_gate(x, *w, y=y, ws=ws, **k), [y], (n, d_in),
                gq.ffn_gate_workspace_size(n, d_in, d_ff))
    fixed = normal(device, n, d_in, seed=5, dtype=BF)
    _, zg, zu = gq.ffn_gate(fixed, *w, save=True)
    o = [new(n, d_in), new(d_ff, d_in), new(d_ff, d_in)]
    return (lambda x, ws=None, **k: gq.ffn_gate_backward(x, fixed, *w, zg, zu, dx=o[0], dG=o[1], dU=o[2], ws=ws, **k), o,
            (n, d_ff), gq.ffn_gate_backward_workspace_size(n, d_in, d_ff))


def bits(ts):
    return [t.view(U8).clone() if t.dtype == FP8 else t.clone() for t in ts]


def same(a, b):
    return all(torch.equal(x.view(U8) if x.dtype == FP8 else x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("n", [3, 40, 300])
@pytest.mark.parametrize("op", OPS)
def test_graph_replays_and_streams(device, op, n):
    """Two captured calls that share a workspace, replayed with new inputs in place between eager
    calls; a workspace from the library; a call on another stream; two streams at once."""
    (one, out1, shape, size), (two, out2, _, _) = program(device, op, n), program(device, op, n)
    xs = [normal(device, *shape, seed=10 + i, dtype=BF) for i in range(4)]
    want = []
    for x in xs:
        one(x)
        want.append(bits(out1))
    ws = torch.full((size + 256,), 255, dtype=U8, device=device)
    x1, x2 = xs[0].clone(), xs[1].clone()
    torch.cuda.synchronize()
    graphs = []
    for call, x in ((one, x1), (two, x2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(x, ws=ws)
        graphs.append(g)
    for turn in range(3):
        x1.copy_(xs[turn]), x2.copy_(xs[turn + 1])
        for t in out1 + out2:
            t.view(U8).fill_(3)
        graphs[0].replay(), graphs[1].replay()
        a, b = bits(out1), bits(out2)
        assert same(out1, want[turn]) and same(out2, want[turn + 1])
        one(xs[3])
        assert same(out1, want[3]) and same(a, want[turn]) and same(b, want[turn + 1])
    one(xs[2], ws=False if op != "quantize" else None)
    assert same(out1, want[2])
    # another stream, and both at once (each with scratch of its own)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    for turn in range(3):
        one(xs[turn], stream=sides[0])
        two(xs[turn + 1], stream=sides[1])
        for s in sides:
            s.synchronize()
        assert same(out1, want[turn]) and same(out2, want[turn + 1])


def test_training_step_on_another_stream_and_in_a_graph(device):
    n, d_in, d_ff = 200, 256, 384
    xs = [normal(device, n, d_in, seed=s, dtype=BF) for s in range(3)]
    W = [normal(device, d_ff, d_in, seed=9 + s, dtype=BF, scale=0.06) for s in range(2)]
    dh = normal(device, n, d_ff, seed=8, dtype=BF)

    def step(x, G, U):
        return torch.autograd.grad(gq.ffn_gate(x, G, U), (x, G, U), dh)

    leaves = lambda x: [t.clone().requires_grad_() for t in (x, *W)]
    want = [step(*leaves(x)) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(*leaves(xs[1]))
    side.synchronize()
    assert same(got, want[1])
    # captured, of leaves that no eager graph holds
    static = leaves(xs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*static)
    for turn in (0, 1, 2, 1):
        with torch.no_grad():
            static[0].copy_(xs[turn])
        for t in got:
            t.fill_(3)
        graph.replay()
        assert same(got, want[turn])
        assert same(step(*leaves(xs[2])), want[2])


def test_one_tensor_for_both_weights_and_an_expanded_gradient(device):
    """G is U: its gradient is the sum of both; the gradient of a sum has strides of zero."""
    n, d_in, d_ff = 33, 264, 130
    x = normal(device, n, d_in, seed=1, dtype=BF).requires_grad_()
    G = normal(device, d_ff, d_in, seed=2, dtype=BF, scale=0.06).requires_grad_()
    gq.ffn_gate(x, G, G).sum().backward()
    ones = torch.ones(n, d_ff, device=device, dtype=BF)
    with torch.no_grad():
        _, zg, zu = gq.ffn_gate(x, G, G, save=True)
        dx, dG, dU = gq.ffn_gate_backward(ones, x, G, G, zg, zu)
    assert torch.equal(zg, zu) and torch.equal(x.grad, dx) and torch.equal(G.grad, dG + dU)
    Q, S = gq.fp8_quantize_weight(G.detach())
    rows = gq.fp8_quantize(x.detach())
    a = gq.fp8_ffn_gate(*rows, Q, S, Q.clone(), S.clone(), d_in)
    assert torch.equal(gq.fp8_ffn_gate(*rows, Q, S, Q, S, d_in), a)


@pytest.mark.parametrize("n,experts,full", [(1600, 200, 7), (1600, 200, 199), (280, 40, 0), (2000, 40, 39)])
@pytest.mark.parametrize("op", ["gemm", "gate8", "gate", "packed"])
def test_one_expert_has_nearly_all_rows(device, op, n, experts, full):
    """Eight rows an expert or fewer on average, so that weights are streamed, and one expert has them all but
    a few; and more rows, by tiles."""
    d_in, d_out = 264, 130
    some = [0 if e % 3 else 1 for e in range(experts)]
    some[full] = n - 5 - (sum(some) - some[full])
    at = [2]
    for c in some:
        at.append(at[-1] + c)
    assert at[-1] == n - 3
    offsets = torch.tensor(at, device=device)
    if op == "gate":
        x = integers(device, n, d_in, seed=1).to(BF)
        g, u = (integers(device, experts, d_out, d_in, seed=s).to(BF) * 2.0 ** -5 for s in (2, 3))
        h, zg, zu = gq.ffn_gate(x, g, u, offsets=offsets, save=True)
        live = slice(at[0], at[-1])
        assert torch.equal(zg[live].double(), sums(x.double(), g.double(), at)[live])
        assert torch.equal(zu[live].double(), sums(x.double(), u.double(), at)[live])
        assert not h[:2].any() and not h[-3:].any()
        return
    XQ, XS, x = packed_rows(device, n, d_in, U8, seed=1)
    Q, S, w = packed_weight(device, (experts,), d_out, d_in, U8, 5, seed=2)
    if op == "gemm":
        y = gq.fp8_gemm(XQ, XS, Q, S, d_in, offsets=offsets, out_dtype=F32)
        assert torch.equal(y.double(), sums(x, w, at))
        return
    # the expert alone, by tiles, has the same sums (exact ones), and the same h and codes from them
    one = slice(at[full], at[full + 1])
    kw = dict(packed=True) if op == "packed" else dict(out_dtype=F32)
    got = gq.fp8_ffn_gate(XQ, XS, Q, S, Q, S, d_in, offsets=offsets, **kw)
    alone = gq.fp8_ffn_gate(XQ[one], XS[one], Q[full], S[full], Q[full], S[full], d_in, **kw)
    got, alone = (t if op == "packed" else (t,) for t in (got, alone))
    for a, b in zip(got, alone):
        assert torch.equal(a.view(U8)[one] if a.dtype == FP8 else a[one], b.view(U8) if b.dtype == FP8 else b)


def test_views_at_odd_places(device):
    """Outputs and gradients that start anywhere an element can, operands of odd rows too."""
    n, d_in, d_ff = 37, 131, 77
    place = lambda t: torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)
    x, dh = normal(device, n, d_in, seed=1, dtype=BF), normal(device, n, d_ff, seed=2, dtype=BF)
    G, U = (normal(device, d_ff, d_in, seed=s, dtype=BF, scale=0.1) for s in (3, 4))
    h, zg, zu = gq.ffn_gate(x, G, U, save=True)
    want = gq.ffn_gate_backward(dh, x, G, U, zg, zu)
    assert place(x).data_ptr() % 4 == 2
    got = gq.ffn_gate(place(x), place(G), place(U), y=place(torch.zeros_like(h)), save=True)
    assert same(got, (h, zg, zu))
    got = gq.ffn_gate_backward(place(dh), place(x), place(G), place(U), place(zg), place(zu),
                               dx=place(torch.zeros_like(x)), dG=place(torch.zeros_like(G)), dU=place(torch.zeros_like(U)))
    assert same(got, want)
    Q, S = gq.fp8_quantize_weight(place(G))
    rows = gq.fp8_quantize(place(x))
    assert torch.equal(gq.fp8_gemm(*rows, Q, S, d_in), gq.fp8_gemm(*rows, Q, S, d_in, y=place(torch.zeros_like(h))))


def test_stages_are_timed(device):
    gq.gq_timing_read()
    gq.gq_timing_enable(True)
    try:
        Q, S = gq.fp8_quantize_weight(normal(device, 64, 256, seed=1))
        rows = gq.fp8_quantize(normal(device, 8, 256, seed=2))
        gq.fp8_dequantize(*rows, 256)
        gq.fp8_dequantize_weight(Q, S, 256)
        gq.fp8_gemm(*rows, Q, S, 256)
        gq.fp8_ffn_gate(*rows, Q, S, Q, S, 256)
        x, G = normal(device, 8, 256, seed=3, dtype=BF), normal(device, 64, 256, seed=4, dtype=BF)
        _, zg, zu = gq.ffn_gate(x, G, G, save=True)
        gq.ffn_gate_dz(normal(device, 8, 64, seed=5), zg, zu)
        gq.ffn_gate_dx(*gq.ffn_gate_dz(normal(device, 8, 64, seed=5), zg, zu), G, G)
    finally:
        gq.gq_timing_enable(False)
    t = gq.gq_timing_read()
    assert {k: t[k][1] for k in ("fp8_pack", "fp8_gemm", "ffn_gate", "ffn_back")} == {
        "fp8_pack": 4, "fp8_gemm": 1, "ffn_gate": 2, "ffn_back": 3}
    assert t["lut_gemv"][1] == 0 and "mxfp4_gemm" not in t and all(t[k][0] > 0 for k in ("fp8_pack", "ffn_gate"))


# ---- past 32 bits -----------------------------------------------------------------------

def test_rows_past_32_bits(device):
    """Codes of more than 4 GiB, outputs of more than 2^31 elements: the last rows are those of a call on
    them alone, of which the sums are exact."""
    n, k, m, t = 1100000, 4096, 2048, 40
    XQ = torch.zeros(n, k, dtype=U8, device=device).view(FP8)
    XS = torch.full((n, 32), 127, dtype=U8, device=device)
    tq, ts, x = packed_rows(device, t, k, U8, seed=1)
    Q, S, w = packed_weight(device, (), m, k, U8, 6, seed=2)
    for at in (n - t, n // 2):
        XQ.view(U8)[at:at + t], XS[at:at + t] = tq.view(U8), ts
    y = gq.fp8_gemm(XQ, XS, Q, S, k)
    want = (x @ w.T).to(F32).to(BF)
    for at in (n - t, n // 2):
        assert torch.equal(y[at:at + t], want)
    assert not y[:1000].any() and not y[n - t - 1000:n - t].any()
    del y
    offsets = torch.tensor([0, n - t, n], device=device)
    y = gq.fp8_gemm(XQ, XS, torch.stack([Q.view(U8)] * 2).view(FP8), torch.stack([S + 1, S]), k, offsets=offsets)
    assert torch.equal(y[n - t:], want) and torch.equal(y[n // 2:n // 2 + t], (2 * (x @ w.T)).to(F32).to(BF))
    del y, XQ, XS
    # rows from the values, and back
    big = torch.zeros(n, k, device=device)
    big[n - t:] = x.float()
    q, s = gq.fp8_quantize(big)
    del big
    assert torch.equal(gq.fp8_dequantize(q, s, k, dtype=F32)[n - t:].double(), x)


def test_weights_past_32_bits(device):
    """Experts' weights of more than 4 GiB: the last one's outputs, and their gradients."""
    E, d_out, d_in, n = 300, 4096, 4096, 64
    Q = torch.zeros(E, d_out, d_in, dtype=U8, device=device).view(FP8)
    S = torch.full((E, 32, 32), 127, dtype=U8, device=device)
    q, s, w = packed_weight(device, (), d_out, d_in, U8, 6, seed=2)
    Q.view(U8)[-1], S[-1] = q.view(U8), s
    XQ, XS, x = packed_rows(device, n, d_in, U8, seed=1)
    offsets = torch.tensor([0] * (E - 1) + [n // 2, n], device=device)
    y = gq.fp8_gemm(XQ, XS, Q, S, d_in, offsets=offsets, out_dtype=F32)
    assert not y[:n // 2].any() and torch.equal(y[n // 2:].double(), x[n // 2:] @ w.T)
    y = gq.fp8_gemm_dx(XQ, XS, Q, S, d_in, offsets=offsets, out_dtype=F32)
    assert not y[:n // 2].any() and torch.equal(y[n // 2:].double(), x[n // 2:] @ w)


def test_gate_and_gradients_past_32_bits(device):
    """bfloat16 rows of more than 4 GiB and products of more than 2^31 elements."""
    n, d_in, d_ff, t = 1060000, 2304, 2048, 40
    x = torch.zeros(n, d_in, dtype=BF, device=device)
    last = integers(device, t, d_in, seed=1).to(BF)
    x[n - t:] = last
    G, U = (integers(device, d_ff, d_in, seed=s).to(BF) * 2.0 ** -6 for s in (2, 3))
    h, zg, zu = gq.ffn_gate(x, G, U, save=True)
    a = gq.ffn_gate(last, G, U, save=True)
    assert torch.equal(zg[n - t:].double(), last.double() @ G.double().T) and same((h[n - t:], zg[n - t:], zu[n - t:]), a)
    assert not h[:n - t].any()
    dh = torch.zeros(n, d_ff, dtype=BF, device=device)
    dh[n - t:] = integers(device, t, d_ff, seed=4).to(BF)
    dx, dG, dU = gq.ffn_gate_backward(dh, x, G, U, zg, zu)
    dzg, dzu = gq.ffn_gate_dz(dh[n - t:].clone(), zg[n - t:].clone(), zu[n - t:].clone())
    assert not dx[:n - t].any()
    # (another split of the sums: two roundings of 2^-8 apart, and the sums' own)
    for got, want, size in ((dx[n - t:], gq.ffn_gate_dx(dzg, dzu, G, U), dzg.abs().double() @ G.abs().double() + dzu.abs().double() @ U.abs().double()),
                            (dG, gq.ffn_gate_dw(dzg, dzu, last)[0], dzg.abs().double().T @ last.abs().double())):
        assert bool(((got.double() - want.double()).abs() <= 2.0 ** -7 * want.double().abs() + 4096 * 2.0 ** -22 * size).all())
