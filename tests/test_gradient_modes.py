"""What the products do where torch follows a call by other means than a backward pass: nothing is lost without a word.

Refusals come before any launch, so host tensors show them.
"""
import pytest
import torch
import torch.autograd.forward_ad as fw

import post_weight_quantization_gq_amd as gq
from post_weight_quantization_gq_amd import binding as B

BF, F32, U8, FP8 = torch.bfloat16, torch.float32, torch.uint8, torch.float8_e4m3fn


def refused(fn, *a, **k):
    with pytest.raises(B.GQError) as e:
        fn(*a, **k)
    return e.value


# ---- forward mode -----------------------------------------------------------------------

def _forward_mode_calls(x, G, z, dz):
    at = dict(x=x, G=G, U=G)
    yield "ffn_gate", gq.ffn_gate, at, "xGU"
    yield "ffn_gate_dz", gq.ffn_gate_dz, dict(dh=z, zg=z, zu=z), ("dh", "zg", "zu")
    yield "ffn_gate_dx", gq.ffn_gate_dx, dict(dzg=dz, dzu=dz, G=G, U=G), ("dzg", "dzu", "G", "U")
    yield "ffn_gate_dw", gq.ffn_gate_dw, dict(dzg=dz, dzu=dz, x=x), ("dzg", "dzu", "x")
    yield "ffn_gate_backward", gq.ffn_gate_backward, dict(dh=z, x=x, G=G, U=G, zg=z, zu=z), ("dh", "x", "G", "U", "zg", "zu")
    Q, S = torch.zeros(64, 128, dtype=U8), torch.zeros(64, 8, dtype=U8)
    yield "mxfp4_gemm", gq.mxfp4_gemm, dict(x=x, Q=Q, S=S), "x"
    yield "mxfp4_gemm_dx", gq.mxfp4_gemm_dx, dict(g=dz, Q=Q, S=S, d_in=200), "g"


def test_tangents_are_refused():
    x, G = torch.zeros(5, 200, dtype=BF), torch.zeros(64, 200, dtype=BF)
    z, dz = torch.zeros(5, 64), torch.zeros(5, 64, dtype=BF)
    with fw.dual_level():
        for name, fn, given, follows in _forward_mode_calls(x, G, z, dz):
            assert "GPU tensor" in refused(fn, **given).message, name            # a level alone changes nothing
            for p in follows:
                dual = fw.make_dual(given[p], torch.ones_like(given[p]))
                for mode in (torch.enable_grad, torch.no_grad):
                    with mode():
                        e = refused(fn, **{**given, p: dual})
                        assert e.status == B.GQ_EINVAL and "tangent" in e.message and e.message.startswith(p), (name, p)


@pytest.mark.gpu
def test_tangents_are_refused_on_the_gpu(device):
    """and a level without them gives the same values."""
    x, G = torch.randn(9, 200, device=device).to(BF), torch.randn(64, 200, device=device).to(BF)
    want = gq.ffn_gate(x, G, G)
    with fw.dual_level():
        assert torch.equal(gq.ffn_gate(x, G, G), want)
        with pytest.raises(B.GQError, match="tangent"):
            gq.ffn_gate(fw.make_dual(x, torch.ones_like(x)), G, G)
    assert torch.equal(gq.ffn_gate(x, G, G), want)


# ---- float32 scales ---------------------------------------------------------------------

def _scaled_calls(device, lead):
    """(name, call, its float32 scales) of everything that reads scales."""
    n, d_in, d_out = 5, 200, 130
    codes = lambda *shape: torch.zeros(shape, dtype=U8, device=device).view(FP8)
    ones = lambda *shape: torch.ones(shape, device=device)
    X, G = (codes(n, 256), ones(n, 4)), (codes(n, 256), ones(n, 4))
    W = (codes(*lead, d_out, 256), ones(*lead, 2, 2))
    off = dict(offsets=torch.tensor([0, 2, 5], device=device)) if lead else {}
    yield "dequantize", lambda xs: gq.fp8_dequantize(X[0], xs, d_in), [X[1]]
    yield "dequantize_weight", lambda s: gq.fp8_dequantize_weight(W[0], s, d_in), [W[1]]
    yield "gemm", lambda xs, s: gq.fp8_gemm(X[0], xs, W[0], s, d_in, **off), [X[1], W[1]]
    yield "gemm_dx", lambda gs, s: gq.fp8_gemm_dx(G[0], gs, W[0], s, d_in, **off), [G[1], W[1]]
    for packed in (False, True):
        yield "gate", lambda xs, g, u: gq.fp8_ffn_gate(X[0], xs, W[0], g, W[0], u, d_in, packed=packed, **off), [X[1], W[1], W[1]]


@pytest.mark.gpu
@pytest.mark.parametrize("lead", [(), (2,)])
def test_scales_that_require_a_gradient(device, lead):
    """are refused while gradients are recorded, and tangents of them too; else the values are the same."""
    for name, fn, scales in _scaled_calls(device, lead):
        value = lambda t: t[0].view(U8) if isinstance(t, tuple) else t
        want = value(fn(*scales))
        for i in range(len(scales)):
            some = [s.clone().requires_grad_(i == k) for k, s in enumerate(scales)]
            with pytest.raises(B.GQError, match="requires a gradient") as e:
                fn(*some)
            assert e.value.status == B.GQ_EINVAL
            with torch.no_grad():
                assert torch.equal(value(fn(*some)), want)
            some[i] = some[i].detach()
            assert torch.equal(value(fn(*some)), want)
            with fw.dual_level():
                assert torch.equal(value(fn(*some)), want)
                some[i] = fw.make_dual(some[i], torch.ones_like(some[i]))
                with pytest.raises(B.GQError, match="tangent"):
                    fn(*some)


# ---- traces -----------------------------------------------------------------------------

class _Counts(torch.utils._python_dispatch.TorchDispatchMode):
    """A mode that only looks on, as counters of operations do."""
    seen = 0

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        _Counts.seen += 1
        return func(*args, **(kwargs or {}))


@pytest.mark.gpu
def test_traces_are_refused(device):
    """A traced call would give memory that nothing has filled; modes that only look on are not meant."""
    from torch.fx.experimental.proxy_tensor import make_fx
    x, w = torch.randn(5, 256, device=device).to(BF), torch.randn(130, 256, device=device).to(BF)
    XQ, XS = gq.fp8_quantize(x)
    Q, S = gq.fp8_quantize_weight(w)
    M = gq.mxfp4_quantize(w)
    GQ, GS = gq.fp8_quantize(torch.randn(5, 130, device=device))
    h, zg, zu = gq.ffn_gate(x, w, w, save=True)
    y = [torch.empty_like(h)]
    leaf = x.clone().requires_grad_()
    calls = [
        (gq.fp8_quantize, (x,)), (gq.fp8_quantize_weight, (w,)), (lambda q, s: gq.fp8_dequantize(q, s, 256), (XQ, XS)),
        (lambda q, s: gq.fp8_dequantize_weight(q, s, 256), (Q, S)), (lambda *t: gq.fp8_gemm(*t, 256), (XQ, XS, Q, S)),
        (lambda *t: gq.fp8_gemm(*t, 256, y=y[0], ws=False), (XQ, XS, Q, S)),
        (lambda *t: gq.fp8_gemm_dx(*t, 256), (GQ, GS, Q, S)), (lambda *t: gq.fp8_ffn_gate(*t, Q, S, 256), (XQ, XS, Q, S)),
        (lambda *t: gq.fp8_ffn_gate(*t, Q, S, 256, packed=True), (XQ, XS, Q, S)), (gq.ffn_gate, (x, w, w)), (gq.ffn_gate, (leaf, w, w)),
        (gq.ffn_gate_dz, (h, zg, zu)), (gq.ffn_gate_dx, (h, h, w, w)), (gq.ffn_gate_dw, (h, h, x)),
        (gq.ffn_gate_backward, (h, x, w, w, zg, zu)), (gq.mxfp4_quantize, (w,)), (lambda *t: gq.mxfp4_gemm(x, *t), M)]
    for fn, args in calls:
        print("traced:", fn, flush=True)
        alone = lambda *t: fn(*t)                                              # (no arguments by name)
        with pytest.raises(B.GQError, match="traced"):
            make_fx(alone)(*args)
        with pytest.raises(B.GQError, match="traced"):
            torch.jit.trace(alone, args, check_trace=False)
    with _Counts():
        assert torch.equal(gq.ffn_gate(x, w, w), h)
    assert _Counts.seen > 0


# ---- gradients of gradients -------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("mask", [(1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1)])
@pytest.mark.parametrize("given", [False, True])
def test_a_gradient_that_depends_on_the_gates_is_refused(device, mask, given):
    """Also where the gradient of h requires none, and beside a term that has a gradient."""
    x, G, U = (torch.randn(s, device=device).to(BF) for s in ((9, 200), (64, 200), (64, 200)))
    leaves = [t.requires_grad_(bool(m)) for t, m in zip((x, G, U), mask)]
    needed = [t for t in leaves if t.requires_grad]
    dh = torch.randn(9, 64, device=device).to(BF).requires_grad_(given)
    want = torch.autograd.grad(gq.ffn_gate(*leaves), needed, dh.detach())
    h = gq.ffn_gate(*leaves)
    got = torch.autograd.grad(h, needed, dh, create_graph=True)
    assert all(torch.equal(a, b) and a.requires_grad for a, b in zip(got, want))
    # a penalty beside the loss: its part of the gradient cannot be left out
    with pytest.raises(B.GQError, match="not differentiable"):
        (h.float().sum() + got[0].float().square().sum()).backward()
    # the loss alone has its gradient, with a graph or without
    for t in needed:
        t.grad = None
    gq.ffn_gate(*leaves).backward(dh.detach(), create_graph=given)
    assert all(torch.equal(t.grad, w) for t, w in zip(needed, want))
    for t in needed:
        t.grad = None


# ---- hooks of saved tensors -------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("experts", [None, 3])
def test_saved_tensors_that_hooks_change(device, experts):
    """Kept on the host and brought back: the same gradients.  Given back as anything but what was saved: refused, before
    a kernel reads it."""
    lead = (experts,) if experts else ()
    x, G, U = (torch.randn(s, device=device).to(BF).requires_grad_() for s in ((9, 200), (*lead, 64, 200), (*lead, 64, 200)))
    offsets = torch.tensor([0, 3, 3, 8], device=device) if experts else None
    dh = torch.randn(9, 64, device=device).to(BF)
    step = lambda: torch.autograd.grad(gq.ffn_gate(x, G, U, offsets=offsets), (x, G, U), dh)
    want = step()
    with torch.autograd.graph.save_on_cpu():
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
    changes = dict(host=lambda t: t.cpu(), type=lambda t: t.to(torch.float16), part=lambda t: t[..., :-1].contiguous(),
                   flat=lambda t: t.flatten(), strides=lambda t: t.transpose(-1, -2).contiguous().transpose(-1, -2) if t.dim() > 1 else t[::2])
    count = 5 if experts else 4
    for name, change in changes.items():
        for which in range(count):
            place = []

            def pack(t):
                place.append(t)
                return len(place) - 1

            def unpack(i):
                return change(place[i]) if i == which else place[i]

            if name == "flat" and which == 4:              # (offsets are flat)
                continue
            print(name, which, flush=True)
            with torch.autograd.graph.saved_tensors_hooks(pack, unpack):
                h = gq.ffn_gate(x, G, U, offsets=offsets)
            assert len(place) == count
            with pytest.raises(B.GQError):
                torch.autograd.grad(h, (x, G, U), dh)


# ---- outputs of the caller's ------------------------------------------------------------

def _writing_calls(device):
    """(name, call that writes into the given tensors, those tensors)."""
    n, d, f = 5, 200, 136
    x, w = torch.randn(n, d, device=device).to(BF), torch.randn(f, d, device=device).to(BF)
    dh = torch.randn(n, f, device=device).to(BF)
    new = lambda *shape, dtype=BF: torch.zeros(shape, device=device, dtype=dtype)
    X, W = gq.fp8_quantize(x, scales=F32), gq.fp8_quantize_weight(w, scales=F32)
    g8, M, XM = gq.fp8_quantize(dh, scales=F32), gq.mxfp4_quantize(w), gq.mxfp4_quantize(x)
    h, zg, zu = gq.ffn_gate(x, w, w, save=True)
    codes = lambda *shape: new(*shape, dtype=U8).view(FP8)
    yield "fp8_quantize", lambda q, s: gq.fp8_quantize(x, Q=q, S=s), [codes(n, 256), new(n, 4, dtype=F32)]
    yield "fp8_quantize_weight", lambda q, s: gq.fp8_quantize_weight(w, Q=q, S=s), [codes(f, 256), new(2, 2, dtype=F32)]
    yield "fp8_dequantize", lambda y: gq.fp8_dequantize(*X, d, y=y), [new(n, d)]
    yield "fp8_dequantize_weight", lambda y: gq.fp8_dequantize_weight(*W, d, y=y), [new(f, d)]
    yield "fp8_gemm", lambda y: gq.fp8_gemm(*X, *W, d, y=y), [new(n, f)]
    yield "fp8_gemm_dx", lambda y: gq.fp8_gemm_dx(*g8, *W, d, y=y), [new(n, d)]
    yield "fp8_ffn_gate", lambda y: gq.fp8_ffn_gate(*X, *W, *W, d, y=y), [new(n, f)]
    yield ("fp8_ffn_gate packed", lambda q, s: gq.fp8_ffn_gate(*X, *W, *W, d, packed=True, HQ=q, HS=s),
           [codes(n, 256), new(n, 4, dtype=F32)])
    yield "ffn_gate", lambda y: gq.ffn_gate(x, w, w, y=y), [new(n, f)]
    yield "ffn_gate_dz", lambda a, b: gq.ffn_gate_dz(dh, zg, zu, dzg=a, dzu=b), [new(n, f), new(n, f)]
    yield "ffn_gate_dx", lambda y: gq.ffn_gate_dx(dh, dh, w, w, y=y), [new(n, d)]
    yield "ffn_gate_dw", lambda a, b: gq.ffn_gate_dw(dh, dh, x, dG=a, dU=b), [new(f, d), new(f, d)]
    yield ("ffn_gate_backward", lambda a, b, c: gq.ffn_gate_backward(dh, x, w, w, zg, zu, dx=a, dG=b, dU=c),
           [new(n, d), new(f, d), new(f, d)])
    yield "mxfp4_quantize", lambda q, s: gq.mxfp4_quantize(w, Q=q, S=s), [new(f, 128, dtype=U8), new(f, 8, dtype=U8)]
    yield "mxfp4_dequantize", lambda y: gq.mxfp4_dequantize(*M, d, y=y), [new(f, d)]
    yield "mxfp4_gemm", lambda y: gq.mxfp4_gemm(x, *M, y=y), [new(n, f)]
    yield "mxfp4_gemm_mx", lambda y: gq.mxfp4_gemm_mx(*XM, *M, d, y=y), [new(n, f)]
    yield "mxfp4_gemm_dx", lambda y: gq.mxfp4_gemm_dx(dh, *M, d, y=y), [new(n, d)]


@pytest.mark.gpu
def test_given_outputs_are_changed_in_place(device):
    """A backward pass that has saved an output's old values refuses; an output that requires a gradient is refused while
    gradients are recorded."""
    for name, fn, outs in _writing_calls(device):
        for i, out in enumerate(outs):
            print(name, i, flush=True)
            if out.dtype in (BF, F32):
                leaf = torch.ones_like(out, requires_grad=True)
                product = (out * leaf).sum()
                fn(*outs)
                with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                    product.backward()
                some = [o.clone().requires_grad_(i == k) if k == i else o for k, o in enumerate(outs)]
                with pytest.raises(B.GQError, match="requires a gradient"):
                    fn(*some)
                with torch.no_grad():
                    fn(*some)
                assert torch.equal(some[i], out)
            else:
                before = out._version
                fn(*outs)
                assert out._version > before
    with torch.inference_mode():
        for name, fn, outs in _writing_calls(device):
            fn(*outs)


# ---- streams ----------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("experts", [None, 3])
def test_a_gate_on_a_stream_of_its_own(device, experts):
    """The forward pass on a given stream, the gradient asked for on another: the backward pass follows the forward one's
    stream, and its results the asker's."""
    n, d_in, d_ff = 600, 512, 1000
    lead = (experts,) if experts else ()
    offsets = torch.tensor([0, 200, 200, 550], device=device) if experts else None
    G, U = ((torch.randn(*lead, d_ff, d_in, device=device) * 0.04).to(BF).requires_grad_() for _ in range(2))
    xs = [torch.randn(n, d_in, device=device).to(BF).requires_grad_() for _ in range(4)]
    dhs = [torch.randn(n, d_ff, device=device).to(BF) for _ in range(4)]
    want = [torch.autograd.grad(gq.ffn_gate(x, G, U, offsets=offsets), (x, G, U), dh) for x, dh in zip(xs, dhs)]
    here, side = torch.cuda.current_stream(), torch.cuda.Stream()
    side.wait_stream(here)
    for turn in range(8):
        x, dh = xs[turn % 4], dhs[turn % 4]
        h = gq.ffn_gate(x, G, U, offsets=offsets, stream=side)
        here.wait_stream(side)
        got = torch.autograd.grad(h, (x, G, U), dh * 1)
        del h
        torch.empty(3 * n * d_ff, device=device).fill_(float("nan"))         # over whatever has been freed here
        assert all(torch.equal(a, b) for a, b in zip(got, want[turn % 4])), turn
