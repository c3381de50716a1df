"""GPU tests of the autograd functions over 8-bit checkpoints: which gradients they give or
refuse, the types they take under autocast, and what a captured step records."""
import ctypes

import pytest

from test_gpu_groups import B, L, tokens, torch  # noqa: F401  (fixtures and helpers)

pytestmark = pytest.mark.gpu

KERNEL, MEMSET = 0, 2    # hipGraphNodeType


def node_types(B, graph):
    """Types of the nodes of a torch.cuda.CUDAGraph that keeps its graph."""
    hip = B.lib()
    handle, count = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert hip.hipGraphGetNodes(handle, None, ctypes.byref(count)) == 0
    nodes = (ctypes.c_void_p * count.value)()
    assert hip.hipGraphGetNodes(handle, nodes, ctypes.byref(count)) == 0
    kinds = []
    for n in nodes:
        kind = ctypes.c_int(-1)
        assert hip.hipGraphNodeGetType(ctypes.c_void_p(n), ctypes.byref(kind)) == 0
        kinds.append(kind.value)
    return kinds


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("m,n", [(50000, 48), (8192, 1024), (3, 5)])
def test_bias_alone_in_a_graph(torch, B, dtype, m, n):
    """A frozen weight under a trained bias: the captured step clears no memory by a memset
    node, and every replay gives the eager gradient."""
    from integer_quantized_nn_amd import checkpoint as C
    dt = getattr(torch, dtype)
    x, w = tokens(torch, m, 64, dt, 1).cuda(), tokens(torch, n, 64, dt, 2).cuda()
    dy = tokens(torch, m, n, dt, 3).cuda()
    b0 = torch.zeros(n, device="cuda", dtype=dt)

    def step(b):
        return torch.autograd.grad(C.linear(x, w, b), b, dy)[0]

    held = b0.clone().requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step(held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        out = step(held)
    kinds = node_types(B, graph)
    assert KERNEL in kinds and MEMSET not in kinds, kinds
    for i in range(4):
        dy.copy_(tokens(torch, m, n, dt, 10 + i))
        graph.replay()
        got = out.clone()
        assert torch.equal(got, step(b0.clone().requires_grad_()))
        u = torch.finfo(dt).eps / 2
        want, mag = dy.double().sum(0), dy.double().abs().sum(0)
        assert ((got.double() - want).abs() <= (m + 4) * 2.0 ** -23 * mag + u * want.abs()).all()


def test_gradients_are_not_dropped(torch, L, B):
    """Calls without a derivative refuse an input that asks for one, in either mode."""
    from torch.autograd import forward_ad
    x = tokens(torch, 4, 64, torch.float32, 1).cuda()
    w = L.quantize_groups(x, B.INT4, group=32)
    lin = L.W4Linear(w[0], w[1], group=32, dtype=torch.float32)
    a = x.clone().requires_grad_()
    for call in (lambda v: lin(v), lambda v: L.ckpt_act(v, B.ACT_GELU)):
        with pytest.raises(ValueError, match="gradient"):
            call(a)
        with torch.no_grad():
            call(a)
        with torch.inference_mode():
            call(x)
        with forward_ad.dual_level():
            call(x)
            with pytest.raises(ValueError, match="gradient"):
                call(forward_ad.make_dual(x, torch.ones_like(x)))


def test_activation_without_gradient_keeps_no_codes(torch, L, B):
    """Where no gradient can be asked for, checkpoint.act allocates its result and nothing
    else, and gives the same values."""
    from integer_quantized_nn_amd import checkpoint as C
    for shape, group, gated in (((2048, 512), 128, False), ((2048, 512), 0, True), ((300, 6000), 0, False), ((33, 70), 32, True)):
        for dt in (torch.bfloat16, torch.float32):
            x = tokens(torch, *shape, dt, 1).cuda()
            p = x.clone().requires_grad_()
            want = C.act(p, B.ACT_SILU, group=group, gated=gated)
            assert want.requires_grad

            def check(v):
                torch.cuda.synchronize()
                torch.cuda.reset_peak_memory_stats()
                before = torch.cuda.memory_stats()["requested_bytes.all.current"]
                y = C.act(v, B.ACT_SILU, group=group, gated=gated)
                assert torch.cuda.memory_stats()["requested_bytes.all.peak"] - before == y.numel() * y.element_size()
                assert torch.equal(y, want) and not y.requires_grad

            check(x)
            for mode in (torch.no_grad, torch.inference_mode):
                with mode():
                    check(p)
            y, q, s = L.ckpt_act(x, B.ACT_SILU, group=group, gated=gated, save=False)
            assert q is None and s is None and torch.equal(y, want)


def test_mixed_types_under_autocast(torch, L, B):
    """A 16-bit activation and a float32 weight, as mixed precision brings them: under autocast
    all take its type, gradients come back in the leaves' own; outside it they are refused."""
    from integer_quantized_nn_amd import checkpoint as C
    w0, b0 = tokens(torch, 24, 64, torch.float32, 2).cuda(), tokens(torch, 1, 24, torch.float32, 4)[0].cuda()
    for dt in (torch.bfloat16, torch.float16):
        x0 = tokens(torch, 40, 64, dt, 1).cuda()
        dy = tokens(torch, 40, 24, dt, 3).cuda()
        x, w, b = (t.clone().requires_grad_() for t in (x0, w0, b0))
        with torch.autocast("cuda", dtype=dt):
            y = C.linear(x, w, b, group=32)
        assert y.dtype == dt
        y.backward(dy)
        assert x.grad.dtype == dt and w.grad.dtype == torch.float32 and b.grad.dtype == torch.float32
        xc, wc, bc = (t.to(dt).requires_grad_() for t in (x0, w0, b0))
        yc = C.linear(xc, wc, bc, group=32)
        yc.backward(dy)
        assert torch.equal(y, yc) and torch.equal(x.grad, xc.grad)
        assert torch.equal(w.grad, wc.grad.float()) and torch.equal(b.grad, bc.grad.float())
        with torch.autocast("cuda", dtype=dt):      # only the bias differs; a type that none of them has
            assert C.linear(x0, w0.to(dt), b0).dtype == dt
            with pytest.raises(ValueError):
                C.linear(x0, w0.double())
        with pytest.raises(ValueError):
            C.linear(x0, w0)
