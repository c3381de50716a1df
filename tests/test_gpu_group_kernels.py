"""GPU tests that reach every kernel the group-scaled operators choose among, and what only
some of them do: products of binary32 operands in pieces, launches of 2^32 threads and more."""
import numpy as np
import pytest

from test_gpu_groups import (  # noqa: F401  (fixtures and helpers)
    B, L, assert_within, check_w4, check_wgrad, make_codes, make_w4, tokens, torch)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------- binary32 operands in pieces

def full_floats(torch, g, *shape):
    """Floats whose 24 significand bits are all at random, of either sign, 2^-3 to 2^4."""
    v = (1 + torch.rand(*shape, generator=g)) * torch.exp2(torch.randint(-3, 4, shape, generator=g).float())
    return torch.where(torch.rand(*shape, generator=g) < 0.5, -v, v).cuda()


@pytest.mark.parametrize("dtype", ["float32", "float16"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("n,k", [(192, 320), (190, 322), (2048, 2048), (2050, 2054)])
def test_wgrad_products_keep_every_piece(torch, L, dtype, group, n, k):
    """One row of dY alone: each gradient is one product dY * (q S) in pieces of bfloat16.
    Off by the rounding of q S or dY S (2^-24), five more sums of the six pieces' products at
    a full step each (2^-23; the first is exact) and the products left out (2^-23.9); a
    piece's product lost would show at up to 2^-14."""
    g = torch.Generator().manual_seed(n + group)
    m = 40
    q = torch.randint(-127, 128, (m, k), generator=g).to(torch.int8).cuda()
    s = full_floats(torch, g, m, -(-k // group) if group else 1).abs()
    for r in (0, 37):
        dy = torch.zeros(m, n, device="cuda", dtype=getattr(torch, dtype))
        dy[r] = full_floats(torch, g, n).to(dy.dtype)
        dw, db = L.ckpt_wgrad(dy, q, s, group=group, out_dtype=torch.float32, bias=True)
        wide = s[r].double().repeat_interleave(group)[:k] if group else s[r].double()
        want = dy[r].double()[:, None] * (q[r].double() * wide)[None]
        assert_within(dw, want, want.abs() * (2.0 ** -24 + 5 * 2.0 ** -23 + 2.0 ** -23.9), (r, n, k))
        assert torch.equal(db, dy[r].float())


@pytest.mark.parametrize("n,k", [(64, 64), (72, 66), (2048, 2048), (2056, 2050)])
def test_wgrad_products_lean_to_no_side(torch, L, n, k):
    """Both operands 1 + 2^-7 - 2^-23 (times powers of two).  The nearest bfloat16 leaves a
    second piece of -2^-23, and three of the pieces' products need a rounding, at most a full
    step of 2^-23 each.  Pieces cut off towards zero leave out 4 - 2^-6 such steps."""
    v = float(np.array([0x3F80FFFF], np.uint32).view(np.float32)[0])
    g = torch.Generator().manual_seed(3)
    m, r = 33, 32
    e = torch.exp2(torch.randint(-8, 9, (n,), generator=g).float()).cuda()
    dy = torch.zeros(m, n, device="cuda")
    dy[r] = v * e
    q = torch.exp2(torch.randint(0, 7, (m, k), generator=g).float()).cuda()
    q = torch.where(torch.rand(m, k, generator=g).cuda() < 0.5, -q, q)
    s = torch.full((m, -(-k // 32)), v, device="cuda")
    dw, _ = L.ckpt_wgrad(dy, q.to(torch.int8), s, group=32)
    units = e.double()[:, None] * q[r].double()[None]          # powers of two
    assert_within(dw.double() / units, torch.full((n, k), v, dtype=torch.float64) * v, 3 * 2.0 ** -23, (n, k))


@pytest.mark.parametrize("zp", [False, True])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("k", [264, 266])
def test_w4_float_products_keep_every_piece(torch, L, B, zp, group, k):
    """One element of each row of x: y is one product x (q - z) S.  The three pieces' products
    are exact, two sums of them are off by a full step of 2^-23 at most, the scale adds 2^-24."""
    g = torch.Generator().manual_seed(k + group)
    for n in (40, 2560, 12293):
        q, s, z, _ = make_w4(torch, L, B, n, k, group, zp, n)
        lin = L.W4Linear(q, s, z, group=group, dtype=torch.float32)
        codes = torch.stack([q & 15, q >> 4], 2).flatten(1).double()
        wide = lambda t: (t.double().repeat_interleave(group, 1)[:, :k] if group else t.double().expand(-1, k))
        w = (codes - wide(z) if zp else torch.where(codes >= 8, codes - 16, codes)) * wide(s)
        for m in (3, 7, 15, 40, 512):
            at = torch.randint(0, k, (m,), generator=g).cuda()
            v = full_floats(torch, g, m)
            x = torch.zeros(m, k, device="cuda")
            x[torch.arange(m, device="cuda"), at] = v
            want = v.double()[:, None] * w.t()[at]
            assert_within(lin(x), want, want.abs() * (2 * 2.0 ** -23 + 2.0 ** -24 + 2.0 ** -44), (m, n))


@pytest.mark.parametrize("dtype", ["float32", "float16"])
@pytest.mark.parametrize("n,k", [(72, 66), (2056, 2050)])
def test_wgrad_pieces_of_the_largest_and_of_infinities(torch, L, dtype, n, k):
    """Finite operands whose nearest bfloat16 would be infinite stay exact; an infinity in dY
    makes its own row non-finite, one in the scales its group's columns, and nothing else."""
    m, r, dt = 33, 7, getattr(torch, dtype)
    top = torch.finfo(dt).max
    dy = torch.zeros(m, n, device="cuda", dtype=dt)
    dy[r] = 2.0 ** -14                       # exact in both types
    dy[r, 5], dy[r, 6] = top, -top
    q = torch.ones(m, k, dtype=torch.int8, device="cuda")
    s = torch.full((m, -(-k // 32)), 2.0 ** -20, device="cuda")
    s[:, 1] = torch.finfo(torch.float32).max
    dw, db = L.ckpt_wgrad(dy, q, s, group=32, out_dtype=torch.float32, bias=True)
    want = dy[r].double()[:, None] * s[r].double().repeat_interleave(32)[:k][None]
    keep = want.abs() < 2.0 ** 127
    assert_within(dw[keep], want[keep], want[keep].abs() * (5 * 2.0 ** -23 + 2.0 ** -23.9), (n, k))
    assert torch.equal(db, dy[r].float())
    s[:, 1] = 2.0 ** -20
    dy[r, 5] = float("inf")
    good = torch.ones(n, dtype=torch.bool, device="cuda")
    good[5] = False
    dw, db = L.ckpt_wgrad(dy, q, s, group=32, out_dtype=torch.float32, bias=True)
    assert not torch.isfinite(dw[5]).any() and torch.isfinite(dw[good]).all() and torch.isinf(db[5]) and torch.isfinite(db[good]).all()
    dy[r, 5] = 1.0
    s[r, 1] = float("inf")
    dw, _ = L.ckpt_wgrad(dy, q, s, group=32, out_dtype=torch.float32)
    assert not torch.isfinite(dw[:, 32:64]).any() and torch.isfinite(dw[:, :32]).all() and torch.isfinite(dw[:, 64:]).all()


# ------------------------------------------------------------- every kernel choice

# rows and output columns at which the choice falls on each kernel (K of them all 264 or 266,
# which ends inside a block of 128): up to 4, 8 and 16 rows with few and many columns, then
# tiles of 32 x 64, 64 x 64, 64 x 128, 128 x 128 and 128 x 128 two to a CU, and f32's 64 x 128
W4_CHOICES = [(m, n) for m in (2, 4, 6, 8, 13, 16) for n in (77, 12293)] + [
    (17, 70), (500, 2040), (509, 4090), (1020, 4090), (2035, 4089), (505, 2555)]


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("zp", [False, True])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("k", [264, 266])
def test_w4_every_kernel(torch, L, B, dtype, zp, group, k):
    dt = getattr(torch, dtype)
    for n in sorted({n for _, n in W4_CHOICES}):
        q, s, z, w = make_w4(torch, L, B, n, k, group, zp, n + group)
        bias = tokens(torch, 1, n, dt, n)[0].cuda()
        lin = L.W4Linear(q, s, z, group=group, bias=bias, dtype=dt)
        for m in [m for m, nn in W4_CHOICES if nn == n]:
            x = tokens(torch, m, k, dt, m).cuda()
            y = lin(x)
            check_w4(torch, y, x, w, bias, group, (m, n, k))
            assert torch.equal(lin(x), y)


@pytest.mark.parametrize("m,n,k,group", [(2049, 520, 1040, 32), (2090, 512, 1024, 0), (70, 2056, 2064, 64), (1, 2056, 2064, 128),
                                         (33, 2200, 2024, 128), (257, 2058, 2050, 32), (257, 2058, 2050, 0), (96, 2048, 4096, 128)])
def test_wgrad_f16_to_float_many_tiles(torch, L, B, m, n, k, group):
    """Two pieces of dY, folded scales and not, in the larger tiles."""
    q, s = make_codes(torch, L, B, m, k, group, m)
    dy = tokens(torch, m, n, torch.float16, n).cuda()
    dw, db = L.ckpt_wgrad(dy, q, s, group=group, out_dtype=torch.float32, bias=True)
    check_wgrad(torch, dw, db, dy, q, s, group, (m, n, k))
    again, none = L.ckpt_wgrad(dy, q, s, group=group, out_dtype=torch.float32)
    assert none is None and torch.equal(again, dw)


# ------------------------------------------------ launches of 2^32 threads and more

def halves_equal(torch, call, whole, rows, *inputs):
    """Every output of `call` on all rows is that of its two halves, which stay below 2^32
    threads a launch."""
    half = rows // 2
    for lo, hi in ((0, half), (half, rows)):
        for a, b in zip(whole, call(*[t[lo:hi] for t in inputs])):
            assert torch.equal(a[lo:hi], b)


@pytest.mark.parametrize("rows,cols,group", [((1 << 26) + 3, 16, 0), ((1 << 28) + 3, 1, 128)])
def test_group_codes_past_a_launch(torch, L, B, rows, cols, group):
    """A wave for each of 2^26 rows, and 16 threads for each of 2^28."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16)
    quant = lambda v: L.quantize_groups(v, B.INT8, group=group)[:2]
    q, s = quant(x)
    halves_equal(torch, quant, (q, s), rows, x)
    back = lambda a, b: (L.dequantize_groups(a, b, None, B.INT8, group=group, dtype=torch.bfloat16),)
    halves_equal(torch, back, back(q, s), rows, q, s)
    act = lambda v: L.ckpt_act(v, B.ACT_GELU, group=group)
    y, aq, sa = act(x)
    halves_equal(torch, act, (y, aq, sa), rows, x)
    grad = lambda d, a, b: (L.ckpt_act_bwd(d, a, b, B.ACT_GELU, group=group),)
    halves_equal(torch, grad, grad(y, aq, sa), rows, y, aq, sa)


def test_w4_past_a_launch(torch, L, B):
    """512 threads for every 16 of 2^27 output columns, and for every 64 of 2^29 rows; a block
    that fills up the last row of blocks stores nothing."""
    g = torch.Generator(device="cuda").manual_seed(1)
    n = (1 << 27) + 5
    q = torch.randint(0, 256, (n, 1), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.rand(n, 1, generator=g, device="cuda")
    x = torch.randn(2, 2, generator=g, device="cuda").bfloat16()
    y = L.W4Linear(q, s, group=128)(x)
    for part in (slice(0, n // 2), slice(n // 2, n)):
        assert torch.equal(y[:, part], L.W4Linear(q[part], s[part], group=128)(x))
    del q, s, y
    rows = (1 << 29) + 5
    x = torch.randn(rows, 2, generator=g, device="cuda", dtype=torch.float16)
    lin = L.W4Linear(torch.full((1, 1), 0x2D, dtype=torch.uint8, device="cuda"), torch.full((1, 1), 0.75, device="cuda"),
                     group=128, dtype=torch.float16)
    buf = torch.full((rows + 1, 1), 7.0, device="cuda", dtype=torch.float16)
    lin(x, out=buf[:rows])
    assert buf[rows].item() == 7.0
    halves_equal(torch, lambda v: (lin(v),), (buf[:rows],), rows, x)
    check_w4(torch, buf[rows - 3:rows], x[-3:], torch.tensor([[-3.0 * 0.75, 2.0 * 0.75]], device="cuda"), None, 128, "last rows")


def test_wgrad_past_a_launch(torch, L):
    """512 threads for every 128 of 2^30 columns."""
    g = torch.Generator(device="cuda").manual_seed(2)
    k = 1 << 30
    q = torch.randint(-127, 128, (1, k), generator=g, device="cuda", dtype=torch.int8)
    s = torch.rand(1, k // 128, generator=g, device="cuda")
    dy = torch.full((1, 1), 1.5, device="cuda", dtype=torch.bfloat16)
    dw, db = L.ckpt_wgrad(dy, q, s, bias=True)
    for part in (slice(0, k // 2), slice(k // 2, k)):
        want, _ = L.ckpt_wgrad(dy, q[:, part], s[:, part.start // 128:part.stop // 128])
        assert torch.equal(dw[:, part], want)
    assert db.item() == 1.5 and dw[:, -1].item() != 0
