"""Codes with group scales, without a GPU: every entry point refuses what include/iqnn.h
excludes before any launch (the pointers here are never read), and the sizes of packed
weights and workspaces."""
import ctypes

import pytest

from integer_quantized_nn_amd import binding as B

P = 0x10000          # an aligned address that no call here may touch
INVALID, UNSUPPORTED, ALIGNMENT = 1, 2, 3


def refused(status, word, fn, *args, **kw):
    with pytest.raises(B.IqnnError) as e:
        fn(*args, stream=0, **kw)
    assert e.value.status == status and word in str(e.value), str(e.value)


def quant(x=P, x_type=B.FLOAT32, rows=2, cols=64, ldx=64, group=32, q=P, qtype=B.INT8, scale=P, zp=P):
    return x, x_type, rows, cols, ldx, group, q, qtype, scale, zp


@pytest.mark.parametrize("kw,status,word", [
    (dict(x_type=3), INVALID, "floating-point"), (dict(x_type=-1), INVALID, "floating-point"),
    (dict(qtype=B.INT32), INVALID, "code type"), (dict(qtype=B.INT8_2OF4), INVALID, "code type"),
    (dict(group=16), INVALID, "group"), (dict(group=-1), INVALID, "group"), (dict(group=256), INVALID, "group"),
    (dict(rows=-1), INVALID, "sizes"), (dict(cols=0), INVALID, "sizes"), (dict(ldx=63), INVALID, "stride"),
    (dict(cols=63, qtype=B.INT4), INVALID, "even"), (dict(cols=63, qtype=B.UINT4), INVALID, "even"),
    (dict(x=0), INVALID, "null"), (dict(q=0), INVALID, "null"), (dict(scale=0), INVALID, "null"),
    (dict(zp=0, qtype=B.UINT8), INVALID, "null"),
    (dict(x=P + 2), ALIGNMENT, "misaligned"), (dict(x=P + 1, x_type=B.FLOAT16), ALIGNMENT, "misaligned"),
    (dict(scale=P + 2), ALIGNMENT, "misaligned"), (dict(zp=P + 1, qtype=B.UINT4), ALIGNMENT, "misaligned"),
    (dict(cols=2 ** 31, ldx=2 ** 31), UNSUPPORTED, "2^30"), (dict(rows=2 ** 41), UNSUPPORTED, "2^40"),
    (dict(rows=2 ** 40, ldx=2 ** 40), UNSUPPORTED, "2^46"), (dict(ldx=2 ** 62), UNSUPPORTED, "2^46"),
    # 2^40 rows of 2 units: more blocks than a launch holds
    (dict(rows=2 ** 40, cols=1, ldx=1), UNSUPPORTED, "blocks"),
])
def test_quantize_groups_refusals(kw, status, word):
    a = quant(**kw)
    refused(status, word, B.iqnn_quantize_groups, *a)
    x, x_type, rows, cols, ldx, group, q, qtype, scale, zp = a
    refused(status, word, B.iqnn_dequantize_groups, q, qtype, rows, cols, group, scale, zp, x, x_type, ldx)


def test_no_rows_is_valid_without_pointers():
    B.iqnn_quantize_groups(*quant(x=0, q=0, scale=0, zp=0, rows=0), stream=0)
    B.iqnn_dequantize_groups(0, B.UINT4, 0, 64, 32, 0, 0, 0, B.FLOAT16, 64, stream=0)
    B.iqnn_ckpt_act_fwd(0, B.FLOAT32, 0, 8, 8, B.ACT_GELU, False, 32, 0, 8, 0, 0, stream=0)
    B.iqnn_ckpt_act_bwd(0, B.FLOAT32, 0, 8, 8, B.ACT_GELU, True, 0, 0, 0, 0, 16, stream=0)
    B.iqnn_w4_fwd(w4(), 0, 0, 64, 0, 0, 0, 8, stream=0)


def act(x=P, t=B.FLOAT32, rows=2, cols=64, ld=64, kind=B.ACT_SILU, gated=False, group=32, y=P, ldy=64, q=P, s=P):
    return x, t, rows, cols, ld, kind, gated, group, y, ldy, q, s


@pytest.mark.parametrize("kw,status,word", [
    (dict(t=7), INVALID, "floating-point"), (dict(kind=4), INVALID, "activation"), (dict(kind=-1), INVALID, "activation"),
    (dict(group=96), INVALID, "group"), (dict(ld=60), INVALID, "stride"), (dict(ldy=60), INVALID, "stride"),
    (dict(gated=True, ld=127), INVALID, "stride"), (dict(rows=-2), INVALID, "sizes"),
    (dict(x=0), INVALID, "null"), (dict(y=0), INVALID, "null"), (dict(q=0), INVALID, "null"), (dict(s=0), INVALID, "null"),
    (dict(y=P + 2), ALIGNMENT, "misaligned"), (dict(s=P + 1), ALIGNMENT, "misaligned"),
])
def test_ckpt_act_refusals(kw, status, word):
    x, t, rows, cols, ld, kind, gated, group, y, ldy, q, s = act(**kw)
    refused(status, word, B.iqnn_ckpt_act_fwd, x, t, rows, cols, ld, kind, gated, group, y, ldy, q, s)
    # backward: dy has y's stride, dx has x's
    refused(status, word, B.iqnn_ckpt_act_bwd, y, t, rows, cols, ldy, kind, gated, group, q, s, x, ld)


def w4(n=8, k=64, w_type=B.INT4, x_type=B.BFLOAT16, group=32):
    d = B.W4Desc()
    d.n, d.k, d.w_type, d.x_type, d.group = n, k, w_type, x_type, group
    return d


@pytest.mark.parametrize("kw,status,word", [
    (dict(n=0), INVALID, "positive"), (dict(k=-2), INVALID, "positive"), (dict(k=63), INVALID, "even"),
    (dict(w_type=B.INT8), INVALID, "INT4"), (dict(x_type=5), INVALID, "floating-point"), (dict(group=48), INVALID, "group"),
    (dict(n=2 ** 31), UNSUPPORTED, "2^30"), (dict(n=2 ** 29, k=2 ** 29), UNSUPPORTED, "2^46"),
])
def test_w4_descriptor_refusals(kw, status, word):
    d = w4(**kw)
    assert B.lib().iqnn_w4_packed_size(ctypes.byref(d)) == 0 and word in B.lib().iqnn_last_error().decode()
    refused(status, word, B.iqnn_w4_fwd, d, 1, P, d.k, P, None, P, d.n)


def test_w4_call_refusals():
    d = w4()
    refused(INVALID, "null", B.iqnn_w4_fwd, d, 1, 0, 64, P, None, P, 8)
    refused(INVALID, "null", B.iqnn_w4_fwd, d, 1, P, 64, 0, None, P, 8)
    refused(INVALID, "null", B.iqnn_w4_fwd, d, 1, P, 64, P, None, 0, 8)
    refused(INVALID, "sizes", B.iqnn_w4_fwd, d, -1, P, 64, P, None, P, 8)
    refused(INVALID, "stride", B.iqnn_w4_fwd, d, 2, P, 63, P, None, P, 8)
    refused(INVALID, "stride", B.iqnn_w4_fwd, d, 2, P, 64, P, None, P, 7)
    refused(ALIGNMENT, "misaligned", B.iqnn_w4_fwd, d, 2, P + 1, 64, P, None, P, 8)
    refused(ALIGNMENT, "misaligned", B.iqnn_w4_fwd, d, 2, P, 64, P + 128, None, P, 8)
    refused(ALIGNMENT, "misaligned", B.iqnn_w4_fwd, d, 2, P, 64, P, P + 1, P, 8)
    L = B.lib()
    size = B.iqnn_w4_packed_size(d)
    ref = ctypes.byref(d)
    assert L.iqnn_w4_prepack(ref, P, P, None, P, size - 1, None) == INVALID
    assert L.iqnn_w4_prepack(ref, 0, P, None, P, size, None) == INVALID
    assert L.iqnn_w4_prepack(ref, P, 0, None, P, size, None) == INVALID
    assert L.iqnn_w4_prepack(ref, P, P, None, P + 16, size, None) == ALIGNMENT
    assert L.iqnn_w4_prepack(ctypes.byref(w4(w_type=B.UINT4)), P, P, None, P, 1 << 20, None) == INVALID


@pytest.mark.parametrize("n,k,group,codes,scales", [
    (1, 2, 32, 1024, 16 * 4 * 4), (16, 128, 128, 1024, 16 * 4), (17, 130, 64, 4 * 1024, 2 * 2 * 16 * 2 * 4),
    (4096, 4096, 0, 4096 * 4096 // 2, 4096 * 4),
])
def test_w4_packed_size(n, k, group, codes, scales):
    """Codes of whole 16 x 128 blocks, float scales and (UINT4) byte zero points, in 256s."""
    up = lambda v: -(-v // 256) * 256
    assert B.iqnn_w4_packed_size(w4(n, k, group=group)) == codes + up(scales)
    assert B.iqnn_w4_packed_size(w4(n, k, B.UINT4, group=group)) == codes + up(scales) + up(scales // 4)


def wg(m=8, n=8, k=64, dy=B.BFLOAT16, dw=B.BFLOAT16, group=32):
    d = B.CkptWgradDesc()
    d.m, d.n, d.k, d.dy_type, d.dw_type, d.group = m, n, k, dy, dw, group
    return d


@pytest.mark.parametrize("kw,status,word", [
    (dict(m=-1), INVALID, "sizes"), (dict(n=0), INVALID, "sizes"), (dict(k=0), INVALID, "sizes"),
    (dict(dy=4), INVALID, "floating-point"), (dict(dw=B.FLOAT16), INVALID, "dw_type"),
    (dict(dy=B.FLOAT32, dw=B.BFLOAT16), INVALID, "dw_type"), (dict(group=8), INVALID, "group"),
    (dict(n=2 ** 31), UNSUPPORTED, "2^30"), (dict(m=2 ** 40, n=2 ** 30), UNSUPPORTED, "2^46"),
])
def test_ckpt_wgrad_descriptor_refusals(kw, status, word):
    d = wg(**kw)
    with pytest.raises(B.IqnnError) as e:
        B.iqnn_ckpt_wgrad_workspace(d)
    assert word in str(e.value)
    refused(status, word, B.iqnn_ckpt_wgrad, d, P, d.n, P, P, P, P, P, 1 << 40)


def test_ckpt_wgrad_call_refusals():
    d = wg()
    assert B.iqnn_ckpt_wgrad_workspace(d) == 0
    for bad in range(4):
        a = [P, P, P, P]
        a[bad] = 0
        refused(INVALID, "null", B.iqnn_ckpt_wgrad, d, a[0], 8, a[1], a[2], a[3], None, None, 0)
    refused(INVALID, "stride", B.iqnn_ckpt_wgrad, d, P, 7, P, P, P, None, None, 0)
    refused(ALIGNMENT, "misaligned", B.iqnn_ckpt_wgrad, d, P, 8, P, P, P + 1, None, None, 0)
    refused(ALIGNMENT, "misaligned", B.iqnn_ckpt_wgrad, d, P, 8, P, P, P, P + 1, None, 0)
    # many rows over few output tiles are shared among blocks through the workspace
    d = wg(m=8192, n=128, k=128)
    size = B.iqnn_ckpt_wgrad_workspace(d)
    assert size >= 2 * (128 * 128 + 128) * 4
    refused(INVALID, "null", B.iqnn_ckpt_wgrad, d, P, 128, P, P, P, None, None, size)
    refused(INVALID, "workspace", B.iqnn_ckpt_wgrad, d, P, 128, P, P, P, None, P, size - 1)
    refused(ALIGNMENT, "misaligned", B.iqnn_ckpt_wgrad, d, P, 128, P, P, P, None, P + 8, size)


def test_ckpt_wgrad_tiles_of_a_launch():
    """2^24 blocks of 256 threads are 2^32 threads, one more than a launch holds."""
    assert B.iqnn_ckpt_wgrad_workspace(wg(m=1, n=2 ** 20 - 128, k=2 ** 18)) == 0
    d = wg(m=1, n=2 ** 20, k=2 ** 18)
    with pytest.raises(B.IqnnError, match="blocks"):
        B.iqnn_ckpt_wgrad_workspace(d)
    refused(UNSUPPORTED, "blocks", B.iqnn_ckpt_wgrad, d, P, d.n, P, P, P, P, P, 1 << 40)


def test_ckpt_act_without_codes():
    """Neither codes nor scales may come alone; the other checks stay."""
    for bad, word in ((dict(x=0), "null"), (dict(y=0), "null"), (dict(s=P), "null"), (dict(q=P), "null"), (dict(y=P + 2), "misaligned"),
                      (dict(group=96), "group"), (dict(kind=4), "activation")):
        status = ALIGNMENT if word == "misaligned" else INVALID
        refused(status, word, B.iqnn_ckpt_act_fwd, *act(**{"q": 0, "s": 0, **bad}))
    B.iqnn_ckpt_act_fwd(*act(rows=0, x=0, y=0, q=0, s=0), stream=0)


@pytest.mark.parametrize("x_type", [B.FLOAT32, B.FLOAT16, B.BFLOAT16])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("k", [264, 266])
def test_gpu_tests_reach_every_w4_kernel(x_type, group, k):
    """The sizes of the GPU test fall on every kernel that any size falls on."""
    from test_gpu_group_kernels import W4_CHOICES
    reached = {B.iqnn_w4_kernel(w4(n, k, x_type=x_type, group=group), m) for m, n in W4_CHOICES}
    rows = list(range(1, 20)) + [2 ** i + d for i in range(5, 15) for d in (-1, 0, 1)]
    cols = [1, 64, 300, 777] + [1024 * i + d for i in range(1, 40) for d in (-5, 0)]
    every = {B.iqnn_w4_kernel(w4(n, k, x_type=x_type, group=group), m) for m in rows for n in cols}
    assert reached == every
    few = (3 if k % 8 else 5) + (x_type == B.FLOAT32 and k % 8 == 0)
    tiles = 2 if k % 8 or x_type == B.FLOAT32 else 5 if group in (0, 128) else 4
    assert len(every) == few + tiles


def test_w4_kernel_refusals():
    for d, m in ((w4(group=48), 1), (w4(), 0)):
        with pytest.raises(B.IqnnError):
            B.iqnn_w4_kernel(d, m)
    # rows that are not aligned in whole vectors fall where an odd K falls
    assert B.iqnn_w4_kernel(w4(4096, 4096), 2048, aligned=False) == B.iqnn_w4_kernel(w4(4096, 4094), 2048)
