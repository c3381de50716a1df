"""Layer objects over the C ABI: torch supplies device memory and streams, every
step runs in libiqnn's kernels.

  QConv / QGemm   prepack a layer once (iqnn_*_prepack), then run it (iqnn_*_fwd)
  quantize / dequantize / maxpool2d   allocate the output and call the kernel
  quantize_groups / dequantize_groups   codes with a scale per group, found on the device
  W4Linear        a linear layer with 4-bit weights of that form
  ckpt_act, ckpt_act_bwd, ckpt_wgrad   activations kept in 8 bits and their use in the
                  backward pass (checkpoint.py has the autograd functions)
"""
import contextlib
import ctypes

import numpy as np
import torch
from torch.autograd import forward_ad

from . import binding as B


def code_bytes(shape, qtype):
    """Byte shape of a code tensor: 4-bit types pack pairs along the last axis."""
    shape = tuple(int(s) for s in shape)
    if qtype in (B.INT4, B.UINT4):
        assert shape[-1] % 2 == 0, "4-bit tensors need an even innermost size"
        return shape[:-1] + (shape[-1] // 2,)
    if qtype == B.INT32:
        return shape[:-1] + (shape[-1] * 4,)
    return shape


def empty_codes(shape, qtype, device="cuda"):
    return torch.empty(code_bytes(shape, qtype), dtype=torch.uint8, device=device)


def _scalar_or_vec(v, dtype, device):
    return torch.as_tensor(np.atleast_1d(np.asarray(v)), dtype=dtype, device=device).contiguous()


def quantize(x, scale, zp, qtype, axis=-1, out=None, stream=None):
    """Codes of float tensor x (device); scale/zp scalars or per-channel along `axis`."""
    axis = axis % x.dim()
    outer = int(np.prod(x.shape[:axis], dtype=np.int64))
    ch = int(x.shape[axis])
    inner = int(np.prod(x.shape[axis + 1:], dtype=np.int64))
    s = scale if torch.is_tensor(scale) else _scalar_or_vec(scale, torch.float32, x.device)
    z = zp if torch.is_tensor(zp) else _scalar_or_vec(zp, torch.int32, x.device)
    per_channel = s.numel() > 1 or z.numel() > 1
    if per_channel and s.numel() == 1:
        s = s.expand(ch).contiguous()
    if per_channel and z.numel() == 1:
        z = z.expand(ch).contiguous()
    if out is None:
        out = empty_codes(x.shape, qtype, x.device)
    B.iqnn_quantize(x, out, outer, ch, inner, s, z, per_channel, qtype, stream)
    return out


def quantize_pad(x, scale, zp, qtype, pad, c_pad, out=None, stream=None):
    """Codes of NHWC float x with a border of `pad` pixels and channels padded to c_pad,
    all padding holding the zero-point code."""
    n, h, w, c = (int(v) for v in x.shape)
    s = scale if torch.is_tensor(scale) else _scalar_or_vec(scale, torch.float32, x.device)
    z = zp if torch.is_tensor(zp) else _scalar_or_vec(zp, torch.int32, x.device)
    per_channel = s.numel() > 1 or z.numel() > 1
    if out is None:
        out = torch.empty((n, h + 2 * pad, w + 2 * pad, c_pad), dtype=torch.uint8, device=x.device)
    B.iqnn_quantize_pad(x, out, n, h, w, c, pad, c_pad, s, z, per_channel, qtype, stream)
    return out


def dequantize(q, shape, scale, zp, qtype, axis=-1, out=None, stream=None):
    shape = tuple(shape)
    axis = axis % len(shape)
    outer = int(np.prod(shape[:axis], dtype=np.int64))
    ch = int(shape[axis])
    inner = int(np.prod(shape[axis + 1:], dtype=np.int64))
    s = scale if torch.is_tensor(scale) else _scalar_or_vec(scale, torch.float32, q.device)
    z = zp if torch.is_tensor(zp) else _scalar_or_vec(zp, torch.int32, q.device)
    per_channel = s.numel() > 1 or z.numel() > 1
    if per_channel and s.numel() == 1:
        s = s.expand(ch).contiguous()
    if per_channel and z.numel() == 1:
        z = z.expand(ch).contiguous()
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=q.device)
    B.iqnn_dequantize(q, out, outer, ch, inner, s, z, per_channel, qtype, stream)
    return out


def maxpool2d(x, n, h, w, c, k, stride, pad, dtype, out=None, stream=None):
    oh = (h + 2 * pad - k) // stride + 1
    ow = (w + 2 * pad - k) // stride + 1
    if out is None:
        out = torch.empty((n, oh, ow, c), dtype=torch.uint8, device=x.device)
    B.iqnn_maxpool2d(x, out, n, h, w, c, k, stride, pad, dtype, stream)
    return out


class QConv:
    """One prepacked quantized conv layer (NHWC, OHWI weights)."""

    def __init__(self, n, h, w, c_in, c_out, k, stride, pad, x_type, w_type, y_type, epi, z_in, z_out,
                 w_bytes, bias, s_in, s_w, s_out, res_type=B.UINT8, z_res=0, s_res=1.0, kw=None,
                 device="cuda", stream=None, z_w=0):
        kw = k if kw is None else kw
        d = B.ConvDesc()
        d.n, d.h, d.w, d.c_in, d.c_out = n, h, w, c_in, c_out
        d.kh, d.kw, d.stride_h, d.stride_w, d.pad_h, d.pad_w = k, kw, stride, stride, pad, pad
        d.x_type, d.w_type, d.y_type, d.res_type, d.epilogue = x_type, w_type, y_type, res_type, epi
        d.z_in, d.z_out, d.z_res, d.z_w = z_in, z_out, z_res, z_w
        self.desc = d
        self.out_shape = (n,) + d.out_hw() + (c_out,)
        s_w = np.atleast_1d(np.asarray(s_w, np.float32))
        self.packed = torch.empty(B.iqnn_qconv_packed_size(d), dtype=torch.uint8, device=device)
        B.iqnn_qconv_prepack(d, w_bytes, bias, s_in, s_w, s_w.size > 1, s_out, s_res, self.packed, stream)
        self.y_type = y_type

    def __call__(self, x, res=None, out=None, stream=None, cfg=None):
        """cfg: kernel configuration (tile, xcd_groups) of this call; None: automatic."""
        if out is None:
            out = empty_codes(self.out_shape, self.y_type, x.device)
        if cfg is None:
            B.iqnn_qconv_fwd(self.desc, x, self.packed, res, out, stream)
        else:
            B.iqnn_qconv_fwd_cfg(self.desc, x, self.packed, res, out, cfg, stream)
        return out

    def pool_shape(self, k=3, stride=2, pad=1):
        n, oh, ow, c = self.out_shape
        return (n, (oh + 2 * pad - k) // stride + 1, (ow + 2 * pad - k) // stride + 1, c)

    def conv_maxpool(self, x, k=3, stride=2, pad=1, out=None, stream=None):
        """maxpool(conv(x)) in one fused launch (iqnn_qconv_maxpool_fwd)."""
        if out is None:
            out = empty_codes(self.pool_shape(k, stride, pad), self.y_type, x.device)
        B.iqnn_qconv_maxpool_fwd(self.desc, x, self.packed, out, k, stride, pad, stream)
        return out


def conv_pair(conv_a, conv_b, x, res=None, out_a=None, out_b=None, stream=None):
    """y_a = conv_a(x, res) and y_b = conv_b(y_a) in one call (iqnn_qconv_pair_fwd):
    conv_b's input is conv_a's output.  Returns (y_a, y_b)."""
    if out_a is None:
        out_a = empty_codes(conv_a.out_shape, conv_a.y_type, x.device)
    if out_b is None:
        out_b = empty_codes(conv_b.out_shape, conv_b.y_type, x.device)
    B.iqnn_qconv_pair_fwd(conv_a.desc, conv_b.desc, x, conv_a.packed, res, conv_b.packed, out_a, out_b, stream)
    return out_a, out_b


class QGemm:
    """One prepacked quantized GEMM: C[M][N] = epilogue(A[M][K] B[N][K]^T)."""

    def __init__(self, m, n, k, a_type, b_type, c_type, epi, z_a, z_out, b_bytes, bias, s_a, s_b, s_out,
                 res_type=B.UINT8, z_res=0, s_res=1.0, device="cuda", stream=None, z_b=0):
        d = B.GemmDesc()
        d.m, d.n, d.k = m, n, k
        d.a_type, d.b_type, d.c_type, d.res_type, d.epilogue = a_type, b_type, c_type, res_type, epi
        d.z_a, d.z_out, d.z_res, d.z_b = z_a, z_out, z_res, z_b
        self.desc = d
        self.out_shape = (m, n)
        s_b = np.atleast_1d(np.asarray(s_b, np.float32))
        self.packed = torch.empty(B.iqnn_qgemm_packed_size(d), dtype=torch.uint8, device=device)
        B.iqnn_qgemm_prepack(d, b_bytes, bias, s_a, s_b, s_b.size > 1, s_out, s_res, self.packed, stream)
        self.c_type = c_type

    def __call__(self, a, res=None, out=None, stream=None, cfg=None):
        if out is None:
            out = empty_codes(self.out_shape, self.c_type, a.device)
        if cfg is None:
            B.iqnn_qgemm_fwd(self.desc, a, self.packed, res, out, stream)
        else:
            B.iqnn_qgemm_fwd_cfg(self.desc, a, self.packed, res, out, cfg, stream)
        return out


_CODES = {B.INT8: False, B.UINT8: False, B.INT4: True, B.UINT4: True}   # code types: 4 bits?
_FTYPES = {torch.float32: B.FLOAT32, torch.float16: B.FLOAT16, torch.bfloat16: B.BFLOAT16}


def _away(device, stream):
    """Whether a call names a stream, or a device that is not the current one."""
    return stream is not None or device.index != torch._C._cuda_getDevice()


@contextlib.contextmanager
def _on(device, stream, *used):
    """Launch and allocate on `stream` (None: the device's current one) of `device`.  A named
    stream is noted on the tensors `used` there, so that one freed after the call is not handed
    out again while the stream still reads or writes it."""
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device=device)
            with torch.cuda.stream(stream):
                yield
            for t in used:
                if isinstance(t, torch.Tensor) and t.is_cuda:
                    t.record_stream(stream)


def _current(device):
    """Raw handle of the device's current stream."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _need(ok, message):
    if not ok:
        raise ValueError(message)


def _ftype(dtype):
    ft = _FTYPES.get(dtype)
    if ft is None:
        raise ValueError("float32, float16 or bfloat16 expected, not %s" % dtype)
    return ft


# The calls below are short: a microsecond of Python is a tenth of many of them.  They pass
# addresses straight to the library and format messages only when they raise.

def _gpu(x, name):
    """(rows, cols, iqnn_ftype) of a float tensor on a GPU, rows of its last axis."""
    if not (isinstance(x, torch.Tensor) and x.is_cuda):
        raise ValueError("%s must be a GPU tensor" % name)
    shape = x.shape
    if not shape or shape[-1] == 0:
        raise ValueError("%s needs a non-empty last axis" % name)
    return x.numel() // shape[-1], shape[-1], _ftype(x.dtype)


def _rows(x, rows, cols):
    """(x, row stride): x itself where its rows are one stride apart and their elements
    adjacent, else a contiguous copy."""
    if x.is_contiguous():
        return x, cols
    if x.dim() == 2 and x.stride(1) == 1 and (x.stride(0) >= cols or rows <= 1):
        return x, max(x.stride(0), cols)
    return x.contiguous(), cols


def _aux(t, rows, cols, dtype, device, name):
    """A contiguous companion tensor on `device` holding rows x cols, checked."""
    if not (isinstance(t, torch.Tensor) and t.device == device and t.dtype is dtype and t.dim() and t.shape[-1] == cols
            and t.numel() == rows * cols):
        raise ValueError("%s must hold %d rows of %d %s on %s" % (name, rows, cols, dtype, device))
    return t if t.is_contiguous() else t.contiguous()


def _span(t):
    """Addresses from a tensor's first element to behind its last."""
    last = sum((n - 1) * st for n, st in zip(t.shape, t.stride())) if t.numel() else -1
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _out(out, shape, dtype, device, like, *others):
    """`out` checked, or a new tensor; `like` and `others` are what the call reads."""
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    _need(out.device == device and out.dtype == dtype and tuple(out.shape) == tuple(shape) and out.is_contiguous(),
          "out must be a contiguous tensor of the result's shape and type on the same device")
    lo, hi = _span(out)
    for t in (like,) + others:
        if t is not None:
            a, b = _span(t)
            _need(hi <= a or b <= lo, "out must not overlap an input")
    return out


def _int8(q):
    """INT8 codes as such: quantize_groups returns their bytes."""
    return q.view(torch.int8) if isinstance(q, torch.Tensor) and q.dtype is torch.uint8 else q


def _ptr(t):
    return None if t is None else t.data_ptr()


def _no_gradient(x, what):
    """Refuses an x that asks for a derivative, in either mode, of a call that has none."""
    if (x.requires_grad and torch.is_grad_enabled()) or (
            forward_ad._current_level >= 0 and forward_ad.unpack_dual(x).tangent is not None):
        raise ValueError("%s has no gradient" % what)


def _done(status):
    if status:
        B._check(status)


def groups_of(cols, group):
    """Groups per row of `cols` elements (group 0: one)."""
    if group not in (0, 32, 64, 128):
        raise ValueError("group must be 0, 32, 64 or 128, not %r" % (group,))
    return -(-cols // group) if group else 1


def quantize_groups(x, qtype, group=128, stream=None):
    """(codes, scale, zp) of float x with parameters per group along the last axis, found on
    the device; codes as code_bytes lays them out, scale and zp x.shape[:-1] + (groups,), zp
    None for the symmetric (signed) types."""
    rows, cols, ft = _gpu(x, "x")
    dev = x.device
    if _away(dev, stream):
        with _on(dev, stream, x):
            return quantize_groups(x, qtype, group)
    four = _CODES.get(qtype)
    if four is None or (four and cols % 2):
        raise ValueError("qtype must be a code type, a 4-bit one with an even innermost size")
    lead, g = x.shape[:-1], groups_of(cols, group)
    xr, ld = _rows(x, rows, cols)
    q = x.new_empty(lead + (cols // 2 if four else cols,), dtype=torch.uint8)
    s = x.new_empty(lead + (g,), dtype=torch.float32)
    z = x.new_empty(lead + (g,), dtype=torch.int32) if qtype in (B.UINT8, B.UINT4) else None
    _done(B.lib().iqnn_quantize_groups(xr.data_ptr(), ft, rows, cols, ld, group, q.data_ptr(), qtype, s.data_ptr(), _ptr(z),
                                       _current(dev)))
    return q, s, z


def dequantize_groups(q, scale, zp, qtype, group=128, dtype=torch.float32, out=None, stream=None):
    """Floats of codes made by quantize_groups."""
    if not (isinstance(q, torch.Tensor) and q.is_cuda and q.dtype in (torch.uint8, torch.int8) and q.dim() and q.shape[-1]):
        raise ValueError("codes must be bytes on the GPU with a non-empty last axis")
    dev = q.device
    if _away(dev, stream):
        with _on(dev, stream, q, scale, zp, out):
            return dequantize_groups(q, scale, zp, qtype, group, dtype, out)
    four, shape = _CODES.get(qtype), q.shape
    if four is None:
        raise ValueError("qtype must be a code type")
    lead, width = shape[:-1], shape[-1]
    cols, rows = 2 * width if four else width, q.numel() // width
    ft, g = _ftype(dtype), groups_of(cols, group)
    s = _aux(scale, rows, g, torch.float32, dev, "scale")
    z = _aux(zp, rows, g, torch.int32, dev, "zp") if qtype in (B.UINT8, B.UINT4) else None
    x = _out(out, lead + (cols,), dtype, dev, q, s, z)
    qc = q if q.is_contiguous() else q.contiguous()
    _done(B.lib().iqnn_dequantize_groups(qc.data_ptr(), qtype, rows, cols, group, s.data_ptr(), _ptr(z), x.data_ptr(), ft, cols,
                                         _current(dev)))
    return x


class W4Linear:
    """y = x W^T + bias with 4-bit weights: q [n][k / 2] and scale [n][groups] as
    quantize_groups makes them (INT4), with zp [n][groups] UINT4.  The weights are laid out
    once; the constructor returns when that is done, so that the layer may be called on any
    stream and q, scale and zp be freed.  dtype: of x, bias and y.  For inference: no gradient
    flows through it."""

    def __init__(self, q, scale, zp=None, group=128, bias=None, dtype=torch.bfloat16, stream=None):
        _need(torch.is_tensor(q) and q.is_cuda and q.dtype == torch.uint8 and q.dim() == 2 and q.numel() > 0,
              "q must be a [n][k / 2] byte tensor on the GPU")
        d = B.W4Desc()
        d.n, d.k = q.shape[0], 2 * q.shape[1]
        d.w_type, d.x_type, d.group = B.INT4 if zp is None else B.UINT4, _ftype(dtype), group
        g, dev = groups_of(d.k, group), q.device
        self.desc, self.dtype, self.device = d, dtype, dev
        self.in_features, self.out_features = int(d.k), int(d.n)
        with _on(dev, stream):
            scale = _aux(scale, d.n, g, torch.float32, dev, "scale")
            zp = None if zp is None else _aux(zp, d.n, g, torch.int32, dev, "zp")
            self.bias = None if bias is None else _aux(bias.detach(), 1, d.n, dtype, dev, "bias")
            self.packed = torch.empty(B.iqnn_w4_packed_size(d), dtype=torch.uint8, device=dev)
            B.iqnn_w4_prepack(d, q.contiguous(), scale, zp, self.packed, _current(dev))
            torch.cuda.current_stream(dev).synchronize()
        # what every call passes, marshalled once
        self._fwd, self._desc = B.lib().iqnn_w4_fwd, ctypes.byref(d)
        self._packed, self._bias = self.packed.data_ptr(), None if self.bias is None else self.bias.data_ptr()

    def __call__(self, x, out=None, stream=None):
        # one token is short of host time: the ordinary call takes as few steps as it can
        if (out is None and stream is None and type(x) is torch.Tensor and x.dtype is self.dtype
                and x.device == self.device and x.dim() and x.shape[-1] == self.in_features and x.is_contiguous()
                and not x.requires_grad and forward_ad._current_level < 0
                and torch._C._cuda_getDevice() == self.device.index):
            n, k = self.out_features, self.in_features
            y = x.new_empty(x.shape[:-1] + (n,))
            status = self._fwd(self._desc, x.numel() // k, x.data_ptr(), k, self._packed, self._bias, y.data_ptr(), n,
                               _current(self.device))
            if status:
                B._check(status)
            return y
        rows, cols, _ = _gpu(x, "x")
        dev, n = x.device, self.out_features
        if cols != self.in_features or x.dtype != self.dtype or dev != self.device:
            raise ValueError("x must be [..., %d] of %s on %s" % (self.in_features, self.dtype, self.device))
        if _away(dev, stream):
            with _on(dev, stream, x, out, self.packed, self.bias):
                return self(x, out)
        _no_gradient(x, "W4Linear")
        xr, ld = _rows(x, rows, cols)
        y = _out(out, x.shape[:-1] + (n,), self.dtype, dev, x, self.packed, self.bias)
        B.iqnn_w4_fwd(self.desc, rows, xr, ld, self.packed, self.bias, y, n, _current(dev))
        return y


def ckpt_act(x, act, group=128, gated=False, out=None, stream=None, save=True):
    """(y, codes, scale): y = act(x), or act(a) * b with x = [a | b] when gated, and the
    8-bit codes and scales of x that ckpt_act_bwd reads, all from one pass over x.  No
    gradient flows through it: checkpoint.act is the function that has one.  save=False: y
    alone, codes and scale None."""
    rows, width, ft = _gpu(x, "x")
    _no_gradient(x, "ckpt_act (checkpoint.act has)")
    dev = x.device
    if _away(dev, stream):
        with _on(dev, stream, x, out):
            return ckpt_act(x, act, group, gated, out, save=save)
    _need(not gated or width % 2 == 0, "a gated activation needs an even last axis")
    cols, lead = (width // 2 if gated else width), x.shape[:-1]
    g = groups_of(cols, group) * (2 if gated else 1)
    xr, ld = _rows(x, rows, width)
    y = _out(out, lead + (cols,), x.dtype, dev, x)
    q = x.new_empty(lead + (width,), dtype=torch.int8) if save else None
    s = x.new_empty(lead + (g,), dtype=torch.float32) if save else None
    _done(B.lib().iqnn_ckpt_act_fwd(xr.data_ptr(), ft, rows, cols, ld, act, gated, group, y.data_ptr(), cols, _ptr(q),
                                    _ptr(s), _current(dev)))
    return y, q, s


def ckpt_act_bwd(dy, q, scale, act, group=128, gated=False, out=None, stream=None):
    """Gradient of ckpt_act's x from dy and the codes, in dy's type."""
    rows, cols, ft = _gpu(dy, "dy")
    dev = dy.device
    if _away(dev, stream):
        with _on(dev, stream, dy, q, scale, out):
            return ckpt_act_bwd(dy, q, scale, act, group, gated, out)
    halves = 2 if gated else 1
    width = cols * halves
    q = _aux(_int8(q), rows, width, torch.int8, dev, "codes")
    s = _aux(scale, rows, groups_of(cols, group) * halves, torch.float32, dev, "scale")
    dyr, ld = _rows(dy, rows, cols)
    dx = _out(out, dy.shape[:-1] + (width,), dy.dtype, dev, dy, q, s)
    _done(B.lib().iqnn_ckpt_act_bwd(dyr.data_ptr(), ft, rows, cols, ld, act, gated, group, q.data_ptr(), s.data_ptr(),
                                    dx.data_ptr(), width, _current(dev)))
    return dx


def ckpt_wgrad(dy, q, scale, group=128, out_dtype=None, bias=False, stream=None):
    """(dW, db): gradients of a linear layer's weight [n][k] and bias [n] (None unless
    `bias`) from dy [..., n] and the 8-bit codes [..., k] of its input.  out_dtype: dy's
    type (the default) or float32."""
    m, n, ft = _gpu(dy, "dy")
    dev = dy.device
    if _away(dev, stream):
        with _on(dev, stream, dy, q, scale):
            return ckpt_wgrad(dy, q, scale, group, out_dtype, bias)
    out_dtype = dy.dtype if out_dtype is None else out_dtype
    _need(torch.is_tensor(q) and q.dim() >= 1 and q.shape[-1] > 0, "codes must be a GPU tensor")
    k = q.shape[-1]
    d = B.CkptWgradDesc(m, n, k, ft, _ftype(out_dtype), group)
    q = _aux(_int8(q), m, k, torch.int8, dev, "codes")
    s = _aux(scale, m, groups_of(k, group), torch.float32, dev, "scale")
    dyr, ld = _rows(dy, m, n)
    dw = dy.new_empty((n, k), dtype=out_dtype)
    db = dy.new_empty(n, dtype=out_dtype) if bias else None
    size = B.iqnn_ckpt_wgrad_workspace(d)
    ws = dy.new_empty(size, dtype=torch.uint8) if size else None
    _done(B.lib().iqnn_ckpt_wgrad(ctypes.byref(d), dyr.data_ptr(), ld, q.data_ptr(), s.data_ptr(), dw.data_ptr(), _ptr(db),
                                  _ptr(ws), size, _current(dev)))
    return dw, db
