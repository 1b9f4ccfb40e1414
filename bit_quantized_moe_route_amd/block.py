"""The block norms and the 8-bit integer products of libmoeq (include/moeq.h:
moe_block_norm, moe_quantize_i8, moe_linear_i8, moe_expert_ffn_i8,
moe_shared_ffn_i8).  Argument marshalling only.

Tensors are 2-D rows of fp32, bf16 or fp16 whose elements lie side by side;
rows may lie further apart (a slice of a wider tensor).  A call runs on its
tensors' device and that device's current stream, and refuses tensors of
several devices.
"""

import ctypes
import struct

from . import MOE_OK, _I32, _I64, _P, _check, _dptr, _torch, lib, route_permute

DT_F32, DT_BF16, DT_F16, DT_I8 = 1, 2, 3, 4
_F32 = ctypes.c_float
_dts = {}


def _dt(dtype):
    if not _dts:
        t = _torch()
        _dts.update({t.float32: DT_F32, t.bfloat16: DT_BF16, t.float16: DT_F16})
    if dtype not in _dts:
        raise ValueError(f"fp32, bf16 or fp16 required, got {dtype}")
    return _dts[dtype]


class BlockC(ctypes.Structure):
    _fields_ = [
        ("y", _P), ("ld_y", _I64),
        ("inv_perm", _P), ("topk_w", _P),
        ("y_shared", _P), ("ld_y_shared", _I64),
        ("shared_gate", _P),
        ("post_w", _P),
        ("gate", _P), ("gate_ld_t", _I64), ("gate_ld_h", _I64),
        ("r", _P), ("ld_r", _I64),
        ("r_out", _P), ("ld_r_out", _I64),
        ("pre_w", _P),
        ("n_out", _P), ("ld_n", _I64),
        ("q_out", _P), ("ld_q", _I64),
        ("q_scale", _P),
        ("k", _I32),
        ("y_dtype", _I32), ("y_shared_dtype", _I32), ("r_dtype", _I32), ("w_dtype", _I32),
        ("gate_dtype", _I32), ("n_dtype", _I32),
        ("y_scale", _F32), ("r_scale", _F32), ("eps", _F32), ("w_offset", _F32),
        ("reserved", _I32),
    ]


# The same struct packed in one call: filling it field by field costs more than
# the kernel of a small batch takes.
_BLOCK = struct.Struct("@PqPPPqPPPqqPqPqPPqPqP7i4fi")
assert _BLOCK.size == ctypes.sizeof(BlockC)


class I8LinearC(ctypes.Structure):
    _fields_ = [("N", _I32), ("K", _I32), ("w", _P), ("w_scale", _P), ("bias", _P)]


class I8LayerC(ctypes.Structure):
    _fields_ = [("E", _I32), ("H", _I32), ("I", _I32), ("reserved", _I32),
                ("w13", _P), ("w13_stride", _I64), ("w2", _P), ("w2_stride", _I64),
                ("w13_scale", _P), ("w2_scale", _P)]


_C = ctypes.c_int
_SZ = ctypes.c_size_t
PROTOS = {
    "moe_block_norm": (_C, [_P, _I64, _I32, _P]),
    "moe_quantize_i8": (_C, [_P, _I32, _I64, _I64, _I32, _P, _I64, _P, _P]),
    "moe_i8_matrix_bytes": (_SZ, [_I32, _I32]),
    "moe_i8_record_bytes": (_SZ, [_C, _I32, _I32]),
    "moe_pack_i8": (_C, [_P, _I64, _I32, _I32, _P, _P]),
    "moe_pack_i8_expert": (_C, [_P, _P, _P, _I32, _I32, _P, _P, _P]),
    "moe_linear_i8_workspace_bytes": (_SZ, [ctypes.POINTER(I8LinearC), _I64]),
    "moe_linear_i8": (_C, [ctypes.POINTER(I8LinearC), _P, _I32, _I64, _P, _I64, _P, _I32, _I64,
                           _P, _SZ, _P]),
    "moe_expert_ffn_i8_workspace_bytes": (_SZ, [ctypes.POINTER(I8LayerC), _I64, _I32]),
    "moe_expert_ffn_i8": (_C, [ctypes.POINTER(I8LayerC), _P, _I32, _I64, _P, _P, _P, _I64, _I32,
                               _P, _I32, _P, _SZ, _P]),
    "moe_shared_ffn_i8": (_C, [ctypes.POINTER(I8LayerC), _P, _I32, _I64, _P, _I64, _P, _I32, _P,
                               _SZ, _P]),
}


# --------------------------------------------------------------------------
# checks
# --------------------------------------------------------------------------

def _rows(t, name, T, H, dev, dtype=None):
    """Checks rows [T, H] on dev; returns their stride in elements."""
    if t.shape != (T, H):
        raise ValueError(f"{name} must be [{T}, {H}], got {list(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, not on {dev}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.is_contiguous():
        return H
    s0, s1 = t.stride()
    if s1 != 1 and H > 1:
        raise ValueError(f"the elements of a row of {name} must lie side by side")
    return s0 if T > 1 else max(s0, H)


def _flat(t, name, n, dev, dtype):
    """Checks a contiguous tensor of n elements of dtype on dev."""
    if t.numel() != n or t.dtype != dtype or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous {dtype} on {dev}, got "
                         f"{list(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


def _cuda(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name}: device tensors required")
    return t.device


_fns = {}


def _bind(L):
    """The library's functions and torch's stream lookup (the raw one where
    this torch has it: a Stream object costs as much as a launch).  The table is
    replaced whole: another thread's call keeps the one it looked up."""
    global _fns
    torch = _torch()
    f = {n: getattr(L, n) for n in PROTOS}
    f["lib"] = L
    f["stream"] = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda i: torch.cuda.current_stream(i).cuda_stream)
    f["device"] = torch.cuda.current_device
    _fns = f
    return f


def _call(name, dev, *args):
    """One library call on dev and its current stream."""
    L = lib()
    f = _fns
    if f.get("lib") is not L:
        f = _bind(L)
    i = dev.index
    if i == f["device"]():
        st = f[name](*args, f["stream"](i))
    else:
        with _torch().cuda.device(dev):
            st = f[name](*args, f["stream"](i))
    if st != MOE_OK:
        _check(st, name)


def codes_width(K):
    """Elements between the code rows of [T, K]: K rounded up to 64."""
    return (K + 63) // 64 * 64


def _codes_like(T, K, q, scale, dev):
    """Checks or allocates the code rows (int8 [T, codes_width(K)]) and scales."""
    torch = _torch()
    if q is None:
        q = torch.empty((T, codes_width(K)), dtype=torch.int8, device=dev)
    elif q.dim() != 2 or q.shape[1] < codes_width(K):
        raise ValueError(f"codes must be [{T}, at least {codes_width(K)}], got {list(q.shape)}")
    if scale is None:
        scale = torch.empty(T, dtype=torch.float32, device=dev)
    ld = _rows(q, "codes", T, q.shape[1], dev, torch.int8)
    _flat(scale, "scale", T, dev, torch.float32)
    return q, ld, scale


# --------------------------------------------------------------------------
# norms before and after a block
# --------------------------------------------------------------------------

def _vector(t, name, H, dev, dtype=None):
    if t.shape != (H,) or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be [{H}], contiguous, on {dev}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError("both norms' weights must be of one type")
    return t.data_ptr()


def _block(dev, T, H, r, y, w, k, inv_perm, topk_w, y_shared, shared_gate, post_w, gate, y_scale,
           r_scale, eps, w_offset, r_out, out, out_dtype, codes, q, scale):
    torch = _torch()
    y_p = y_ld = y_t = inv_p = tw_p = ys_p = ys_ld = ys_t = sg_p = 0
    w_p = pw_p = w_t = g_p = g_ld = g_lh = g_t = 0
    r_p = r_ld = r_t = ro_p = ro_ld = n_p = n_ld = n_t = q_p = q_ld = qs_p = 0
    if y is not None:
        y_ld = _rows(y, "y_perm" if k else "y", T * (k or 1), H, dev)
        y_p, y_t = y.data_ptr(), _dt(y.dtype)
        if k:
            inv_p = _flat(inv_perm, "inv_perm", T * k, dev, torch.int32)
            tw_p = _flat(topk_w, "topk_w", T * k, dev, torch.float32)
            if y_shared is not None:
                ys_ld = _rows(y_shared, "y_shared", T, H, dev)
                ys_p, ys_t = y_shared.data_ptr(), _dt(y_shared.dtype)
            if shared_gate is not None:
                sg_p = _flat(shared_gate, "shared_gate", T, dev, torch.float32)
    if w is not None:
        w_p, w_t = _vector(w, "w", H, dev), _dt(w.dtype)
    if post_w is not None:
        pw_p = _vector(post_w, "post_w", H, dev, None if w is None else w.dtype)
        w_t = _dt(post_w.dtype)
    if gate is not None:
        if gate.dim() != 2 or gate.device != dev or gate.shape[0] not in (1, T) \
                or gate.shape[1] not in (1, H) or (gate.shape[1] > 1 and gate.stride(1) != 1):
            raise ValueError(f"gate must be [{T}, 1], [1, {H}] or [{T}, {H}] on {dev}, the "
                             "elements of a row side by side")
        g_p, g_t = gate.data_ptr(), _dt(gate.dtype)
        g_ld = gate.stride(0) if gate.shape[0] > 1 else 0
        g_lh = 1 if gate.shape[1] > 1 else 0
    if r is not None:
        r_ld = _rows(r, "r", T, H, dev)
        r_p, r_t = r.data_ptr(), _dt(r.dtype)
    if r_out is not None:
        ro_ld = _rows(r_out, "r_out", T, H, dev, r.dtype if r is not None else None)
        ro_p, r_t = r_out.data_ptr(), _dt(r_out.dtype)
    if out is None and w is not None:
        out = torch.empty((T, H), dtype=out_dtype or (r_out if r is None else r).dtype, device=dev)
    if out is False:
        out = None
    if out is not None:
        n_ld = _rows(out, "out", T, H, dev, out_dtype)
        n_p, n_t = out.data_ptr(), _dt(out.dtype)
    if codes:
        q, q_ld, scale = _codes_like(T, H, q, scale, dev)
        q_p, qs_p = q.data_ptr(), scale.data_ptr()
    elif q is not None or scale is not None:
        raise ValueError("q and scale go with codes=True")
    if T:
        _call("moe_block_norm", dev,
              _BLOCK.pack(y_p, y_ld, inv_p, tw_p, ys_p, ys_ld, sg_p, pw_p, g_p, g_ld, g_lh, r_p,
                          r_ld, ro_p, ro_ld, w_p, n_p, n_ld, q_p, q_ld, qs_p, k, y_t, ys_t, r_t,
                          w_t, g_t, n_t, y_scale, r_scale, eps, w_offset, 0), T, H)
    return out, q, scale


def block_norm(r, w, *, eps=1e-5, w_offset=0.0, out=None, out_dtype=None, codes=False, q=None,
               scale=None):
    """The norm before a block: n = r / sqrt(mean(r^2) + eps) * (w_offset + w)
    for rows r [T, H], as `out` (of out_dtype, r's by default).  With codes,
    also the 8-bit code of n: returns (n, q, scale); out=False then leaves n
    itself unwritten (returned as None)."""
    dev = _cuda(r, "block_norm")
    T, H = r.shape
    n, q, scale = _block(dev, T, H, r, None, w, 0, None, None, None, None, None, None, 1.0, 1.0,
                         eps, w_offset, None, out, out_dtype, codes, q, scale)
    return (n, q, scale) if codes else n


def block_residual(r, y, w=None, *, post_w=None, gate=None, y_scale=1.0, r_scale=1.0, eps=1e-5,
                   w_offset=0.0, r_out=None, out=None, out_dtype=None, codes=False, q=None,
                   scale=None):
    """What follows a block whose output is y [T, H], up to the next block:
        r' = r_scale * r + y_scale * gate * (N(y; post_w) or y)
        n  = N(r'; w)
    gate: [T, 1], [1, H] or [T, H].  r_out may be r (the residual stream
    updated in place).  Returns (r', n), n None without w; with codes
    (r', n, q, scale), as block_norm."""
    torch = _torch()
    dev = _cuda(r, "block_residual")
    T, H = r.shape
    if r_out is None:
        r_out = torch.empty((T, H), dtype=r.dtype, device=dev)
    n, q, scale = _block(dev, T, H, r, y, w, 0, None, None, None, None, post_w, gate, y_scale,
                         r_scale, eps, w_offset, r_out, out, out_dtype, codes, q, scale)
    return (r_out, n, q, scale) if codes else (r_out, n)


def combine_residual(r, y_perm, inv_perm, topk_w, w=None, *, y_shared=None, shared_gate=None,
                     post_w=None, gate=None, y_scale=1.0, r_scale=1.0, eps=1e-5, w_offset=0.0,
                     r_out=None, out=None, out_dtype=None, codes=False, q=None, scale=None):
    """block_residual after a routed layer: y = sum_j topk_w[t, j] *
    y_perm[inv_perm[t*k + j]] (ascending j) + shared_gate[t] * y_shared[t],
    without writing y.  y_perm [T*k, H] and y_shared [T, H] of any float type;
    shared_gate fp32 [T] (1 if not given).  r None: no residual stream, r' is
    the gated sum itself (fp32, or of r_out's type)."""
    torch = _torch()
    if topk_w.dim() != 2 or topk_w.shape[1] < 1:
        raise ValueError(f"topk_w must be [T, k] with k at least 1, got {list(topk_w.shape)}")
    dev = _cuda(y_perm, "combine_residual")
    T, k = topk_w.shape
    H = y_perm.shape[1]
    if r_out is None:
        r_out = torch.empty((T, H), dtype=torch.float32 if r is None else r.dtype, device=dev)
    if shared_gate is not None and y_shared is None:
        raise ValueError("shared_gate needs y_shared")
    n, q, scale = _block(dev, T, H, r, y_perm, w, k, inv_perm, topk_w, y_shared, shared_gate,
                         post_w, gate, y_scale, r_scale, eps, w_offset, r_out, out, out_dtype,
                         codes, q, scale)
    return (r_out, n, q, scale) if codes else (r_out, n)


# --------------------------------------------------------------------------
# 8-bit integer products
# --------------------------------------------------------------------------

def quantize_i8(x, q=None, scale=None):
    """Rows x [T, K] -> (q int8 [T, codes_width(K)], scale fp32 [T]): x[t, k] is
    about q[t, k] * scale[t]; the codes past K are 0."""
    dev = _cuda(x, "quantize_i8")
    T, K = x.shape
    ld = _rows(x, "x", T, K, dev)
    q, ldq, scale = _codes_like(T, K, q, scale, dev)
    if T:
        _call("moe_quantize_i8", dev, x.data_ptr(), _dt(x.dtype), ld, T, K, q.data_ptr(), ldq,
              scale.data_ptr())
    return q, scale


def _x(x, scale, K, dev, name="x"):
    """(pointer, type, row stride, scale pointer) of a product's left operand:
    float rows [T, K], or codes with their scales."""
    torch = _torch()
    T = x.shape[0]
    if x.dtype == torch.int8:
        if scale is None:
            raise ValueError("codes need their scales")
        if x.dim() != 2 or x.shape[1] < codes_width(K):
            raise ValueError(f"codes must be [T, at least {codes_width(K)}], got {list(x.shape)}")
        return (x.data_ptr(), DT_I8, _rows(x, name, T, x.shape[1], dev),
                _flat(scale, "scale", T, dev, torch.float32))
    if scale is not None:
        raise ValueError("scales go with int8 codes only")
    return x.data_ptr(), _dt(x.dtype), _rows(x, name, T, K, dev), None


def _ws(ws, dev):
    if ws.device != dev or ws.dtype != _torch().uint8 or not ws.is_contiguous():
        raise ValueError(f"the workspace must be contiguous uint8 on {dev}")
    return ws


class I8Linear:
    """A matrix [N, K] in 8-bit codes with a scale per output channel, packed
    on its GPU.  codes int8 [N, K], scale fp32 [N], bias fp32 [N] or None."""

    def __init__(self, codes, scale, bias=None):
        torch = _torch()
        dev = _cuda(codes, "I8Linear")
        N, K = codes.shape
        ld = _rows(codes, "codes", N, K, dev, torch.int8)
        _flat(scale, "scale", N, dev, torch.float32)
        if bias is not None:
            _flat(bias, "bias", N, dev, torch.float32)
        n = lib().moe_i8_matrix_bytes(N, K)
        if not n:
            raise ValueError(f"unsupported matrix [{N}, {K}]")
        self.N, self.K, self.device = N, K, dev
        self.scale, self.bias = scale, bias
        self.packed = torch.empty(n, dtype=torch.uint8, device=dev)
        _call("moe_pack_i8", dev, codes.data_ptr(), ld, N, K, self.packed.data_ptr())
        self._c = I8LinearC(N=N, K=K, w=self.packed.data_ptr(), w_scale=scale.data_ptr(),
                            bias=bias.data_ptr() if bias is not None else None)

    @classmethod
    def quantized(cls, w, bias=None):
        """From float weights [N, K]: codes and scales of each row."""
        q, s = quantize_i8(w)
        return cls(q[:, :w.shape[1]], s, bias)

    def c(self):
        return self._c


def linear_i8_workspace(linear, T):
    """Workspace of linear_i8 for T rows of a float type."""
    n = lib().moe_linear_i8_workspace_bytes(ctypes.byref(linear.c()), T)
    return _torch().empty(max(n, 256), dtype=_torch().uint8, device=linear.device)


def linear_i8(linear, x, scale=None, out=None, out_dtype=None, ws=None):
    """x [T, K] times the matrix, in 8 bits: [T, N] of out_dtype (x's type, bf16
    for codes, by default).  x: float rows, coded in the call, or int8 codes
    from quantize_i8 or a block norm with their scale."""
    torch = _torch()
    dev = _cuda(x, "linear_i8")
    if dev != linear.device:
        raise ValueError(f"x is on {dev}, the matrix on {linear.device}")
    T = x.shape[0]
    px, dt, ldx, ps = _x(x, scale, linear.K, dev)
    if out is None:
        out = torch.empty((T, linear.N), device=dev, dtype=out_dtype or (
            torch.bfloat16 if dt == DT_I8 else x.dtype))
    ldo = _rows(out, "out", T, linear.N, dev, out_dtype)
    if dt != DT_I8:
        ws = linear_i8_workspace(linear, T) if ws is None else _ws(ws, dev)
    if T:
        _call("moe_linear_i8", dev, ctypes.byref(linear.c()), px, dt, ldx, ps, T, out.data_ptr(),
              _dt(out.dtype), ldo, _dptr(ws), ws.numel() if ws is not None else 0)
    return out


class I8Layer:
    """E experts in 8-bit codes, packed on their GPU.
    w13 int8 [E, 2I, H] (gate rows, then up rows) with scales fp32 [E, 2I];
    w2 int8 [E, H, I] with scales fp32 [E, H]."""

    def __init__(self, w13, s13, w2, s2):
        torch = _torch()
        dev = _cuda(w13, "I8Layer")
        if w13.dim() != 3 or w13.shape[1] % 2:
            raise ValueError("w13 must be [E, 2I, H]")
        E, I, H = w13.shape[0], w13.shape[1] // 2, w13.shape[2]
        for t, name, shape, dtype in ((w13, "w13", (E, 2 * I, H), torch.int8),
                                      (w2, "w2", (E, H, I), torch.int8),
                                      (s13, "s13", (E, 2 * I), torch.float32),
                                      (s2, "s2", (E, H), torch.float32)):
            if tuple(t.shape) != shape or t.dtype != dtype or t.device != dev \
                    or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous {dtype} {list(shape)} on {dev}")
        n13, n2 = (lib().moe_i8_record_bytes(which, H, I) for which in (0, 1))
        if not n13 or not n2:
            raise ValueError(f"unsupported sizes H {H}, I {I}")
        self.E, self.H, self.I, self.device = E, H, I, dev
        self.s13, self.s2 = s13, s2
        self.w13 = torch.empty(E * n13, dtype=torch.uint8, device=dev)
        self.w2 = torch.empty(E * n2, dtype=torch.uint8, device=dev)
        for e in range(E):
            _call("moe_pack_i8_expert", dev, w13.data_ptr() + e * 2 * I * H,
                  w13.data_ptr() + (2 * e + 1) * I * H, w2.data_ptr() + e * H * I, H, I,
                  self.w13.data_ptr() + e * n13, self.w2.data_ptr() + e * n2)
        self._c = I8LayerC(E=E, H=H, I=I, w13=self.w13.data_ptr(), w13_stride=n13,
                           w2=self.w2.data_ptr(), w2_stride=n2, w13_scale=s13.data_ptr(),
                           w2_scale=s2.data_ptr())

    @classmethod
    def quantized(cls, gate, up, down):
        """From float weights gate, up [E, I, H] and down [E, H, I]: codes and
        scales of each row."""
        torch = _torch()
        E, I, H = gate.shape
        w13 = torch.cat([gate, up], 1).reshape(E * 2 * I, H)
        q13, s13 = quantize_i8(w13)
        q2, s2 = quantize_i8(down.reshape(E * H, I))
        return cls(q13[:, :H].contiguous().view(E, 2 * I, H), s13.view(E, 2 * I),
                   q2[:, :I].contiguous().view(E, H, I), s2.view(E, H))

    def c(self):
        return self._c


def ffn_i8_workspace(layer, T, k=1):
    """Workspace of expert_ffn_i8 (k = 1: of shared_ffn_i8)."""
    n = lib().moe_expert_ffn_i8_workspace_bytes(ctypes.byref(layer.c()), T, k)
    return _torch().empty(max(n, 256), dtype=_torch().uint8, device=layer.device)


def _ffn(name, layer, x, scale, maps, T, k, y, y_dtype, ws):
    torch = _torch()
    dev = _cuda(x, name)
    if dev != layer.device:
        raise ValueError(f"x is on {dev}, the layer on {layer.device}")
    px, dt, ldx, ps = _x(x, scale, layer.H, dev)
    if y is None:
        y = torch.empty((T * k, layer.H), device=dev, dtype=y_dtype or (
            torch.bfloat16 if dt == DT_I8 else x.dtype))
    if _rows(y, "y", T * k, layer.H, dev, y_dtype) != layer.H and T * k > 1:
        raise ValueError("y must be contiguous")
    ws = ffn_i8_workspace(layer, T, k) if ws is None else _ws(ws, dev)
    if T:
        _call(name, dev, ctypes.byref(layer.c()), px, dt, ldx, ps, *maps, y.data_ptr(),
              _dt(y.dtype), ws.data_ptr(), ws.numel())
    return y


def expert_ffn_i8(layer, x, perm_src, offsets, k, scale=None, y_perm=None, y_dtype=None, ws=None):
    """expert_ffn_q for an I8Layer: y_perm [T*k, H] of y_dtype (x's type, bf16 for
    codes, by default).  x: float rows, or int8 codes with their scale."""
    torch = _torch()
    T = x.shape[0]
    maps = (_flat(perm_src, "perm_src", T * k, x.device, torch.int32),
            _flat(offsets, "offsets", layer.E + 1, x.device, torch.int32), T, k)
    return _ffn("moe_expert_ffn_i8", layer, x, scale, maps, T, k, y_perm, y_dtype, ws)


def shared_ffn_i8(shared, x, scale=None, y=None, y_dtype=None, ws=None):
    """shared_ffn for a one-expert I8Layer: [T, H]."""
    T = x.shape[0]
    return _ffn("moe_shared_ffn_i8", shared, x, scale, (T,), T, 1, y, y_dtype, ws)


def forward_i8(layer, x, logits, k, shared=None, scale=None):
    """forward() for an I8Layer (and a one-expert I8Layer `shared`): the rows
    coded once (or given as codes with their scale), route -> permute -> expert
    FFN -> combine.  Returns a dict of every intermediate; out is fp32 [T, H]."""
    torch = _torch()
    q = x
    if scale is None:
        q, scale = quantize_i8(x)
    ids, w, counts, offsets, perm_src, inv_perm = route_permute(logits, k, layer.E)
    y_perm = expert_ffn_i8(layer, q, perm_src, offsets, k, scale, y_dtype=torch.float32)
    r = dict(q=q, scale=scale, topk_ids=ids, topk_w=w, counts=counts, offsets=offsets,
             perm_src=perm_src, inv_perm=inv_perm, y_perm=y_perm)
    if shared is None:
        r["out"] = combine_residual(None, y_perm, inv_perm, w)[0]
    else:
        r["y_shared"] = shared_ffn_i8(shared, q, scale, y_dtype=torch.float32)
        r["out"] = combine_residual(None, y_perm, inv_perm, w, y_shared=r["y_shared"])[0]
    return r
