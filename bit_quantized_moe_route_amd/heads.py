"""What reads a projection of libmoeq (include/moeq.h: moe_head_norm_rope,
moe_token_logprobs): norms and rotation of query and key heads, and the log
probabilities behind a projection to logits.  Argument marshalling only.

A call runs on its tensors' device and that device's current stream, and
refuses tensors of several devices.
"""

import ctypes
import struct

from . import _I32, _I64, _P, _torch, lib
from .block import DT_F32, _call_on, _dt, _dts

MAX_TOP = 32          # MOE_MAX_TOP
_F32 = ctypes.c_float


class HeadSetC(ctypes.Structure):
    _fields_ = [("x", _P), ("ld_t", _I64), ("ld_h", _I64),
                ("out", _P), ("ld_out_t", _I64), ("ld_out_h", _I64),
                ("w", _P), ("heads", _I32), ("reserved", _I32)]


class HeadsC(ctypes.Structure):
    _fields_ = [("q", HeadSetC), ("k", HeadSetC), ("pos", _P), ("table", _P), ("table_rows", _I64),
                ("D", _I32), ("R", _I32), ("interleaved", _I32), ("pos_bits", _I32),
                ("dtype", _I32), ("w_dtype", _I32), ("eps", _F32), ("w_offset", _F32)]


class LogprobsC(ctypes.Structure):
    _fields_ = [("logits", _P), ("ld", _I64), ("scale", _P), ("ids", _P), ("logprob", _P),
                ("entropy", _P), ("top_ids", _P), ("top_logprob", _P),
                ("V", _I32), ("m", _I32), ("top", _I32), ("dtype", _I32), ("id_bits", _I32),
                ("reserved", _I32)]


# The same structs packed in one call each: filling them field by field costs more
# than the kernel of a small batch takes.
_HEADS = struct.Struct("@PqqPqqPiiPqqPqqPiiPPq6iff")
_LOGPROBS = struct.Struct("@Pq6P6i")
assert _HEADS.size == ctypes.sizeof(HeadsC) and _LOGPROBS.size == ctypes.sizeof(LogprobsC)

PROTOS = {
    "moe_head_norm_rope": (ctypes.c_int, [_P, _I64, _P]),
    "moe_token_logprobs_workspace_bytes": (ctypes.c_size_t, [_I64, _I32, _I32]),
    "moe_token_logprobs": (ctypes.c_int, [_P, _I64, _P, ctypes.c_size_t, _P]),
}


# The checks go by a tensor's device index: comparing device objects costs twice that, and a
# call of a few rows is bound by its host side.

_bits = {}


def _gpu(t, name):
    i = t.get_device()
    if i < 0:
        raise ValueError(f"{name}: device tensors required")
    return i


def _type(dtype):
    return _dts.get(dtype) or _dt(dtype)


def _flat_on(t, name, n, i, dtype):
    """Checks a contiguous tensor of n elements of dtype on GPU i."""
    if t.numel() != n or t.dtype is not dtype or t.get_device() != i or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous {dtype} on GPU {i}, got "
                         f"{list(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


def _whole(t, name, shape, i):
    """Checks whole numbers of `shape` on GPU i; returns their address and bits."""
    if not _bits:
        torch = _torch()
        _bits.update({torch.int32: 32, torch.int64: 64})
    bits = _bits.get(t.dtype)
    if bits is None or t.shape != shape or t.get_device() != i or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 or int64 {list(shape)} on GPU {i}, got "
                         f"{list(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr(), bits


# --------------------------------------------------------------------------
# query and key heads
# --------------------------------------------------------------------------

def rope_table(positions, rotated, base=10000.0, *, freq=None, scale=1.0, device="cuda"):
    """The table of head_norm_rope for positions 0 .. positions - 1: fp32
    [positions, rotated], the cosines of the rotated / 2 angles of a position,
    then their sines, each times `scale`.  Angle i is position * base^(-2i /
    rotated), or position * freq[i]; taken in 64 bits, since at a far position
    the fp32 product would be off by whole thousandths of a turn."""
    torch = _torch()
    if positions < 1 or rotated < 2 or rotated % 2:
        raise ValueError("positions must be at least 1 and rotated even")
    if freq is None:
        freq = base ** (-torch.arange(0, rotated, 2, dtype=torch.float64, device=device) / rotated)
    freq = torch.as_tensor(freq, dtype=torch.float64, device=device)
    if tuple(freq.shape) != (rotated // 2,):
        raise ValueError(f"freq must be [{rotated // 2}], got {list(freq.shape)}")
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([angle.cos() * scale, angle.sin() * scale], 1).float()


def _head_set(x, name, w, out, T, D, i, dtype, w_dtype):
    """The fields of a head set, and its output tensor."""
    shape = x.shape
    if len(shape) != 3 or shape[0] != T or shape[2] != D or x.dtype is not dtype \
            or x.get_device() != i:
        raise ValueError(f"{name} must be {dtype} [{T}, heads, {D}] on GPU {i}, got "
                         f"{list(shape)} {x.dtype} on {x.device}")
    if out is None:
        out = _torch().empty(shape, dtype=dtype, device=x.device)
    elif out.shape != shape or out.dtype is not dtype or out.get_device() != i:
        raise ValueError(f"{name}_out must be {dtype} {list(shape)} on GPU {i}, got "
                         f"{list(out.shape)} {out.dtype} on {out.device}")
    t, h, e = x.stride()
    ot, oh, oe = out.stride()
    if (e != 1 or oe != 1) and D > 1:
        raise ValueError(f"the elements of a head of {name} must lie side by side")
    wp = 0
    if w is not None:
        if w.shape != (D,) or w.dtype is not w_dtype or w.get_device() != i \
                or not w.is_contiguous():
            raise ValueError(f"{name}_w must be {w_dtype} [{D}], contiguous, on GPU {i}, got "
                             f"{list(w.shape)} {w.dtype} on {w.device}")
        wp = w.data_ptr()
    return (x.data_ptr(), t, h, out.data_ptr(), ot, oh, wp, shape[1], 0), out


_NO_HEADS = (0, 0, 0, 0, 0, 0, 0, 0, 0)


def head_norm_rope(q, k=None, q_w=None, k_w=None, *, pos=None, table=None, interleaved=False,
                   eps=1e-5, w_offset=0.0, q_out=None, k_out=None):
    """The norm of each query and key head and its rotation by the token's
    position, in one pass: q [T, Hq, D] and k [T, Hk, D], parts of a wider tensor
    as they are.  n = v / sqrt(mean(v^2) + eps) * (w_offset + w) over a head (no
    norm without its weights), then the pairs (a, b) of n's first R elements,
    halves i and R/2 + i or, interleaved, 2i and 2i + 1, turned to (a c - b s,
    b c + a s) with the cosine and sine of table [P, R] (rope_table) at pos [T]
    (none without pos).  q_out and k_out may be q and k.  Returns (q_out, k_out),
    k_out None without k."""
    i = _gpu(q, "head_norm_rope")
    shape = q.shape
    if len(shape) != 3:
        raise ValueError(f"q must be [T, heads, D], got {list(shape)}")
    T, _, D = shape
    dtype = q.dtype
    w_dtype = q_w.dtype if q_w is not None else k_w.dtype if k_w is not None else dtype
    fq, q_out = _head_set(q, "q", q_w, q_out, T, D, i, dtype, w_dtype)
    if k is not None:
        fk, k_out = _head_set(k, "k", k_w, k_out, T, D, i, dtype, w_dtype)
    elif k_w is not None or k_out is not None:
        raise ValueError("k_w and k_out need k")
    else:
        fk = _NO_HEADS
    pp = tp = bits = rows = R = 0
    if pos is not None:
        if table is None:
            raise ValueError("pos needs a table (rope_table)")
        size = table.shape
        if len(size) != 2 or _type(table.dtype) != DT_F32 or table.get_device() != i \
                or not table.is_contiguous():
            raise ValueError(f"table must be contiguous fp32 [positions, R] on GPU {i}")
        pp, bits = _whole(pos, "pos", (T,), i)
        rows, R = size
        tp = table.data_ptr()
    elif table is not None:
        raise ValueError("table needs pos")
    if T:
        _call_on("moe_head_norm_rope", i,
                 _HEADS.pack(*fq, *fk, pp, tp, rows, D, R, 1 if interleaved else 0, bits,
                             _type(dtype), _type(w_dtype), eps, w_offset), T)
    return q_out, k_out


# --------------------------------------------------------------------------
# log probabilities
# --------------------------------------------------------------------------

def token_logprobs_workspace(logits, top=0):
    """Workspace of token_logprobs for logits like these."""
    T, V = logits.shape
    n = lib().moe_token_logprobs_workspace_bytes(T, V, top)
    return _torch().empty(max(n, 256), dtype=_torch().uint8, device=logits.device)


def token_logprobs(logits, ids=None, *, top=0, scale=None, logprob=None, entropy=None, top_ids=None,
                   top_logprob=None, ws=None):
    """Of p = softmax(scale[t] * logits[t]), logits [T, V] of a float type and
    scale fp32 [T] (1 / temperature; 1 if not given): (logprob, entropy), and with
    top > 0 also (.., top_ids, top_logprob).
        logprob      fp32, log p of the tokens ids [T] or [T, m] (int32 or int64),
                     of their shape; None without ids
        entropy      fp32 [T]
        top_ids      int32 [T, top]: the most likely tokens, equal ones by the lower id
        top_logprob  fp32 [T, top]
    A logit of -inf masks its token; a list that runs out of tokens goes on with -1
    and -inf.  A row that is masked as a whole: entropy 0, -inf everywhere.  A row
    with a NaN or +inf, or a scale that is not positive and finite: NaN and -1."""
    i = _gpu(logits, "token_logprobs")
    size = logits.shape
    if len(size) != 2:
        raise ValueError(f"logits must be [T, V], got {list(size)}")
    T, V = size
    ld, one = logits.stride()
    if one != 1 and V > 1:
        raise ValueError("the elements of a row of logits must lie side by side")
    if T == 1 and ld < V:
        ld = V
    if not 0 <= top <= MAX_TOP:
        raise ValueError(f"top must be in [0, {MAX_TOP}], got {top}")
    torch = _torch()
    f32 = torch.float32
    ip = bits = m = lp = sp = tp = tl = 0
    if ids is not None:
        at = ids.shape
        if len(at) not in (1, 2):
            raise ValueError(f"ids must be [T] or [T, m], got {list(at)}")
        m = 1 if len(at) == 1 else at[1]
        ip, bits = _whole(ids, "ids", (T,) if len(at) == 1 else (T, m), i)
        if logprob is None:
            logprob = torch.empty(at, dtype=f32, device=logits.device)
        lp = _flat_on(logprob, "logprob", T * m, i, f32)
    elif logprob is not None:
        raise ValueError("logprob needs ids")
    if scale is not None:
        sp = _flat_on(scale, "scale", T, i, f32)
    if entropy is None:
        entropy = torch.empty(T, dtype=f32, device=logits.device)
    ep = _flat_on(entropy, "entropy", T, i, f32)
    if top:
        if top_ids is None:
            top_ids = torch.empty((T, top), dtype=torch.int32, device=logits.device)
        if top_logprob is None:
            top_logprob = torch.empty((T, top), dtype=f32, device=logits.device)
        tp = _flat_on(top_ids, "top_ids", T * top, i, torch.int32)
        tl = _flat_on(top_logprob, "top_logprob", T * top, i, f32)
    elif top_ids is not None or top_logprob is not None:
        raise ValueError("top_ids and top_logprob go with top > 0")
    if ws is None:
        ws = token_logprobs_workspace(logits, top)
    n = ws.numel()
    wp = _flat_on(ws, "the workspace", n, i, torch.uint8)
    if T:
        if m == 0:
            ip = lp = 0
        _call_on("moe_token_logprobs", i,
                 _LOGPROBS.pack(logits.data_ptr(), ld, sp, ip, lp, ep, tp, tl, V, m, top,
                                _type(logits.dtype), bits, 0), T, wp, n)
    return (logprob, entropy, top_ids, top_logprob) if top else (logprob, entropy)
