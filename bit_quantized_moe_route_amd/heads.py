"""What reads a projection of libmoeq (include/moeq.h: moe_head_norm_rope,
moe_token_logprobs): norms and rotation of query and key heads, and the log
probabilities behind a projection to logits.  Argument marshalling only.

A call runs on its tensors' device and that device's current stream, and
refuses tensors of several devices.
"""

import ctypes
import struct

from . import _I32, _I64, _P, _torch, lib
from .block import _call, _cuda, _dt, _flat, _rows, _ws

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


def _whole(t, name, shape, dev):
    """Checks whole numbers of `shape` on dev; returns their address and bits."""
    torch = _torch()
    if tuple(t.shape) != shape or t.dtype not in (torch.int32, torch.int64) or t.device != dev \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 or int64 {list(shape)} on {dev}, got "
                         f"{list(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr(), 32 if t.dtype == torch.int32 else 64


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


def _head_set(x, name, w, out, T, D, dev, dtype, w_dtype):
    """The fields of a head set, and its output tensor."""
    torch = _torch()
    if x.dim() != 3 or x.shape[0] != T or x.shape[2] != D or x.device != dev or x.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} [{T}, heads, {D}] on {dev}, got "
                         f"{list(x.shape)} {x.dtype} on {x.device}")
    if out is None:
        out = torch.empty(x.shape, dtype=dtype, device=dev)
    elif out.shape != x.shape or out.device != dev or out.dtype != dtype:
        raise ValueError(f"{name}_out must be {dtype} {list(x.shape)} on {dev}, got "
                         f"{list(out.shape)} {out.dtype} on {out.device}")
    s, o = x.stride(), out.stride()
    if D > 1 and (s[2] != 1 or o[2] != 1):
        raise ValueError(f"the elements of a head of {name} must lie side by side")
    wp = 0
    if w is not None:
        if w.shape != (D,) or w.device != dev or w.dtype != w_dtype or not w.is_contiguous():
            raise ValueError(f"{name}_w must be {w_dtype} [{D}], contiguous, on {dev}, got "
                             f"{list(w.shape)} {w.dtype} on {w.device}")
        wp = w.data_ptr()
    return (x.data_ptr(), s[0], s[1], out.data_ptr(), o[0], o[1], wp, x.shape[1], 0), out


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
    torch = _torch()
    dev = _cuda(q, "head_norm_rope")
    if q.dim() != 3:
        raise ValueError(f"q must be [T, heads, D], got {list(q.shape)}")
    T, _, D = q.shape
    w_dtype = q_w.dtype if q_w is not None else k_w.dtype if k_w is not None else q.dtype
    if k is None and (k_w is not None or k_out is not None):
        raise ValueError("k_w and k_out need k")
    fq, q_out = _head_set(q, "q", q_w, q_out, T, D, dev, q.dtype, w_dtype)
    fk = (0, 0, 0, 0, 0, 0, 0, 0, 0)
    if k is not None:
        fk, k_out = _head_set(k, "k", k_w, k_out, T, D, dev, q.dtype, w_dtype)
    pp = tp = bits = rows = R = 0
    if pos is not None:
        if table is None:
            raise ValueError("pos needs a table (rope_table)")
        if table.dim() != 2 or table.dtype != torch.float32 or table.device != dev \
                or not table.is_contiguous():
            raise ValueError(f"table must be contiguous fp32 [positions, R] on {dev}")
        pp, bits = _whole(pos, "pos", (T,), dev)
        rows, R = table.shape
        tp = table.data_ptr()
    elif table is not None:
        raise ValueError("table needs pos")
    if T:
        _call("moe_head_norm_rope", dev,
              _HEADS.pack(*fq, *fk, pp, tp, rows, D, R, 1 if interleaved else 0, bits, _dt(q.dtype),
                          _dt(w_dtype), eps, w_offset), T)
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
    torch = _torch()
    dev = _cuda(logits, "token_logprobs")
    if logits.dim() != 2:
        raise ValueError(f"logits must be [T, V], got {list(logits.shape)}")
    T, V = logits.shape
    ld = _rows(logits, "logits", T, V, dev)
    if not 0 <= top <= MAX_TOP:
        raise ValueError(f"top must be in [0, {MAX_TOP}], got {top}")
    ip = bits = m = lp = sp = tp = tl = 0
    if ids is not None:
        if ids.dim() not in (1, 2):
            raise ValueError(f"ids must be [T] or [T, m], got {list(ids.shape)}")
        m = 1 if ids.dim() == 1 else ids.shape[1]
        ip, bits = _whole(ids, "ids", (T,) if ids.dim() == 1 else (T, m), dev)
        if logprob is None:
            logprob = torch.empty(ids.shape, dtype=torch.float32, device=dev)
        lp = _flat(logprob, "logprob", T * m, dev, torch.float32)
    elif logprob is not None:
        raise ValueError("logprob needs ids")
    if scale is not None:
        sp = _flat(scale, "scale", T, dev, torch.float32)
    if entropy is None:
        entropy = torch.empty(T, dtype=torch.float32, device=dev)
    ep = _flat(entropy, "entropy", T, dev, torch.float32)
    if top:
        if top_ids is None:
            top_ids = torch.empty((T, top), dtype=torch.int32, device=dev)
        if top_logprob is None:
            top_logprob = torch.empty((T, top), dtype=torch.float32, device=dev)
        tp = _flat(top_ids, "top_ids", T * top, dev, torch.int32)
        tl = _flat(top_logprob, "top_logprob", T * top, dev, torch.float32)
    elif top_ids is not None or top_logprob is not None:
        raise ValueError("top_ids and top_logprob go with top > 0")
    ws = token_logprobs_workspace(logits, top) if ws is None else _ws(ws, dev)
    if T:
        if m == 0:
            ip = lp = 0
        _call("moe_token_logprobs", dev,
              _LOGPROBS.pack(logits.data_ptr(), ld, sp, ip, lp, ep, tp, tl, V, m, top,
                             _dt(logits.dtype), bits, 0), T, ws.data_ptr(), ws.numel())
    return (logprob, entropy, top_ids, top_logprob) if top else (logprob, entropy)
