"""Low-rank adapters of many requests beside a projection that they share, in
libmoeq (include/moeq.h: moe_pack_adapter, moe_adapter_plan, moe_add_adapters).
Argument marshalling only.

    set = Adapters(n, rank, K, N)            # slots on one GPU, for one projection
    set.load(slot, a, b, scale)              # A [r, K], B [N, r]
    plan = adapter_plan(slots, n)            # a batch's tokens, once for all projections
    y = add_adapters(set, x, plan, y)        # y[t] + scale * B (A x[t])

A call runs on its tensors' device and that device's current stream, and
refuses tensors of several devices.
"""

import ctypes

from . import MOE_EINVAL, MOE_EWORKSPACE, MoeError, _I32, _I64, _P, _torch, lib
from .block import DT_I8, _call, _call_on, _cuda, _dt, _flat, _rows, _x, codes_width
from .heads import _flat_on, _gpu, _type

MAX_ADAPTERS, MAX_RANK = 1023, 256      # MOE_MAX_ADAPTERS, MOE_MAX_RANK


class AdaptersC(ctypes.Structure):
    _fields_ = [("n", _I32), ("rank", _I32), ("K", _I32), ("N", _I32), ("w_dtype", _I32),
                ("reserved", _I32), ("a", _P), ("b", _P), ("ranks", _P), ("scales", _P)]


_C, _SZ, _S = ctypes.c_int, ctypes.c_size_t, ctypes.POINTER(AdaptersC)
PROTOS = {
    "moe_adapter_bytes": (_SZ, [_C, _I32, _I32, _I32]),
    "moe_pack_adapter": (_C, [_S, _I32, _P, _I64, _P, _I64, _I32, ctypes.c_float, _P]),
    "moe_adapter_plan_bytes": (_SZ, [_I64, _I32]),
    "moe_adapter_plan": (_C, [_P, _I64, _I32, _P, _SZ, _P]),
    "moe_add_adapters_workspace_bytes": (_SZ, [_S, _I64]),
    "moe_add_adapters": (_C, [_S, _P, _I32, _I64, _P, _P, _I64, _P, _I64, _P, _I64, _I32, _P, _SZ,
                              _P]),
}


class Adapters:
    """n slots of low-rank adapters of one projection [N, K], each of its own rank
    up to `rank` (at most 256), in bf16 or fp16 on one GPU; empty at first."""

    def __init__(self, n, rank, K, N, dtype=None, device="cuda"):
        torch = _torch()
        dtype = torch.bfloat16 if dtype is None else dtype
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"adapters are bf16 or fp16, got {dtype}")
        if not 1 <= n <= MAX_ADAPTERS:
            raise ValueError(f"n must be in [1, {MAX_ADAPTERS}], got {n}")
        na, nb = (lib().moe_adapter_bytes(which, rank, K, N) for which in (0, 1))
        if not na or not nb:
            raise ValueError(f"unsupported sizes: rank {rank}, K {K}, N {N}")
        self.n, self.rank, self.K, self.N, self.dtype = n, rank, K, N, dtype
        self.a = torch.empty(n * na, dtype=torch.uint8, device=device)
        self.b = torch.empty(n * nb, dtype=torch.uint8, device=device)
        self.ranks = torch.zeros(n, dtype=torch.int32, device=device)
        self.scales = torch.zeros(n, dtype=torch.float32, device=device)
        self.device, self.index, self.w_dtype = self.a.device, self.a.get_device(), _dt(dtype)
        self._c = AdaptersC(n=n, rank=rank, K=K, N=N, w_dtype=_dt(dtype), a=self.a.data_ptr(),
                            b=self.b.data_ptr(), ranks=self.ranks.data_ptr(),
                            scales=self.scales.data_ptr())
        self.at = ctypes.byref(self._c)
        self.bytes = torch.uint8
        self.space = None, 0        # a number of tokens and the workspace they need

    def load(self, slot, a, b, scale=1.0):
        """Puts A [r, K] and B [N, r] (of the set's type) with their scale into a
        slot, on the current stream."""
        dev = _cuda(a, "Adapters.load")
        if dev != self.device:
            raise ValueError(f"a is on {dev}, the adapters on {self.device}")
        if not 0 <= slot < self.n:
            raise ValueError(f"slot must be in [0, {self.n}), got {slot}")
        r = a.shape[0] if a.dim() == 2 else 0
        if not 1 <= r <= self.rank:
            raise ValueError(f"a must be [1 to {self.rank}, {self.K}], got {list(a.shape)}")
        lda = _rows(a, "a", r, self.K, dev, self.dtype)
        ldb = _rows(b, "b", self.N, r, dev, self.dtype)
        _call("moe_pack_adapter", dev, ctypes.byref(self._c), slot, a.data_ptr(), lda, b.data_ptr(),
              ldb, r, scale)

    def unload(self, slot):
        """Empties a slot: its tokens get nothing added."""
        _call("moe_pack_adapter", self.device, ctypes.byref(self._c), slot, None, 0, None, 0, 0, 0.0)

    def c(self):
        return self._c


class AdapterPlan:
    """A batch's tokens by adapter (adapter_plan), for T tokens and n slots."""

    def __init__(self, T, n, data):
        self.T, self.n, self.data, self.device = T, n, data, data.device
        self.at, self.index = data.data_ptr(), data.get_device()


def adapter_plan(ids, n, plan=None):
    """The tokens of a batch by their adapter: ids int32 [T], each token's slot,
    outside [0, n) for none.  One plan serves every projection of every layer.
    `plan`: one of the same T and n, written anew (a captured graph's, say)."""
    torch = _torch()
    dev = _cuda(ids, "adapter_plan")
    T = ids.numel()
    p = _flat(ids, "ids", T, dev, torch.int32)
    if plan is None:
        size = lib().moe_adapter_plan_bytes(T, n)
        if not size:
            raise ValueError(f"unsupported sizes: {T} tokens, {n} adapters")
        plan = AdapterPlan(T, n, torch.empty(max(size, 256), dtype=torch.uint8, device=dev))
    elif plan.T != T or plan.n != n or plan.device != dev:
        raise ValueError(f"the plan is of {plan.T} tokens and {plan.n} adapters on {plan.device}")
    if T:
        _call("moe_adapter_plan", dev, p, T, n, plan.data.data_ptr(), plan.data.numel())
    return plan


def _pitch(t, name, T, H):
    """Elements between the rows of t [T, H], whose own lie side by side."""
    ld, one = t.stride()
    if one != 1 and H > 1:
        raise ValueError(f"the elements of a row of {name} must lie side by side")
    return ld if T > 1 else max(ld, H)


def add_adapters_workspace(adapters, T):
    """Workspace of add_adapters for T tokens."""
    n = lib().moe_add_adapters_workspace_bytes(ctypes.byref(adapters.c()), T)
    return _torch().empty(max(n, 256), dtype=_torch().uint8, device=adapters.device)


def check_workspace(adapters, T, ws):
    """Refuses a workspace that add_adapters would refuse, in the same way."""
    of, need = adapters.space
    if of != T:
        need = lib().moe_add_adapters_workspace_bytes(adapters.at, T)
        adapters.space = T, need
    at = _flat_on(ws, "the workspace", ws.numel(), adapters.index, adapters.bytes)
    if T and ws.numel() < need:
        raise MoeError(MOE_EWORKSPACE, "moe_add_adapters", f"workspace needs {need} bytes")
    if T and at % 256:
        raise MoeError(MOE_EINVAL, "moe_add_adapters", "workspace must be 256-byte aligned")


def add_adapters(adapters, x, plan, y, scale=None, out=None, ws=None):
    """out[t] = y[t] + s * B (A x[t]) with the adapter of token t: x [T, K] of the
    adapters' type, or int8 codes with their scale (quantize_i8, block norms); y
    [T, N] of any float type.  out: of y's type, y itself if not given.  Returns
    out."""
    i = _gpu(x, "add_adapters")
    if adapters.index != i or plan.index != i:
        raise ValueError(f"x is on {x.device}, the adapters on {adapters.device}, the plan on "
                         f"{plan.device}")
    torch = _torch()
    T, width = x.shape
    K, N = adapters.K, adapters.N
    if plan.T != T or plan.n != adapters.n:
        raise ValueError(f"the plan is of {plan.T} tokens and {plan.n} adapters, the call of {T} "
                         f"and {adapters.n}")
    ps = 0
    if x.dtype is adapters.dtype:
        dt = adapters.w_dtype
        if scale is not None:
            raise ValueError("scales go with int8 codes only")
        if width != K:
            raise ValueError(f"x must be [T, {K}], got {list(x.shape)}")
    elif x.dtype is torch.int8:
        dt = DT_I8
        if scale is None:
            raise ValueError("codes need their scales")
        if width < codes_width(K):
            raise ValueError(f"codes must be [T, at least {codes_width(K)}], got {list(x.shape)}")
        ps = _flat_on(scale, "scale", T, i, torch.float32)
    else:
        raise ValueError(f"x must be {adapters.dtype} or int8 codes, got {x.dtype}")
    ldx = _pitch(x, "x", T, width)
    if out is None:
        out = y
    for t, name in ((y, "y"), (out, "out")):
        if t.shape != (T, N) or t.dtype is not y.dtype or t.get_device() != i:
            raise ValueError(f"{name} must be [{T}, {N}] of y's type on GPU {i}, got "
                             f"{list(t.shape)} {t.dtype} on {t.device}")
    ldy, ldo = _pitch(y, "y", T, N), _pitch(out, "out", T, N)
    yt = _type(y.dtype)
    if ws is None:
        ws = add_adapters_workspace(adapters, T)
    size = ws.numel()
    wp = _flat_on(ws, "the workspace", size, i, torch.uint8)
    if T:
        _call_on("moe_add_adapters", i, adapters.at, x.data_ptr(), dt, ldx, ps, plan.at, T,
                 y.data_ptr(), ldy, out.data_ptr(), ldo, yt, wp, size)
    return out
