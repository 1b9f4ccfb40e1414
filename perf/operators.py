"""The operators around and inside a low-bit MoE layer, and what measuring them takes.

    norm      N(r; w) before a block (moeq.block_norm)
    residual  r' = r_scale r + y_scale gate N(y; post_w), then N(r'; pre_w): the norm after one
              block and before the next, with the gate, the scales and the residual stream
              (moeq.block_residual)
    combine   the same with y = sum_j w_j y_perm[inv_perm] + y_shared, a routed layer's gated sum
              (moeq.combine_residual)
    linear    a product in 8-bit integers, a scale per token and per channel (moeq.linear_i8)
    ffn       the routed experts' gated feed-forward in 8-bit integers, rows in the order of
              moeq.permute (moeq.expert_ffn_i8)
    shared    the same for one expert that every token passes through (moeq.shared_ffn_i8)

with N(v; w) = v / sqrt(mean(v^2) + eps) * w, and the 8-bit codes of a row
q = rint(v * (127 / max|v|)) with its scale max|v| / 127.

H 6144, I 2048, 256 experts and 8 per token are this repository's layer.
"""

import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # one decoded token entering a block: nothing but latency
        dict(name="norm T1", kind="norm", T=1, H=6144, type="bf16"),
        # a short odd batch of a small model whose residual stream is kept in fp32
        dict(name="residual T333 H1003", kind="residual", T=333, H=1003, type="fp32", post=True,
             gate="token"),
        # prefill between two blocks: norm after, a gate per channel, norm before
        dict(name="residual T4096", kind="residual", T=4096, H=6144, type="bf16", post=True,
             gate="channel"),
        # the end of the routed layer at a decode step, with a shared expert
        dict(name="combine T8", kind="combine", T=8, H=6144, k=8, E=256, type="bf16", post=True,
             gate="none", shared=True),
        # and at prefill
        dict(name="combine T4096", kind="combine", T=4096, H=6144, k=8, E=256, type="bf16",
             post=False, gate="none", shared=False),
        # a projection of one decoded token: the weights' stream
        dict(name="linear T1", kind="linear", T=1, K=6144, N=6144, type="bf16", bias=False),
        # a small odd batch through odd widths
        dict(name="linear T37 K1001 N2500", kind="linear", T=37, K=1001, N=2500, type="fp16",
             bias=True),
        # a projection at prefill: the matrix cores
        dict(name="linear T4096", kind="linear", T=4096, K=6144, N=6144, type="bf16", bias=False),
        # the routed experts of one token, of a decode batch and of a prefill batch
        dict(name="ffn T1", kind="ffn", T=1, H=6144, I=2048, E=256, k=8, type="bf16"),
        dict(name="ffn T32", kind="ffn", T=32, H=6144, I=2048, E=256, k=8, type="bf16"),
        dict(name="ffn T4096", kind="ffn", T=4096, H=6144, I=2048, E=256, k=8, type="bf16"),
        # the shared expert on a ragged prefill chunk
        dict(name="shared T500", kind="shared", T=500, H=6144, I=2048, type="bf16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "residual", "combine", "linear", "ffn", "shared"])
    T = _spread(rng, 1, 4096)
    if kind == "norm":
        return dict(kind=kind, T=T, H=_spread(rng, 64, 8192), type=rng.choice(sorted(TYPES)))
    if kind == "residual":
        return dict(kind=kind, T=T, H=_spread(rng, 64, 8192), type=rng.choice(sorted(TYPES)),
                    post=rng.random() < 0.5, gate=rng.choice(["none", "token", "channel", "full"]))
    if kind == "combine":
        E = _spread(rng, 8, 256)
        return dict(kind=kind, T=T, H=4 * _spread(rng, 64, 1536), k=rng.randint(1, min(E, 8)), E=E,
                    type=rng.choice(sorted(TYPES)), post=rng.random() < 0.5,
                    gate=rng.choice(["none", "token", "channel"]), shared=rng.random() < 0.5)
    if kind == "linear":
        return dict(kind=kind, T=T, K=_spread(rng, 64, 6144), N=_spread(rng, 16, 6144),
                    type=rng.choice(["bf16", "fp16"]), bias=rng.random() < 0.5)
    H, I = 16 * _spread(rng, 16, 384), 16 * _spread(rng, 4, 128)
    if kind == "shared":
        return dict(kind=kind, T=T, H=H, I=I, type=rng.choice(["bf16", "fp16"]))
    E = _spread(rng, 4, 128)
    return dict(kind=kind, T=T, H=H, I=I, E=E, k=rng.randint(1, min(E, 8)),
                type=rng.choice(["bf16", "fp16"]))


# ---------------------------------------------------------------- inputs

def _codes_of_weights(g, *shape):
    """8-bit codes of normally distributed weights, a row's largest near 4 sigma."""
    out = torch.empty(shape, dtype=torch.int8, device="cuda")
    flat = out.view(-1)
    step = 1 << 28
    for at in range(0, flat.numel(), step):
        part = flat[at:at + step]
        w = torch.empty(part.shape, dtype=torch.float32, device="cuda").normal_(0, 31, generator=g)
        part.copy_(w.round_().clamp_(-127, 127))
    return out


def _scales(g, *shape):
    return (torch.randn(shape, generator=g, device="cuda") * 0.2).exp() * (0.02 * 4 / 127)


def _activations(g, T, H, dtype, scale=1.0):
    """Rows as a decoder's: normal values under channel scales, some of them large."""
    ch = (torch.randn(H, generator=g, device="cuda") * 0.5).exp() * scale
    return (torch.randn(T, H, generator=g, device="cuda") * ch).to(dtype)


def _route(g, T, E, k, skew):
    """Expert ids [T, k] of a router that is nearly balanced, and the permutation by expert."""
    logits = torch.rand(T, E, generator=g, device="cuda")
    logits = logits + skew * torch.randn(E, generator=g, device="cuda")
    top, ids = torch.topk(logits, k, dim=1)
    flat = ids.reshape(-1)
    perm = torch.argsort(flat, stable=True)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device="cuda")
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return torch.softmax(top, 1), perm.to(torch.int32), inv.to(torch.int32), offsets, counts


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind, T, dt = case["kind"], case["T"], TYPES[case["type"]]
    st = dict(case)
    if kind in ("norm", "residual", "combine"):
        H = case["H"]
        st["r"] = _activations(g, T, H, dt, 2.0)
        st["pre_w"] = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(dt)
        st["n"] = torch.empty_like(st["r"])
        if kind != "norm":
            st["r_out"] = torch.empty_like(st["r"])
            st["post_w"] = ((1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(dt)
                            if case["post"] else None)
            shape = {"none": None, "token": (T, 1), "channel": (1, H), "full": (T, H)}[case["gate"]]
            st["g"] = (torch.sigmoid(torch.randn(shape, generator=g, device="cuda")).to(dt)
                       if shape else None)
            st["y_scale"], st["r_scale"] = 0.7, 1.0
        if kind == "residual":
            st["y"] = _activations(g, T, H, dt)
        if kind == "combine":
            k = case["k"]
            st["w"], _, st["inv"], _, _ = _route(g, T, case["E"], k, 0.02)
            st["y"] = _activations(g, T * k, H, dt)
            st["y_shared"] = _activations(g, T, H, dt) if case["shared"] else None
    elif kind == "linear":
        K, N = case["K"], case["N"]
        st["x"] = _activations(g, T, K, dt)
        st["w"], st["s"] = _codes_of_weights(g, N, K), _scales(g, N)
        st["b"] = 0.1 * torch.randn(N, generator=g, device="cuda") if case["bias"] else None
        st["out"] = torch.empty(T, N, dtype=dt, device="cuda")
    else:
        H, I = case["H"], case["I"]
        E, k = case.get("E", 1), case.get("k", 1)
        st["x"] = _activations(g, T, H, dt)
        st["w13"], st["s13"] = _codes_of_weights(g, E, 2 * I, H), _scales(g, E, 2 * I)
        st["w2"], st["s2"] = _codes_of_weights(g, E, H, I), _scales(g, E, H)
        st["out"] = torch.empty(T * k, H, dtype=dt, device="cuda")
        if kind == "ffn":
            _, st["perm"], _, st["offsets"], counts = _route(g, T, E, k, 0.02)
            # a plan for products over padded groups: the experts in use, the longest group
            st["used"] = torch.nonzero(counts).flatten()
            st["most"] = int(counts.max())
    if own:
        import bit_quantized_moe_route_amd as moeq

        if kind == "linear":
            st["lin"] = moeq.I8Linear(st["w"], st["s"], bias=st["b"])
            st["ws"] = moeq.linear_i8_workspace(st["lin"], T)
        elif kind in ("ffn", "shared"):
            st["layer"] = moeq.I8Layer(st["w13"], st["s13"], st["w2"], st["s2"])
            st["ws"] = moeq.ffn_i8_workspace(st["layer"], T, case.get("k", 1))
    return st


# ---------------------------------------------------------------- plain forms

def _norm(v, w):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * w.float()


def _codes(v):
    """Integer codes (as fp32) and scales of the rows of v."""
    a = v.abs().amax(-1, keepdim=True)
    return torch.round(v * (127.0 / a)), a / 127.0


def _after(st, y):
    r = st["r"]
    if st["post_w"] is not None:
        y = _norm(y, st["post_w"])
    if st["g"] is not None:
        y = y * st["g"].float()
    r = st["r_scale"] * r.float() + st["y_scale"] * y
    return r.to(st["r"].dtype), _norm(r, st["pre_w"]).to(st["r"].dtype)


def _gated(gu, I):
    g, u = gu[..., :I], gu[..., I:]
    return g / (1 + torch.exp(-g)) * u


def _ffn(st):
    I, k = st["I"], st["k"]
    q, s = _codes(st["x"].float())
    used, most = st["used"], st["most"]
    at = torch.arange(st["T"] * k, device="cuda")
    group = torch.searchsorted(st["offsets"][1:][used], at, right=True)    # place in `used`
    e, row = used[group], at - st["offsets"][used[group]]
    token = torch.div(st["perm"], k, rounding_mode="floor").long()
    pad = torch.zeros(len(used), most, st["H"], device="cuda")
    pad[group, row] = q[token]
    gu = torch.bmm(pad, st["w13"][used].float().transpose(1, 2))[group, row]
    h, sh = _codes(_gated(gu * s[token] * st["s13"][e], I))
    pad = torch.zeros(len(used), most, I, device="cuda")
    pad[group, row] = h
    y = torch.bmm(pad, st["w2"][used].float().transpose(1, 2))[group, row]
    return (y * sh * st["s2"][e]).to(st["x"].dtype)


def run(st):
    kind = st["kind"]
    if own:
        import bit_quantized_moe_route_amd as moeq

        if kind == "norm":
            return moeq.block_norm(st["r"], st["pre_w"], eps=EPS, out=st["n"])
        if kind == "residual":
            return moeq.block_residual(st["r"], st["y"], st["pre_w"], post_w=st["post_w"],
                                       gate=st["g"], y_scale=st["y_scale"], r_scale=st["r_scale"],
                                       eps=EPS, r_out=st["r_out"], out=st["n"])
        if kind == "combine":
            return moeq.combine_residual(st["r"], st["y"], st["inv"], st["w"], st["pre_w"],
                                         y_shared=st["y_shared"], post_w=st["post_w"],
                                         gate=st["g"], y_scale=st["y_scale"],
                                         r_scale=st["r_scale"], eps=EPS, r_out=st["r_out"],
                                         out=st["n"])
        if kind == "linear":
            return moeq.linear_i8(st["lin"], st["x"], out=st["out"], ws=st["ws"])
        if kind == "ffn":
            return moeq.expert_ffn_i8(st["layer"], st["x"], st["perm"], st["offsets"], st["k"],
                                      y_perm=st["out"], ws=st["ws"])
        return moeq.shared_ffn_i8(st["layer"], st["x"], y=st["out"], ws=st["ws"])
    if kind == "norm":
        return _norm(st["r"].float(), st["pre_w"]).to(st["r"].dtype)
    if kind == "residual":
        return _after(st, st["y"].float())
    if kind == "combine":
        y = st["y"][st["inv"].long()].float().view(st["T"], st["k"], st["H"])
        y = (y * st["w"][:, :, None]).sum(1)
        return _after(st, y if st["y_shared"] is None else y + st["y_shared"].float())
    if kind == "linear":
        q, s = _codes(st["x"].float())
        y = q @ st["w"].float().t() * s * st["s"]
        return (y if st["b"] is None else y + st["b"]).to(st["x"].dtype)
    if kind == "ffn":
        return _ffn(st)
    q, s = _codes(st["x"].float())
    h, sh = _codes(_gated(q @ st["w13"][0].float().t() * s * st["s13"], st["I"]))
    return (h @ st["w2"][0].float().t() * sh * st["s2"]).to(st["x"].dtype)


# ---------------------------------------------------------------- work

def work(case):
    kind, T, b = case["kind"], case["T"], SIZE[case["type"]]
    if kind in ("norm", "residual", "combine"):
        H = case["H"]
        rows = 2 if kind == "norm" else 4                        # r, n; y (or its sum), r'
        extra = 1
        flops = 4
        if kind == "combine":
            rows += case["k"] - 1 + case["shared"]
            flops += 2 * case["k"]
        if kind != "norm":
            extra += case["post"] + (case["gate"] == "channel")
            rows += case["gate"] == "full"
            flops += 8
        return dict(bytes=(rows * T + extra) * H * b, flops=flops * T * H)
    if kind == "linear":
        K, N = case["K"], case["N"]
        return dict(bytes=N * K + 4 * N + T * (K + N) * b, flops=2 * T * N * K)
    H, I, E, k = case["H"], case["I"], case.get("E", 1), case.get("k", 1)
    used = E * (1 - (1 - k / E) ** T) if E > k else E
    return dict(bytes=used * (3 * H * I + 4 * (2 * I + H)) + T * H * b + T * k * (H * b + 4),
                flops=6 * T * k * H * I)


# ---------------------------------------------------------------- in 64 bits

def _codes64(v):
    most = v.abs().max(dim=1).values[:, None]
    return (v * 127 / most).round(), most / 127


def _rms64(v, w):
    return v / ((v * v).sum(1, keepdim=True) / v.shape[1] + EPS).sqrt() * w.double()


def _expert64(q, s, w13, s13, w2, s2):
    gu = (q @ w13.double().T) * s * s13.double()
    g, u = gu.chunk(2, dim=1)
    q, s = _codes64(g * torch.sigmoid(g) * u)
    return (q @ w2.double().T) * s * s2.double()


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        return _rms64(st["r"].double(), st["pre_w"])
    if kind in ("residual", "combine"):
        v = st["y"].double()
        if kind == "combine":
            total = torch.zeros(st["r"].shape, dtype=torch.float64, device="cuda")
            slots = st["inv"].long().view(-1, case["k"])
            for j in range(case["k"]):
                total += st["w"][:, j, None].double() * v[slots[:, j]]
            v = total if st["y_shared"] is None else total + st["y_shared"].double()
        if case["post"]:
            v = _rms64(v, st["post_w"])
        if st["g"] is not None:
            v = v * st["g"].double()
        v = st["r"].double() * st["r_scale"] + v * st["y_scale"]
        return v, _rms64(v, st["pre_w"])
    q, s = _codes64(st["x"].double())
    if kind == "linear":
        y = (q @ st["w"].double().T) * s * st["s"].double()
        return y if st["b"] is None else y + st["b"].double()
    if kind == "shared":
        return _expert64(q, s, st["w13"][0], st["s13"][0], st["w2"][0], st["s2"][0])
    out = torch.empty(st["out"].shape, dtype=torch.float64, device="cuda")
    bounds = st["offsets"].tolist()
    token = st["perm"].long() // case["k"]
    for e in range(case["E"]):
        at = slice(bounds[e], bounds[e + 1])
        if at.start < at.stop:
            out[at] = _expert64(q[token[at]], s[token[at]], st["w13"][e], st["s13"][e],
                                st["w2"][e], st["s2"][e])
    return out
