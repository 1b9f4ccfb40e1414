"""What stands beside and behind a projection of a decoder step, and what measuring it takes.

    heads     queries and keys as a projection leaves them, each head's norm and the rotation by
              its token's position in one pass (moeq.head_norm_rope):
              n = v / sqrt(mean(v^2) + eps) * w over the D elements of a head, then for the pairs
              (a, b) of its first R elements a cos - b sin, b cos + a sin
    logprob   log probabilities of given tokens, the distribution's entropy and its best tokens
              (moeq.token_logprobs): p = softmax(scale[t] * logits[t]),
              log p[ids], -sum p log p, the top largest (ties: lower id first) with their log p
    adapters  low-rank adapters of many requests beside a projection they share
              (moeq.add_adapters): y[t] + s[a] * B[a] (A[a] x[t]), a the adapter of token t's
              request (-1: none), each of its own rank

H 6144 is this repository's layer.
"""

import math

import torch

own = False

EPS = 1e-5
BASE = 10000.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "codes": 1}


def listed():
    return [
        # one decoded token's queries and keys: nothing but latency
        dict(name="heads T1", kind="heads", T=1, Hq=64, Hk=8, D=128, R=128, pairs="halves",
             P=131072, type="bf16"),
        # a ragged chunk of a small model kept in fp32, part of each head rotated
        dict(name="heads T333 D80", kind="heads", T=333, Hq=12, Hk=12, D=80, R=32,
             pairs="neighbours", P=4096, type="fp32"),
        # a prefill chunk
        dict(name="heads T4096", kind="heads", T=4096, Hq=64, Hk=8, D=128, R=128, pairs="halves",
             P=131072, type="bf16"),
        # one decoded token, its log probability and what a user sees beside it
        dict(name="logprob T1", kind="logprob", T=1, V=131072, m=1, top=5, masked=False,
             type="fp32"),
        # a decode batch with a temperature per request and tokens that a grammar forbids
        dict(name="logprob T32", kind="logprob", T=32, V=131072, m=1, top=20, masked=True,
             type="fp32"),
        # a short prompt of a small vocabulary of odd size, no alternatives asked for
        dict(name="logprob T333 V50257", kind="logprob", T=333, V=50257, m=2, top=0, masked=False,
             type="fp16"),
        # a prompt's tokens scored at prefill
        dict(name="logprob T2048", kind="logprob", T=2048, V=131072, m=1, top=8, masked=False,
             type="bf16"),
        # one decoded token of one request
        dict(name="adapters T1", kind="adapters", T=1, K=6144, N=6144, n=32, least=16, most=16,
             x="bf16", w="bf16", y="bf16", spread="tokens"),
        # a decode batch, nearly every token with an adapter of its own, ranks from 8 to 64
        dict(name="adapters T64", kind="adapters", T=64, K=6144, N=2048, n=64, least=8, most=64,
             x="codes", w="bf16", y="bf16", spread="tokens"),
        # a ragged batch through odd widths
        dict(name="adapters T500 K1001", kind="adapters", T=500, K=1001, N=2500, n=7, least=3,
             most=40, x="fp16", w="fp16", y="fp32", spread="tokens"),
        # prompts of eight requests in one prefill batch
        dict(name="adapters T4096", kind="adapters", T=4096, K=6144, N=6144, n=8, least=64,
             most=64, x="bf16", w="bf16", y="bf16", spread="requests"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["heads", "logprob", "adapters"])
    if kind == "heads":
        D = 2 * _spread(rng, 16, 128)
        Hk = _spread(rng, 1, 8)
        Hq = Hk * rng.choice([1, 2, 4, 8])
        most = max(1, min(4096, 4096 * 72 * 128 // ((Hq + Hk) * D)))
        return dict(kind=kind, T=_spread(rng, 1, most), Hq=Hq, Hk=Hk, D=D,
                    R=D if rng.random() < 0.5 else 2 * rng.randint(1, D // 2),
                    pairs=rng.choice(["halves", "neighbours"]), P=_spread(rng, 4096, 131072),
                    type=rng.choice(sorted(TYPES)))
    if kind == "logprob":
        V = _spread(rng, 1000, 160000)
        dt = rng.choice(sorted(TYPES))
        most = 2048 * 131072 * 2 // (V * SIZE[dt])
        return dict(kind=kind, T=_spread(rng, 1, min(4096, most)), V=V, m=rng.randint(1, 4),
                    top=rng.choice([0, 1, 5, 8, 20]), masked=rng.random() < 0.3, type=dt)
    w = rng.choice(["bf16", "fp16"])
    least, most = sorted((_spread(rng, 2, 64), _spread(rng, 2, 64)))
    return dict(kind=kind, T=_spread(rng, 1, 4096), K=_spread(rng, 64, 6144),
                N=_spread(rng, 16, 6144), n=_spread(rng, 1, 64), least=least, most=most,
                x=rng.choice([w, w, "codes"]), w=w, y=rng.choice([w, "fp32"]),
                spread=rng.choice(["tokens", "requests"]))


# ---------------------------------------------------------------- inputs

def _activations(g, T, H, dtype):
    """Rows as a decoder's: normal values under channel scales, some of them large."""
    ch = (torch.randn(H, generator=g, device="cuda") * 0.5).exp()
    return (torch.randn(T, H, generator=g, device="cuda") * ch).to(dtype)


def _frequencies(R):
    return BASE ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)


def _heads(st, g, dt):
    T, Hq, Hk, D, R, P = (st[n] for n in ("T", "Hq", "Hk", "D", "R", "P"))
    # queries, keys and values side by side, as one projection writes them
    rows = _activations(g, T, (Hq + 2 * Hk) * D, dt)
    st["q"] = rows[:, :Hq * D].view(T, Hq, D)
    st["k"] = rows[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    for n in ("q_w", "k_w"):
        st[n] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
    # a prompt's chunk somewhere in the context, or tokens of as many requests
    first = int(torch.randint(0, max(1, P - T), (1,), generator=g, device="cuda"))
    st["pos"] = torch.arange(first, first + T, device="cuda", dtype=torch.int32).clamp_(max=P - 1)
    if T <= 64:
        st["pos"] = torch.randint(0, P, (T,), generator=g, device="cuda", dtype=torch.int32)
    angle = torch.arange(P, dtype=torch.float64, device="cuda")[:, None] * _frequencies(R)
    st["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    st["q_out"] = torch.empty(T, Hq, D, dtype=dt, device="cuda")
    st["k_out"] = torch.empty(T, Hk, D, dtype=dt, device="cuda")


def _logits(st, g, dt):
    T, V = st["T"], st["V"]
    # a bulk of unlikely tokens and some that the model finds likely, fewer the likelier
    out = torch.empty(T, V, dtype=dt, device="cuda")
    for t in range(0, T, 256):
        n = min(256, T - t)
        v = torch.randn(n, V, generator=g, device="cuda") * 2 - 3
        at = torch.randint(0, V, (n, 1), generator=g, device="cuda")
        at = (at + torch.arange(40, device="cuda") * (V // 40)) % V     # no place twice
        v.scatter_add_(1, at, 14 * torch.rand(n, 40, generator=g, device="cuda") ** 2)
        if st["masked"]:
            v[torch.rand(n, V, generator=g, device="cuda") < 0.6] = -math.inf
            v.scatter_(1, at[:, :32], torch.rand(n, 32, generator=g, device="cuda") * 8)
        out[t:t + n] = v
    st["logits"] = out
    # the sampled tokens: among the likely ones
    near = out[:, :V // 2].float().argmax(1, keepdim=True)
    far = out[:, V // 2:].float().argmax(1, keepdim=True) + V // 2
    st["ids"] = torch.cat([near, far] * 2, 1)[:, :st["m"]].to(torch.int32).contiguous()
    st["scale"] = 0.5 + torch.rand(T, generator=g, device="cuda") if T > 1 else None
    st["logprob"] = torch.empty(T, st["m"], device="cuda")
    st["entropy"] = torch.empty(T, device="cuda")
    if st["top"]:
        st["top_ids"] = torch.empty(T, st["top"], dtype=torch.int32, device="cuda")
        st["top_logprob"] = torch.empty(T, st["top"], device="cuda")


def _adapters(st, g):
    T, K, N, n = st["T"], st["K"], st["N"], st["n"]
    dt = TYPES[st["w"]]
    ranks = torch.linspace(st["least"], st["most"], n).round().int().tolist()
    st["ranks"] = ranks
    st["a"] = [(torch.randn(r, K, generator=g, device="cuda") * K ** -0.5).to(dt) for r in ranks]
    st["b"] = [(torch.randn(N, r, generator=g, device="cuda") * 0.3 * r ** -0.5).to(dt)
               for r in ranks]
    st["s"] = (0.5 + torch.rand(n, generator=g, device="cuda")).tolist()
    if st["spread"] == "requests":      # prompts of unequal lengths, one after the other
        cuts = torch.sort(torch.randint(0, T + 1, (n - 1,), generator=g, device="cuda")).values
        ids = torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)
    else:                               # any adapter for any token, some tokens without
        ids = torch.randint(0, n, (T,), generator=g, device="cuda")
        if T > 1:
            ids[torch.rand(T, generator=g, device="cuda") < 0.1] = -1
    st["ids"] = ids.to(torch.int32)
    x = _activations(g, T, K, dt)
    st["x_scale"] = None
    if st["x"] == "codes":
        width = (K + 63) // 64 * 64
        most = x.float().abs().amax(1, keepdim=True)
        st["x_scale"] = (most / 127).flatten()
        q = torch.zeros(T, width, dtype=torch.int8, device="cuda")
        q[:, :K] = torch.round(x.float() * (127 / most))
        x = q
    st["in"] = x
    st["y_in"] = _activations(g, T, N, TYPES[st["y"]])
    st["out"] = torch.empty_like(st["y_in"])
    # the tokens of each adapter, and the matrices padded to one rank, side by side: what a
    # product over padded groups takes
    order = torch.argsort(st["ids"], stable=True)
    order = order[st["ids"][order] >= 0]
    used, counts = torch.unique_consecutive(st["ids"][order], return_counts=True)
    st["order"], st["group"] = order, torch.repeat_interleave(counts)
    begin = counts.cumsum(0) - counts
    st["row"] = torch.arange(len(order), device="cuda") - begin[st["group"]]
    st["used"], st["longest"] = used.long(), int(counts.max()) if len(order) else 0
    st["at"] = torch.zeros(n, max(ranks), K, dtype=dt, device="cuda")
    st["bt"] = torch.zeros(n, max(ranks), N, dtype=dt, device="cuda")
    for i, r in enumerate(ranks):
        st["at"][i, :r] = st["a"][i]
        st["bt"][i, :r] = st["b"][i].t()
    st["at"] = st["at"].transpose(1, 2).contiguous()
    st["st"] = torch.tensor(st["s"], device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)
    if case["kind"] == "heads":
        _heads(st, g, TYPES[case["type"]])
    elif case["kind"] == "logprob":
        _logits(st, g, TYPES[case["type"]])
    else:
        _adapters(st, g)
    if own:
        import bit_quantized_moe_route_amd as moeq

        if case["kind"] == "logprob":
            st["ws"] = moeq.token_logprobs_workspace(st["logits"], top=case["top"])
        elif case["kind"] == "adapters":
            st["set"] = moeq.Adapters(case["n"], case["most"], case["K"], case["N"],
                                      dtype=TYPES[case["w"]], device="cuda")
            for i, (a, b, s) in enumerate(zip(st["a"], st["b"], st["s"])):
                st["set"].load(i, a, b, s)
            # one plan of a batch serves every projection of every layer
            st["plan"] = moeq.adapter_plan(st["ids"], case["n"])
            st["ws"] = moeq.add_adapters_workspace(st["set"], case["T"])
    return st


# ---------------------------------------------------------------- plain forms

def _head_norm_rope(st, x, w):
    R = st["R"]
    v = x.float()
    v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * w.float()
    row = st["table"][st["pos"].long()][:, None]
    cos, sin = row[..., :R // 2], row[..., R // 2:]
    out = v.clone()
    if st["pairs"] == "halves":
        a, b = v[..., :R // 2], v[..., R // 2:R]
        out[..., :R // 2], out[..., R // 2:R] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = v[..., 0:R:2], v[..., 1:R:2]
        out[..., 0:R:2], out[..., 1:R:2] = a * cos - b * sin, b * cos + a * sin
    return out.to(x.dtype)


def _token_logprobs(st):
    z = st["logits"].float()
    if st["scale"] is not None:
        z = z * st["scale"][:, None]
    z = z - z.amax(1, keepdim=True)
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    z = z - torch.log(total)
    entropy = -(e * z.clamp_min(-1e30)).sum(1) / total[:, 0]
    logprob = z.gather(1, st["ids"].long())
    if not st["top"]:
        return logprob, entropy
    # whole numbers that order as the values do, equal ones by their place
    bits = (st["logits"].float() + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -2147483648 - bits, bits) * st["V"] \
        - torch.arange(st["V"], device="cuda")
    ids = (-torch.topk(key, st["top"], 1).values) % st["V"]
    return logprob, entropy, ids.to(torch.int32), z.gather(1, ids)


def _add_adapters(st):
    group, row, used = st["group"], st["row"], st["used"]
    x = st["in"][:, :st["K"]].float()
    if st["x_scale"] is not None:
        x = x * st["x_scale"][:, None]
    y = st["y_in"].to(torch.float32, copy=True)
    if len(used) == 0:
        return y.to(st["y_in"].dtype)
    pad = torch.zeros(len(used), st["longest"], st["K"], device="cuda")
    pad[group, row] = x[st["order"]]
    h = torch.bmm(pad, st["at"][used].float()) * st["st"][used][:, None, None]
    y[st["order"]] += torch.bmm(h, st["bt"][used].float())[group, row]
    return y.to(st["y_in"].dtype)


def run(st):
    if own:
        import bit_quantized_moe_route_amd as moeq

        if st["kind"] == "heads":
            return moeq.head_norm_rope(st["q"], st["k"], st["q_w"], st["k_w"], pos=st["pos"],
                                       table=st["table"], interleaved=st["pairs"] == "neighbours",
                                       eps=EPS, q_out=st["q_out"], k_out=st["k_out"])
        if st["kind"] == "logprob":
            return moeq.token_logprobs(st["logits"], st["ids"], top=st["top"], scale=st["scale"],
                                       logprob=st["logprob"], entropy=st["entropy"],
                                       top_ids=st.get("top_ids"),
                                       top_logprob=st.get("top_logprob"), ws=st["ws"])
        return moeq.add_adapters(st["set"], st["in"], st["plan"], st["y_in"],
                                 scale=st["x_scale"], out=st["out"], ws=st["ws"])
    if st["kind"] == "heads":
        return (_head_norm_rope(st, st["q"], st["q_w"]), _head_norm_rope(st, st["k"], st["k_w"]))
    if st["kind"] == "logprob":
        return _token_logprobs(st)
    return _add_adapters(st)


# ---------------------------------------------------------------- work

def work(case):
    T = case["T"]
    if case["kind"] == "heads":
        D, heads, b = case["D"], case["Hq"] + case["Hk"], SIZE[case["type"]]
        return dict(bytes=T * (2 * heads * D * b + 4 + 4 * case["R"]) + 2 * D * b,
                    flops=T * heads * (4 * D + 3 * case["R"]))
    if case["kind"] == "logprob":
        return dict(bytes=T * (case["V"] * SIZE[case["type"]] + 8 * case["m"] + 8
                               + 8 * case["top"]),
                    flops=6 * T * case["V"])
    K, N, n = case["K"], case["N"], case["n"]
    rank = (case["least"] + case["most"]) / 2
    used = n * (1 - (1 - 1 / n) ** T)
    return dict(bytes=used * rank * (K + N) * SIZE[case["w"]] + T * K * SIZE[case["x"]]
                + 2 * T * N * SIZE[case["y"]],
                flops=2 * T * rank * (K + N))


# ---------------------------------------------------------------- in 64 bits

def _heads64(st, x, w):
    v = x.double()
    v = v / (v.pow(2).sum(2, keepdim=True) / st["D"] + EPS).sqrt() * w.double()
    R = st["R"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       st["pos"].double()[:, None, None] * _frequencies(R))
    first, rest = v[:, :, :R], v[:, :, R:]
    if st["pairs"] == "halves":
        z = torch.complex(*first.chunk(2, dim=2)) * turn
        return torch.cat([z.real, z.imag, rest], 2)
    z = torch.view_as_real(torch.view_as_complex(first.unflatten(2, (-1, 2)).contiguous()) * turn)
    return torch.cat([z.flatten(2), rest], 2)


def _logprobs64(st):
    said = []
    for t in range(0, st["T"], 128):
        at = slice(t, t + 128)
        z = st["logits"][at].double()
        order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :st["top"]]
        if st["scale"] is not None:
            z = z * st["scale"][at, None].double()
        z = z - torch.logsumexp(z, 1, keepdim=True)
        p = z.exp()
        said.append((z.gather(1, st["ids"][at].long()),
                     -torch.where(p > 0, p * z, torch.zeros_like(p)).sum(1),
                     order.to(torch.int32), z.gather(1, order)))
    said = [torch.cat(parts) for parts in zip(*said)]
    return tuple(said if st["top"] else said[:2])


def _adapters64(st):
    out = st["y_in"].double()
    x = st["in"][:, :st["K"]].double()
    if st["x_scale"] is not None:
        x = x * st["x_scale"].double()[:, None]
    for i in range(st["n"]):
        rows = torch.nonzero(st["ids"] == i).flatten()
        if len(rows):
            out[rows] += (x[rows] @ st["a"][i].double().T) @ st["b"][i].double().T * st["s"][i]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "heads":
        return _heads64(st, st["q"], st["q_w"]), _heads64(st, st["k"], st["k_w"])
    if case["kind"] == "logprob":
        return _logprobs64(st)
    return _adapters64(st)
