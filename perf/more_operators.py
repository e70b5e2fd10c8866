"""Cases of the norm with its 8-bit output and its gradient, the microscaled 4-bit product and the whole layer of
experts for a few tokens.

`run` computes a case with elementary torch operations, in 32 bits, or in 64 where codes are chosen, or, where `own`
is true, with the library's entry points; `exact` gives the same outputs from the definitions in 64 bits.
"""
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # One token: the norm in front of a square 8-bit projection.
        {"name": "norm 8-bit one token", "op": "norm8", "M": 1, "K": 4096, "N": 4096, "type": "bf16", "residual": True},
        # A long prompt in front of the narrow projection to shared keys and values: the norm takes most of it.
        {"name": "norm 8-bit prompt", "op": "norm8", "M": 8192, "K": 8192, "N": 1024, "type": "bf16", "residual": True},
        # Odd widths in full precision, the first norm of a model: nothing to add yet.
        {"name": "norm 8-bit odd", "op": "norm8", "M": 1000, "K": 777, "N": 1500, "type": "f32", "residual": False},
        # A training batch: the norm of the residual stream, forward and backward.
        {"name": "norm training", "op": "norm", "M": 16384, "K": 4096, "type": "bf16"},
        # One token through a square projection held in 4 bits.
        {"name": "4-bit one token", "op": "mx4", "E": 1, "M": 1, "K": 4096, "N": 4096, "type": "bf16", "out": "bf16",
         "bias": False},
        # A long prompt through a large projection: the largest product here.
        {"name": "4-bit prompt", "op": "mx4", "E": 1, "M": 8192, "K": 8192, "N": 8192, "type": "bf16", "out": "bf16",
         "bias": False},
        # Odd widths, whose last block of 32 is not whole, with a bias, from and to 32 bits.
        {"name": "4-bit odd", "op": "mx4", "E": 1, "M": 1000, "K": 777, "N": 1500, "type": "f32", "out": "f32",
         "bias": True},
        # A serving batch sorted by expert, experts held in 4 bits.
        {"name": "4-bit experts", "op": "mx4", "E": 16, "M": 256, "K": 4096, "N": 2048, "type": "bf16", "out": "bf16",
         "bias": False},
        # One decoding step of one sequence through a gated layer, two experts a token.
        {"name": "layer bf16 one token", "op": "layer", "E": 16, "T": 1, "top": 2, "D": 4096, "F": 2048, "type": "bf16",
         "weights": "bf16", "gated": True, "padding": 0},
        # Eight sequences over many experts held in 4 bits.
        {"name": "layer 4-bit eight tokens", "op": "layer", "E": 32, "T": 8, "top": 2, "D": 4096, "F": 2048,
         "type": "bf16", "weights": "mx4", "gated": True, "padding": 0},
        # A batch filled up to a captured size, experts held in 8 bits: nearly every expert is used.
        {"name": "layer 8-bit batch", "op": "layer", "E": 16, "T": 64, "top": 2, "D": 4096, "F": 2048, "type": "bf16",
         "weights": "int8", "gated": True, "padding": 5},
        # A small layer in full precision on odd widths, without a gate.
        {"name": "layer f32 odd", "op": "layer", "E": 6, "T": 5, "top": 2, "D": 777, "F": 500, "type": "f32",
         "weights": "f32", "gated": False, "padding": 0},
    ]


def _spread(rng, low, high):
    """A size between low and high, even over its logarithm; one in three is rounded to a multiple of 64."""
    n = int(round(low * (high / low) ** rng.random()))
    return max(64, n // 64 * 64) if low >= 64 and rng.random() < 1 / 3 else n


def draw(rng):
    op = rng.choice(("norm8", "norm", "mx4", "mx4", "layer", "layer"))
    kind = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "norm8":
        while True:
            M, K, N = _spread(rng, 1, 16384), _spread(rng, 64, 16384), _spread(rng, 64, 4096)
            if M * K <= 1 << 26 and M * K * N <= 1 << 37:
                return {"op": op, "M": M, "K": K, "N": N, "type": kind, "residual": rng.random() < 0.7}
    if op == "norm":
        while True:
            M, K = _spread(rng, 1, 16384), _spread(rng, 64, 16384)
            if M * K <= 1 << 26:
                return {"op": op, "M": M, "K": K, "type": kind}
    if op == "mx4":
        E = 1 if rng.random() < 0.5 else int(round(2 * 32 ** rng.random()))
        while True:
            M, K, N = _spread(rng, 1, 16384), _spread(rng, 64, 8192), _spread(rng, 64, 8192)
            if M * K * N <= 1 << 37 and E * K * N <= 1 << 27:
                return {"op": op, "E": E, "M": M, "K": K, "N": N, "type": kind,
                        "out": rng.choice(("bf16", "f16", "f32")), "bias": rng.random() < 0.5}
    E = int(round(2 * 32 ** rng.random()))
    while True:
        D, F = _spread(rng, 64, 4096), _spread(rng, 64, 4096)
        if E * D * F <= 1 << 28:
            break
    T = int(round(64 ** rng.random()))
    return {"op": op, "E": E, "T": T, "top": rng.randint(1, min(8, E)), "D": D, "F": F, "type": kind,
            "weights": rng.choice((kind, "int8", "mx4")), "gated": rng.random() < 0.7, "padding": rng.randint(0, T // 4)}


def _shares(E):
    """How often each expert is chosen: some six times as often as others."""
    w = [1.0 + 5.0 * ((7 * e + 3) % E) / E for e in range(E)]
    return [x / sum(w) for x in w]


def _tokens(g, M, K, kind):
    """Activations: unit variance, a few channels eight times as large."""
    loud = 1 + 7 * (torch.rand(K, device="cuda", generator=g) < 0.01).float()
    return (torch.randn(M, K, device="cuda", generator=g) * loud).to(TYPES[kind])


def _codes(g, *shape):
    """Weights in 8 bits: codes and a scale for each channel."""
    q = torch.empty(shape, dtype=torch.int8, device="cuda")
    for part in q if len(shape) == 3 else (q,):  # an expert at a time, for the room that floats take
        part.copy_((torch.randn(part.shape, device="cuda", generator=g) * 40).round().clamp(-127, 127))
    return q, (0.5 + torch.rand(shape[:-1], device="cuda", generator=g)) * (shape[-1] ** -0.5 / 40)


def _blocks(g, *shape):
    """Weights in 4 bits: two codes a byte and a scale for each 32, most of them within a few powers of two."""
    K = shape[-1]
    q = torch.randint(0, 256, (*shape[:-1], (K + 1) // 2), dtype=torch.uint8, device="cuda", generator=g)
    if K % 2:
        q[..., -1] &= 15
    low = 124 - (K - 1).bit_length() // 2
    scale = torch.randint(low, low + 4, (*shape[:-1], (K + 31) // 32), dtype=torch.uint8, device="cuda", generator=g)
    return q, scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, kind = case["op"], TYPES[case["type"]]
    if op == "layer":
        E, T, top, D, F = (case[k] for k in ("E", "T", "top", "D", "F"))
        shares = torch.tensor(_shares(E), device="cuda").expand(T, E)
        ids = torch.multinomial(shares, top, generator=g).to(torch.int32)
        if case["padding"]:
            ids[T - case["padding"]:] = -1
        s = {"op": op, "ids": ids, "share": torch.rand(T, top, device="cuda", generator=g).softmax(1),
             "x": _tokens(g, T, D, case["type"]), "y": torch.empty(T, D, dtype=kind, device="cuda"),
             "gated": case["gated"], "scales_in": None, "scales_out": None}
        up, down = (E, 2 * F if case["gated"] else F, D), (E, D, F)
        if case["weights"] == "int8":
            (s["w_in"], s["scales_in"]), (s["w_out"], s["scales_out"]) = _codes(g, *up), _codes(g, *down)
        elif case["weights"] == "mx4":
            (s["w_in"], s["scales_in"]), (s["w_out"], s["scales_out"]) = _blocks(g, *up), _blocks(g, *down)
        else:
            for name, shape in (("w_in", up), ("w_out", down)):
                s[name] = torch.empty(shape, dtype=kind, device="cuda")
                for part in s[name]:
                    part.copy_(torch.randn(shape[1:], device="cuda", generator=g) * shape[2] ** -0.5)
        return s
    M, K = case["M"], case["K"]
    x = _tokens(g, M, K, case["type"])
    s = {"op": op, "x": x}
    if op == "mx4":
        E, N = case["E"], case["N"]
        s["w"], s["ws"] = _blocks(g, E, N, K)
        s["bias"] = torch.randn(E, N, device="cuda", generator=g) if case["bias"] else None
        s["q"] = torch.empty(M, (K + 1) // 2, dtype=torch.uint8, device="cuda")
        s["qs"] = torch.empty(M, (K + 31) // 32, dtype=torch.uint8, device="cuda")
        s["y"] = torch.empty(M, N, dtype=TYPES[case["out"]], device="cuda")
        s["offsets"], s["largest"] = None, M
        if E == 1:
            s["w"], s["ws"], s["bias"] = s["w"][0], s["ws"][0], s["bias"][0] if case["bias"] else None
        else:
            sizes = torch.multinomial(torch.tensor(_shares(E), device="cuda"), M, replacement=True, generator=g)
            sizes = sizes.bincount(minlength=E)
            s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
            s["offsets"][1:] = sizes.cumsum(0)
            s["largest"] = int(sizes.max())
        return s
    s["weight"] = (1 + 0.2 * torch.randn(K, device="cuda", generator=g)).to(kind)
    # The residual stream is a few times as large as what a layer adds to it.
    s["r"] = 3 * _tokens(g, M, K, case["type"]) if op == "norm" or case["residual"] else None
    s["h"] = torch.empty_like(x) if s["r"] is not None else None
    if op == "norm":
        s["dy"] = torch.randn(M, K, device="cuda", generator=g).to(kind)
        s["dh"] = torch.randn(M, K, device="cuda", generator=g).to(kind)
        s["y"], s["dx"] = torch.empty_like(x), torch.empty_like(x)
        s["dw"] = torch.empty(K, dtype=torch.float32, device="cuda")
        return s
    s["q"] = torch.empty(M, K, dtype=torch.int8, device="cuda")
    s["qs"] = torch.empty(M, dtype=torch.float32, device="cuda")
    s["w"], s["ws"] = _codes(g, case["N"], K)
    s["y"] = torch.empty(M, case["N"], dtype=kind, device="cuda")
    return s


def _plain_norm8(s):
    # Codes in 64 bits: in 32, values next to the border between two codes fall on either side of it.
    h = s["x"].double() if s["r"] is None else s["x"].double() + s["r"].double()
    v = h * s["weight"].double()
    top = v.abs().amax(1, keepdim=True)
    q = torch.round(v * 127 / torch.where(top > 0, top, 1.0)).float()
    scale = (top / 127 * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)).float()
    y = ((q @ s["w"].float().t()) * scale * s["ws"]).to(s["y"].dtype)
    return (y, scale[:, 0]) if s["r"] is None else (y, scale[:, 0], h.to(s["h"].dtype))


def _plain_norm(s):
    w = s["weight"].float()
    h = s["x"].float() + s["r"].float()
    y = (h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * w).to(s["y"].dtype)
    kept = h.to(s["h"].dtype)
    # The backward pass starts from what the forward pass kept.
    h, dy = kept.float(), s["dy"].float()
    r = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    n, v = h * r, dy * w
    dx = r * (v - n * (v * n).mean(1, keepdim=True)) + s["dh"].float()
    return y, kept, dx.to(s["dx"].dtype), (dy * n).sum(0)


def _unpack(q, scale, K):
    """Codes of 4 bits and a scale for each 32 of them as 32-bit values."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    v = table[torch.stack((q & 15, q >> 4), -1).int()].flatten(-2)[..., :K]
    return v * torch.exp2(scale.float() - 127).repeat_interleave(32, -1)[..., :K]


def _round_to_blocks(x):
    """The 4-bit values of x and their scales multiplied, in 32 bits: products of powers of two, so nothing is lost."""
    M, K = x.shape
    b = torch.nn.functional.pad(x.double(), (0, -K % 32)).view(M, -1, 32)
    top = b.abs().amax(2, keepdim=True)
    e = (torch.frexp(top).exponent - 3).clamp(-127, 127).double()
    step = torch.exp2(torch.where(top > 0, e, -127.0))
    v = b / step
    a = v.abs()
    a = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2)).clamp(max=6)
    return (torch.copysign(a, v) * step).view(M, -1)[:, :K].float()


def _plain_mx4(s):
    x, K = _round_to_blocks(s["x"]), s["x"].shape[1]
    w = _unpack(s["w"], s["ws"], K)
    if s["offsets"] is None:
        y = x @ w.t()
        return (y if s["bias"] is None else y + s["bias"]).to(s["y"].dtype)
    # Each row's place in a stack that gives every expert room for the largest one.
    E, cap, row = w.shape[0], s["largest"], torch.arange(x.shape[0], device="cuda")
    expert = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    slot = expert * cap + row - s["offsets"].long()[expert]
    p = torch.zeros(E * cap, K, device="cuda")
    p[slot] = x
    y = torch.bmm(p.view(E, cap, K), w.transpose(1, 2)).flatten(0, 1)[slot]
    return (y if s["bias"] is None else y + s["bias"][expert]).to(s["y"].dtype)


def _wide(w, scale, K):
    if w.dtype == torch.int8:
        return w.float() * scale[..., None]
    return _unpack(w, scale, K) if w.dtype == torch.uint8 else w.float()


def _act(u, gated):
    if not gated:
        return u * torch.sigmoid(u)
    a, b = u.chunk(2, -1)
    return a * torch.sigmoid(a) * b


def _plain_layer(s):
    x, ids, w_in, w_out = s["x"].float(), s["ids"].long(), s["w_in"], s["w_out"]
    (T, D), E, top = x.shape, w_in.shape[0], ids.shape[1]
    F = w_in.shape[1] // 2 if s["gated"] else w_in.shape[1]
    share = torch.where(ids >= 0, s["share"], 0.0)
    ids = ids.clamp(min=0)
    part = lambda t, e: None if t is None else t[e]  # noqa: E731
    if T * top < E:  # the chosen experts' weights, one copy for each use
        e = ids.flatten()
        u = torch.bmm(_wide(w_in[e], part(s["scales_in"], e), D), x.repeat_interleave(top, 0)[:, :, None])[..., 0]
        h = _act(u, s["gated"]) * share.flatten()[:, None]
        y = torch.bmm(_wide(w_out[e], part(s["scales_out"], e), F), h[:, :, None])[..., 0].view(T, top, D).sum(1)
    else:  # every expert for every token, with a share of zero where it was not chosen
        each = torch.zeros(T, E, device="cuda").scatter_add_(1, ids, share)
        u = (x @ _wide(w_in, s["scales_in"], D).flatten(0, 1).t()).view(T, E, -1)
        h = _act(u, s["gated"]) * each[:, :, None]
        y = torch.bmm(h.transpose(0, 1), _wide(w_out, s["scales_out"], F).transpose(1, 2)).sum(0)
    return y.to(s["y"].dtype)


def run(state):
    s = state
    if not own:
        return {"norm8": _plain_norm8, "norm": _plain_norm, "mx4": _plain_mx4, "layer": _plain_layer}[s["op"]](s)
    import fp32_gemm_amd as lib
    if s["op"] == "norm8":
        lib.rms_norm(s["x"], s["weight"], residual=s["r"], H=s["h"], Q=s["q"], scale=s["qs"], eps=EPS)
        y = lib.igemm(s["q"], s["qs"], s["w"], s["ws"], s["y"])
        return (y, s["qs"]) if s["r"] is None else (y, s["qs"], s["h"])
    if s["op"] == "norm":
        lib.rms_norm(s["x"], s["weight"], s["y"], residual=s["r"], H=s["h"], eps=EPS)
        lib.rms_norm_grad(s["dy"], s["h"], s["weight"], s["dx"], s["dw"], residual_grad=s["dh"], eps=EPS)
        return s["y"], s["h"], s["dx"], s["dw"]
    if s["op"] == "mx4":
        lib.quantize_mx4(s["x"], s["q"], s["qs"])
        return lib.gemm_mx4(s["q"], s["qs"], s["w"], s["ws"], s["y"], bias=s["bias"], offsets=s["offsets"])
    return lib.expert_layer(s["x"], s["ids"], s["share"], s["w_in"], s["w_out"], s["y"], scale_in=s["scales_in"],
                            scale_out=s["scales_out"], gated=s["gated"])


def work(case):
    op, size = case["op"], SIZE[case["type"]]
    if op == "layer":
        E, T, top, D, F = (case[k] for k in ("E", "T", "top", "D", "F"))
        T -= case["padding"]
        # Experts that no token chose keep their weights unread: the expected number of the others.
        used = sum(1 - (1 - min(1, top * p)) ** T for p in _shares(E))
        rows = 3 * F if case["gated"] else 2 * F
        each = {"int8": rows * D + 4 * (rows - F + D), "mx4": rows * D * (1 / 2 + 1 / 32)}.get(case["weights"], rows * D * size)
        return {"bytes": used * each + T * (2 * D * size + 8 * top), "flops": 2 * T * top * rows * D}
    M, K = case["M"], case["K"]
    if op == "norm":  # x, r and y, h; dy, h, dh and dx
        return {"bytes": 8 * M * K * size + 2 * K * size + 4 * K, "flops": 18 * M * K}
    N = case["N"]
    if op == "norm8":
        adds = 3 if case["residual"] else 1
        return {"bytes": adds * M * K * size + K * size + 4 * M + N * (K + 4) + M * N * size, "flops": 2 * M * K * N}
    used = sum(1 - (1 - p) ** M for p in _shares(case["E"]))
    total = M * K * size + used * N * (K * (1 / 2 + 1 / 32) + 4 * case["bias"]) + M * N * SIZE[case["out"]]
    return {"bytes": total, "flops": 2 * M * K * N}


def _exact_values(q, scale, K):
    """What 4-bit codes stand for: sign, two bits of exponent, one of mantissa, times 2 to the scale less 127."""
    c = torch.empty(*q.shape, 2, dtype=torch.float64, device="cuda")
    for i, part in enumerate((q % 16, q // 16)):
        e, m = (part // 2 % 4).double(), (part % 2).double()
        c[..., i] = torch.where(e > 0, 2.0 ** (e - 1) * (1 + m / 2), m / 2) * (1 - 2 * (part // 8).double())
    c = c.flatten(-2)[..., :K]
    block = torch.arange(K, device="cuda") // 32
    return c * 2.0 ** (scale.double()[..., block] - 127)


def _exact_rounding(x):
    """The nearest of the values 0, 1/2, 1, 3/2, 2, 3, 4, 6 to each of a block's, scaled so that the largest is in [4, 8)."""
    K = x.shape[1]
    block = torch.arange(K, device="cuda") // 32
    top = torch.zeros(x.shape[0], (K + 31) // 32, dtype=torch.float64, device="cuda")
    top.scatter_reduce_(1, block.expand_as(x), x.abs(), "amax")
    e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    e += (2.0 ** (e + 1) <= top).double() - (2.0 ** e > top).double()  # where the logarithm was rounded across
    unit = (2.0 ** (e - 2).clamp(-127, 127))[:, block]
    a = x.abs() / unit
    y = torch.zeros_like(a)
    for i in range(1, 8):  # from one value to the next past their middle; at the middle to the even code
        middle = (E2M1[i - 1] + E2M1[i]) / 2
        y = torch.where((a >= middle) if i % 2 == 0 else (a > middle), E2M1[i], y)
    return torch.where(x < 0, -y, y) * unit


def exact(case, seed):
    s = prepare(case, seed)
    op, K = case["op"], case.get("K")
    x = s["x"].double()
    if op == "layer":
        y = torch.zeros_like(x)
        for t, (row, part) in enumerate(zip(s["ids"].tolist(), s["share"].double().tolist())):
            for e, p in zip(row, part):
                if e < 0:
                    continue
                w = []
                for name, scales, depth in (("w_in", "scales_in", case["D"]), ("w_out", "scales_out", case["F"])):
                    one = s[name][e]
                    w.append(one.double() * s[scales][e].double()[:, None] if one.dtype == torch.int8 else
                             _exact_values(one, s[scales][e], depth) if one.dtype == torch.uint8 else one.double())
                u = w[0] @ x[t]
                h = u / (1 + torch.exp(-u))
                if case["gated"]:
                    h = h[:case["F"]] * u[case["F"]:]
                y[t] += p * (w[1] @ h)
        return y
    M = case["M"]
    if op == "mx4":
        q, y = _exact_rounding(x), torch.zeros(M, case["N"], dtype=torch.float64, device="cuda")
        at = [0, M] if s["offsets"] is None else s["offsets"].tolist()
        E, N = case["E"], case["N"]
        w, ws = s["w"].reshape(E, N, -1), s["ws"].reshape(E, N, -1)
        for e in range(E):
            y[at[e]:at[e + 1]] = q[at[e]:at[e + 1]] @ _exact_values(w[e], ws[e], K).t()
            if s["bias"] is not None:
                y[at[e]:at[e + 1]] += s["bias"].reshape(E, N)[e].double()
        return y
    w = s["weight"].double()
    h = x if s["r"] is None else x + s["r"].double()
    rms = torch.sqrt((h ** 2).sum(1, keepdim=True) / K + EPS)
    if op == "norm8":
        top = (h * w).abs().max(dim=1, keepdim=True).values
        codes = torch.where(top > 0, torch.round((h * w) * 127 / torch.where(top > 0, top, 1)), 0)
        scale = top / rms / 127
        y = (codes @ s["w"].double().t()) * scale * s["ws"].double()
        return (y, scale[:, 0]) if s["r"] is None else (y, scale[:, 0], h)
    y = h / rms * w
    k = s["h"].copy_(h).double()  # as the forward pass keeps it
    rms = torch.sqrt((k ** 2).sum(1, keepdim=True) / K + EPS)
    dy = s["dy"].double()
    dx = dy * w / rms - k * (dy * w * k).sum(1, keepdim=True) / (K * rms ** 3) + s["dh"].double()
    return y, h, dx, (dy * k / rms).sum(0)
