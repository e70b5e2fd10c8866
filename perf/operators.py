"""Cases of the grouped products, their weight gradient and the 8-bit integer product.

`run` computes a case with elementary torch operations in 32 bits, or, where
`own` is true, with the library's entry points; `exact` gives the same outputs
from the definitions in 64 bits.
"""
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # One decoding step of eight sequences, two experts a token: most experts get nothing or one row.
        {"name": "experts bf16 decode", "op": "grouped", "E": 32, "M": 16, "K": 2048, "N": 1024,
         "type": "bf16", "out": "bf16", "transposed": True},
        # The up projection of a long training batch, weights stored as they multiply.
        {"name": "experts bf16 batch", "op": "grouped", "E": 16, "M": 16384, "K": 4096, "N": 2048,
         "type": "bf16", "out": "bf16", "transposed": False},
        # The same layer's input gradient: the same weights, read transposed.
        {"name": "experts bf16 input gradient", "op": "grouped", "E": 16, "M": 16384, "K": 2048, "N": 4096,
         "type": "bf16", "out": "bf16", "transposed": True},
        # A short prompt on odd widths: no row of X, W or Y after the first is aligned to 16 bytes.
        {"name": "experts f16 odd", "op": "grouped", "E": 8, "M": 1000, "K": 1500, "N": 777,
         "type": "f16", "out": "f16", "transposed": False},
        # Full-precision training of a small model.
        {"name": "experts f32", "op": "grouped", "E": 8, "M": 4097, "K": 2048, "N": 1024,
         "type": "f32", "out": "f32", "transposed": False},
        # The weight gradient of the long batch, kept in 32 bits for the optimiser.
        {"name": "weight gradient bf16 batch", "op": "wgrad", "E": 16, "M": 16384, "K": 4096, "N": 2048,
         "type": "bf16", "out": "f32"},
        # A small batch over many experts: short sums, some of them empty.
        {"name": "weight gradient bf16 short", "op": "wgrad", "E": 32, "M": 512, "K": 1024, "N": 1024,
         "type": "bf16", "out": "bf16"},
        # Odd widths in full precision.
        {"name": "weight gradient f32 odd", "op": "wgrad", "E": 8, "M": 1000, "K": 777, "N": 1500,
         "type": "f32", "out": "f32"},
        # One token through a square projection.
        {"name": "int8 one token", "op": "int8", "E": 1, "M": 1, "K": 4096, "N": 4096,
         "type": "bf16", "out": "bf16", "bias": False},
        # A long prompt through a large projection: the largest product here.
        {"name": "int8 prompt", "op": "int8", "E": 1, "M": 8192, "K": 8192, "N": 8192,
         "type": "bf16", "out": "bf16", "bias": False},
        # Odd widths, with a bias, from and to 32 bits.
        {"name": "int8 odd", "op": "int8", "E": 1, "M": 1000, "K": 777, "N": 1500,
         "type": "f32", "out": "f32", "bias": True},
        # A serving batch over experts held in 8 bits.
        {"name": "int8 experts", "op": "int8", "E": 16, "M": 256, "K": 4096, "N": 2048,
         "type": "bf16", "out": "bf16", "bias": False},
    ]


def _spread(rng, low, high):
    """A size between low and high, even over its logarithm; one in three is rounded to a multiple of 64."""
    n = int(round(low * (high / low) ** rng.random()))
    return max(64, n // 64 * 64) if low >= 64 and rng.random() < 1 / 3 else n


def draw(rng):
    op = rng.choice(("grouped", "grouped", "wgrad", "int8", "int8"))
    E = 1 if op == "int8" and rng.random() < 0.5 else int(round(2 * 32 ** rng.random()))
    while True:
        M, K, N = _spread(rng, 1, 16384), _spread(rng, 64, 8192), _spread(rng, 64, 8192)
        # No more work than the largest listed case, no more weights than the largest listed stack of experts.
        if M * K * N <= 1 << 37 and E * K * N <= 1 << 27:
            break
    if op == "int8":
        return {"op": op, "E": E, "M": M, "K": K, "N": N, "type": rng.choice(("bf16", "f16", "f32")),
                "out": rng.choice(("bf16", "f16", "f32")), "bias": rng.random() < 0.5}
    kind = rng.choice(("bf16", "bf16", "f16", "f32"))
    case = {"op": op, "E": E, "M": M, "K": K, "N": N, "type": kind,
            "out": rng.choice((kind, "f32"))}
    return dict(case, transposed=rng.random() < 0.5) if op == "grouped" else case


def _shares(E):
    """How often each expert is chosen: some six times as often as others."""
    w = [1.0 + 5.0 * ((7 * e + 3) % E) / E for e in range(E)]
    return [x / sum(w) for x in w]


def _tokens(g, M, K, kind):
    """Activations: unit variance, a few channels eight times as large."""
    loud = 1 + 7 * (torch.rand(K, device="cuda", generator=g) < 0.01).float()
    return (torch.randn(M, K, device="cuda", generator=g) * loud).to(TYPES[kind])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, E, M, K, N = (case[k] for k in ("op", "E", "M", "K", "N"))
    shares = torch.tensor(_shares(E), device="cuda")
    sizes = torch.multinomial(shares, M, replacement=True, generator=g).bincount(minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = sizes.cumsum(0)
    s = {"op": op, "offsets": offsets, "largest": int(sizes.max()), "x": _tokens(g, M, K, case["type"])}
    out = TYPES[case["out"]]
    if op == "wgrad":
        s["dy"] = torch.randn(M, N, device="cuda", generator=g).to(TYPES[case["type"]])
        s["dw"] = torch.empty(E, K, N, dtype=out, device="cuda")
        return s
    s["y"] = torch.empty(M, N, dtype=out, device="cuda")
    if op == "grouped":
        s["transposed"] = case["transposed"]
        shape = (E, N, K) if case["transposed"] else (E, K, N)
        s["w"] = (torch.randn(shape, device="cuda", generator=g) * K ** -0.5).to(TYPES[case["type"]])
        return s
    if E == 1:
        s["offsets"] = None
    s["q"] = torch.empty(M, K, dtype=torch.int8, device="cuda")
    s["qs"] = torch.empty(M, dtype=torch.float32, device="cuda")
    s["w"] = (torch.randn(E, N, K, device="cuda", generator=g) * 40).round().clamp(-127, 127).to(torch.int8)
    s["ws"] = (0.5 + torch.rand(E, N, device="cuda", generator=g)) * (K ** -0.5 / 40)
    s["bias"] = torch.randn(E, N, device="cuda", generator=g) if case["bias"] else None
    if E == 1:
        s["w"], s["ws"], s["bias"] = s["w"][0], s["ws"][0], s["bias"][0] if case["bias"] else None
    return s


def _slots(s):
    """Each row's place in a stack that gives every expert room for the largest one."""
    row = torch.arange(s["x"].shape[0], device="cuda")
    expert = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    return expert, expert * s["largest"] + row - s["offsets"].long()[expert]


def _stack(s, x, slot):
    E, cap = s["offsets"].numel() - 1, s["largest"]
    p = torch.zeros(E * cap, x.shape[1], dtype=torch.float32, device="cuda")
    p[slot] = x.float()
    return p.view(E, cap, x.shape[1])


def _plain(s):
    if s["op"] == "wgrad":
        _, slot = _slots(s)
        return torch.bmm(_stack(s, s["x"], slot).transpose(1, 2), _stack(s, s["dy"], slot)).to(s["dw"].dtype)
    if s["op"] == "grouped":
        _, slot = _slots(s)
        w = s["w"].float()
        y = torch.bmm(_stack(s, s["x"], slot), w.transpose(1, 2) if s["transposed"] else w)
        return y.flatten(0, 1)[slot].to(s["y"].dtype)
    # In 64 bits: in 32, values next to the border between two codes fall on either side of it.
    x = s["x"].double()
    top = x.abs().amax(1)
    q = torch.round(x * 127 / torch.where(top > 0, top, 1.0)[:, None]).float()
    scale = (top / 127).float()
    if s["offsets"] is None:
        y = (q @ s["w"].float().t()) * scale[:, None] * s["ws"]
        y = y if s["bias"] is None else y + s["bias"]
        return y.to(s["y"].dtype), scale
    expert, slot = _slots(s)
    y = torch.bmm(_stack(s, q, slot), s["w"].float().transpose(1, 2)).flatten(0, 1)[slot]
    y = y * scale[:, None] * s["ws"][expert]
    y = y if s["bias"] is None else y + s["bias"][expert]
    return y.to(s["y"].dtype), scale


def run(state):
    s = state
    if not own:
        return _plain(s)
    import fp32_gemm_amd as lib
    if s["op"] == "grouped":
        return lib.gemm_grouped(s["x"], s["w"], s["offsets"], s["y"], transpose_w=s["transposed"])
    if s["op"] == "wgrad":
        return lib.gemm_grouped_wgrad(s["x"], s["dy"], s["offsets"], s["dw"])
    lib.quantize_rows(s["x"], s["q"], s["qs"])
    y = lib.igemm(s["q"], s["qs"], s["w"], s["ws"], s["y"], bias=s["bias"], offsets=s["offsets"])
    return y, s["qs"]


def work(case):
    op, E, M, K, N = (case[k] for k in ("op", "E", "M", "K", "N"))
    # Experts that no row chose keep their weights unread: the expected number of the others.
    used = sum(1 - (1 - p) ** M for p in _shares(E))
    size, out = SIZE[case["type"]], SIZE[case["out"]]
    if op == "wgrad":
        total = M * (K + N) * size + E * K * N * out
    elif op == "grouped":
        total = M * K * size + used * K * N * size + M * N * out
    else:
        total = M * K * size + used * N * (K + 4 + 4 * case["bias"]) + M * N * out + 4 * M
    return {"bytes": total, "flops": 2 * M * K * N}


def exact(case, seed):
    s = prepare(case, seed)
    M, E = case["M"], case["E"]
    at = [0, M] if s["offsets"] is None else s["offsets"].tolist()
    x = s["x"].double()
    if case["op"] == "wgrad":
        dw = torch.zeros(E, case["K"], case["N"], dtype=torch.float64, device="cuda")
        for e in range(E):
            dw[e] = x[at[e]:at[e + 1]].t() @ s["dy"][at[e]:at[e + 1]].double()
        return dw
    y = torch.zeros(M, case["N"], dtype=torch.float64, device="cuda")
    if case["op"] == "grouped":
        for e in range(E):
            w = s["w"][e].double()
            y[at[e]:at[e + 1]] = x[at[e]:at[e + 1]] @ (w.t() if case["transposed"] else w)
        return y
    # The largest magnitude of a token becomes 127; a token of zeros keeps zeros.
    top = x.abs().max(dim=1, keepdim=True).values
    codes = torch.where(top > 0, torch.round(x * 127 / torch.where(top > 0, top, 1)), 0)
    n = case["N"]
    w, ws = s["w"].reshape(E, n, -1), s["ws"].reshape(E, n)
    for e in range(E):
        part = codes[at[e]:at[e + 1]] @ w[e].double().t()
        y[at[e]:at[e + 1]] = part * (top[at[e]:at[e + 1]] / 127) * ws[e].double()
        if s["bias"] is not None:
            y[at[e]:at[e + 1]] += s["bias"].reshape(E, n)[e].double()
    return y, top[:, 0] / 127
