"""The operators in 4 bits (E2M1 codes in blocks with a scale), in plain torch operations and as the framework's
own calls:

* quant   - rows of activations or weights to codes and scales, and back to the values that they stand for;
* product - y = alpha x w^T of two matrices in 4 bits;
* append  - queries and keys normalised per head and rotated, keys and values appended in 4 bits to the cache's
            pages, and the pages expanded for attention that wants bf16;
* decode  - one decode step over the cache in 4 bits, requests of different lengths.

mxfp4: a power of two (E8M0) per 32 elements; nvfp4: an E4M3 scale per 16 elements, times a constant of the tensor.
Codes are two a byte, the even element in the low half. The scales of `quant` and `product` lie in tiles of 128 rows x
4 scales, [rows / 128, scales / 4, 32, 4, 4]: row r's scale c at [r / 128, c / 4, r % 32, r / 32 % 4, c % 4]; those of the
cache beside its rows, [pages, page, Hkv, D / 16].
"""
import math
import random

import torch

own = False   # True: the framework's calls; False: the plain forms

EPS = 1e-6
BLOCK = {"mxfp4": 32, "nvfp4": 16}
HEADS = ((32, 8, 128), (16, 2, 64), (16, 8, 128), (8, 1, 128), (8, 8, 64), (4, 4, 128))
PAGES = (5, 8, 12, 16, 16, 32, 64)
TENSOR = {"x": 0.5, "k": 0.25, "v": 0.125}    # tensor scales of nvfp4


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one generated token's activations before a projection: latency alone
        {"name": "quant 1x4096", "op": "quant", "M": 1, "K": 4096, "kind": "nvfp4"},
        # a projection's weights, laid out once
        {"name": "quant 14336x4096", "op": "quant", "M": 14336, "K": 4096, "kind": "mxfp4"},
        # a projection of one token: the weights' bytes
        {"name": "product 1", "op": "product", "M": 1, "K": 4096, "N": 14336, "kind": "nvfp4", "out": "bf16"},
        # a decode step of 64 requests, the way back from the wide layer
        {"name": "product 64", "op": "product", "M": 64, "K": 14336, "N": 4096, "kind": "mxfp4", "out": "bf16"},
        # an odd batch, a narrow layer, results kept in 32 bits
        {"name": "product 777", "op": "product", "M": 777, "K": 2176, "N": 1000, "kind": "nvfp4", "out": "f32"},
        # the packed prompts of one prefill step
        {"name": "product 8192", "op": "product", "M": 8192, "K": 4096, "N": 14336, "kind": "nvfp4", "out": "bf16"},
        # a decode step of 64 requests, heads normalised
        {"name": "append 64", "op": "append", "tokens": 64, "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "rot": 128,
         "pairs": "halves", "norm": True, "far": 9000, "mix": 12},
        # the packed prompts of one prefill step
        {"name": "append 8192", "op": "append", "tokens": 8192, "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "rot": 128,
         "pairs": "halves", "norm": False, "far": 8192, "mix": 13},
        # one short conversation
        {"name": "decode 1x700", "op": "decode", "tokens": 1, "longest": 700, "shortest": 700, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 16, "mix": 1},
        # one long document
        {"name": "decode 1x32768", "op": "decode", "tokens": 1, "longest": 32768, "shortest": 32768, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 16, "mix": 2},
        # small heads, contexts of all lengths, some places of the batch empty, odd pages
        {"name": "decode 133 ragged", "op": "decode", "tokens": 133, "longest": 6000, "shortest": 1, "Hq": 16, "Hkv": 2,
         "D": 64, "page": 12, "mix": 3},
        # the largest step
        {"name": "decode 256x8192", "op": "decode", "tokens": 256, "longest": 8192, "shortest": 1000, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 16, "mix": 4},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    case = {"op": rng.choice(("quant", "product", "product", "append", "decode", "decode")), "mix": rng.randrange(1 << 20)}
    if case["op"] in ("quant", "product"):
        case["kind"] = rng.choice(("mxfp4", "nvfp4"))
        case["K"] = 128 * _log(rng, 1, 112)
        case["M"] = _log(rng, 1, 8192)
        if case["op"] == "product":
            case["N"] = 8 * _log(rng, 1, 1792)
            case["out"] = rng.choice(("bf16", "bf16", "f32"))
            case["M"] = max(1, min(case["M"], (8192 * 4096 * 14336) // (case["K"] * case["N"])))
        else:
            case["M"] = max(1, min(case["M"], (14336 * 4096) // case["K"]))
        return case
    case["Hq"], case["Hkv"], case["D"] = rng.choice(HEADS)
    case["page"] = rng.choice(PAGES)
    if case["op"] == "append":
        case["tokens"] = _log(rng, 1, 8192)
        case["rot"] = rng.choice((case["D"], case["D"], case["D"] // 2))
        case["pairs"] = rng.choice(("halves", "neighbours"))
        case["norm"] = case["tokens"] <= 256 and rng.random() < 0.75
        case["far"] = _log(rng, 10000, 120000)
    else:
        case["tokens"] = _log(rng, 1, 256)
        room = 256 * 8192 * 1024 // (case["tokens"] * case["Hkv"] * case["D"])
        case["longest"] = _log(rng, 1, min(32768, room))
        case["shortest"] = rng.choice((case["longest"], 1))
    return case


def _lengths(case):
    """Decode: the keys that each token sees, 0 in an empty place of the batch."""
    r = random.Random(case["mix"])
    out = [case["longest"]] + [r.randint(case["shortest"], case["longest"]) for _ in range(case["tokens"] - 1)]
    if case["shortest"] == 1:
        out = [out[0]] + [0 if r.random() < 0.05 else n for n in out[1:]]
    r.shuffle(out)
    return out


# ------------------------------------------------------------------------------------ the format

def _codes(y):
    """E2M1 codes of values in units of their block's scale: nearest, ties to even, at most 6."""
    a = y.abs()
    steps = (a > 0.25), (a >= 0.75), (a > 1.25), (a >= 1.75), (a > 2.5), (a >= 3.5), (a > 5)
    code = torch.zeros_like(y, dtype=torch.uint8)
    for s in steps:
        code += s
    return code | (torch.signbit(y).to(torch.uint8) << 3)


def _quantise(x, kind, tensor):
    """x [..., C] -> packed codes [..., C / 2] and the scales' bytes [..., C / block]."""
    x = x.float().unflatten(-1, (-1, BLOCK[kind]))
    most = x.abs().amax(-1, keepdim=True)
    if kind == "mxfp4":
        e = torch.where(most > 0, torch.frexp(most).exponent - 3, -127).clamp(-127, 127)
        byte = (e + 127).to(torch.uint8)
        y = torch.ldexp(x, -e)
    else:
        byte = (most / torch.full_like(most, 6 * tensor)).clamp(max=448).to(torch.float8_e4m3fn)   # (a quotient, no reciprocal)
        scale = byte.float() * tensor
        y = torch.where(scale > 0, x / scale, x * 0)
        byte = byte.view(torch.uint8)
    code = _codes(y).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte.squeeze(-1)


def _values(codes, scales, kind, tensor):
    """The values in 32 bits of packed codes [..., C / 2] with scale bytes [..., C / block]."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(-2)
    v = v.unflatten(-1, (-1, BLOCK[kind]))
    if kind == "mxfp4":
        s = torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127)
    else:
        s = scales.view(torch.float8_e4m3fn).float() * tensor
    return (v * s[..., None]).flatten(-2)


def _tile(s):
    """Scales [R, C] in tiles of 128 rows x 4."""
    R, C = s.shape
    t = torch.zeros((-(-R // 128) * 128, C), dtype=torch.uint8, device=s.device)
    t[:R] = s
    return t.view(-1, 4, 32, C // 4, 4).permute(0, 3, 2, 1, 4).contiguous()


def _untile(t, R):
    return t.permute(0, 3, 2, 1, 4).reshape(-1, 4 * t.shape[1])[:R]


# ------------------------------------------------------------------------------------ inputs

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=g.device, dtype=torch.float32).to(torch.bfloat16)


def _table(g, counts, spare=3):
    """Page tables of requests with `counts` pages each, pages handed out in a random order; -1 behind them."""
    total = sum(counts)
    order = torch.randperm(total + spare, generator=g, device=g.device).to(torch.int32)
    n = torch.tensor(counts, device=g.device)
    at = torch.arange(max(max(counts), 1), device=g.device)
    table = torch.where(at < n[:, None], order[((n.cumsum(0) - n)[:, None] + at).clamp(max=total + spare - 1)], -1)
    return table.to(torch.int32), total + spare


def _matrix(g, rows, K, kind, scale):
    """A matrix in 4 bits: codes [rows, K / 2], scales in tiles."""
    codes, scales = _quantise(_normal(g, rows, K).float() * scale, kind, TENSOR["x"])
    return codes, _tile(scales)


def _inputs(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7 + 3)
    s = {"case": case}
    if case["op"] == "quant":
        s["x"] = _normal(g, case["M"], case["K"])
        return s
    if case["op"] == "product":
        s["x"], s["sx"] = _matrix(g, case["M"], case["K"], case["kind"], 1.0)
        s["w"], s["sw"] = _matrix(g, case["N"], case["K"], case["kind"], 0.02)
        s["alpha"] = 1.0 if case["kind"] == "mxfp4" else 0.75
        return s
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    if case["op"] == "append":
        # requests of 257 tokens at most, each a run of positions that ends at most at `far`
        T, r = case["tokens"], random.Random(case["mix"])
        seqs, runs = -(-T // 257), []
        for b in range(seqs):
            n = min(257, T - 257 * b)
            runs.append((r.randint(0, case["far"] - n), n))
        s["q_seq"] = torch.arange(T, device=dev, dtype=torch.int32) // 257
        s["q_pos"] = torch.cat([torch.arange(a, a + n, device=dev, dtype=torch.int32) for a, n in runs])
        first = [a // page for a, _ in runs]
        counts = [(a + n - 1) // page - f + 1 for (a, n), f in zip(runs, first)]
        own_pages, pages = _table(g, counts)
        s["table"] = torch.full((seqs, max(f + c for f, c in zip(first, counts))), -1, dtype=torch.int32, device=dev)
        for b in range(seqs):
            s["table"][b, first[b]:first[b] + counts[b]] = own_pages[b, :counts[b]]
        s["pages"] = torch.arange(pages, device=dev, dtype=torch.int32)
        s["qkv"] = _normal(g, T, (Hq + 2 * Hkv) * D)
        if case["norm"]:
            s["gq"] = (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16)
            s["gk"] = (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16)
        half = case["rot"] // 2
        rate = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        angle = torch.arange(case["far"], device=dev, dtype=torch.float64)[:, None] * rate
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
    else:
        n = _lengths(case)
        s["table"], pages = _table(g, [-(-a // page) for a in n])
        s["q_seq"] = torch.arange(len(n), device=dev, dtype=torch.int32)
        s["q_pos"] = torch.tensor(n, device=dev, dtype=torch.int32) - 1
        s["max_pos"] = max(n) - 1
        s["q"] = _normal(g, len(n), Hq, D)
    for name in ("k", "v"):
        s[name + "_codes"] = torch.randint(0, 256, (pages, page, Hkv, D // 2), generator=g, device=dev, dtype=torch.uint8)
        s[name + "_scales"] = torch.randint(0x34, 0x44, (pages, page, Hkv, D // 16), generator=g, device=dev,
                                            dtype=torch.uint8)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import invariant_bi_gemm_gb300 as bi
        if case["op"] == "quant":
            s["handle"] = bi.BiQuant4(case["K"], case["kind"], tensor_scale=_tensor(case))
        elif case["op"] == "product":
            s["handle"] = bi.BiGemm4(case["K"], case["N"], case["kind"], out=case["out"])
        else:
            heads = case["Hq"], case["Hkv"], case["D"], case["page"]
            s["handle"] = bi.BiAttention4(*heads, k_scale=TENSOR["k"], v_scale=TENSOR["v"])
            if case["op"] == "append":
                s["rope"] = bi.BiQkRope(*heads, rot_dim=case["rot"], eps=EPS, interleaved=case["pairs"] == "neighbours")
    return s


def _tensor(case):
    return TENSOR["x"] if case["kind"] == "nvfp4" else 1.0


# ------------------------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if c["op"] == "quant":
        if own:
            codes, scales = s["handle"].run(s["x"])
            return s["handle"].expand(codes, scales)
        codes, scales = _quantise(s["x"], c["kind"], _tensor(c))
        return _values(codes, scales, c["kind"], _tensor(c)).to(torch.bfloat16)
    if c["op"] == "product":
        if own:
            return s["handle"].run(s["x"], s["sx"], s["w"], s["sw"], alpha=s["alpha"])
        x, w = (_values(s[a], _untile(s["s" + a], s[a].shape[0]), c["kind"], 1.0) for a in ("x", "w"))
        return torch.matmul(x, w.T).mul_(s["alpha"]).to(torch.bfloat16 if c["out"] == "bf16" else torch.float32)
    cache = s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"]
    if c["op"] == "append":
        if own:
            q = s["rope"].run4(s["qkv"], s.get("gq"), s.get("gk"), s["cos_sin"], s["q_seq"], s["q_pos"], *cache, s["table"],
                               k_scale=TENSOR["k"], v_scale=TENSOR["v"])
            k, v = s["handle"].expand(*cache, s["pages"])
            return {"q": q, "k": k, "v": v}
        q = _append(s)
        k, v = (_values(s[a + "_codes"], s[a + "_scales"], "nvfp4", TENSOR[a]).to(torch.bfloat16) for a in ("k", "v"))
        return {"q": q, "k": k, "v": v}
    if own:
        return s["handle"].run(s["q"], s["q_seq"], s["q_pos"], *cache, s["table"], s["max_pos"])
    return _decode(s)


def _append(s):
    c = s["case"]
    Hq, Hkv, D, page, rot = c["Hq"], c["Hkv"], c["D"], c["page"], c["rot"]
    q, k, v = s["qkv"].view(-1, Hq + 2 * Hkv, D).split((Hq, Hkv, Hkv), 1)
    pos = s["q_pos"].long()
    cos, sin = s["cos_sin"][pos].split(rot // 2, 1)

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * weight.float()
        r, rest = x[..., :rot], x[..., rot:]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["pairs"] == "neighbours" else (r[..., :rot // 2], r[..., rot // 2:])
        # (a block's codes turn on the last bit: the sums in 64 bits, of one product rounded to 32)
        co, si = cos[:, None].double(), sin[:, None]
        a, b = (a.double() * co - b * si).float(), (b.double() * co + a * si).float()
        r = torch.stack((a, b), -1).flatten(-2) if c["pairs"] == "neighbours" else torch.cat((a, b), -1)
        return torch.cat((r, rest), -1).to(torch.bfloat16)

    slot = s["table"][s["q_seq"].long(), pos // page].long() * page + pos % page
    for name, rows in (("k", turned(k, s.get("gk"))), ("v", v)):
        codes, scales = _quantise(rows, "nvfp4", TENSOR[name])
        s[name + "_codes"].view(-1, Hkv, D // 2)[slot] = codes
        s[name + "_scales"].view(-1, Hkv, D // 16)[slot] = scales
    return turned(q, s.get("gq"))


def _decode(s):
    c = s["case"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    T, L = s["q"].shape[0], s["max_pos"] + 1
    at = torch.arange(L, device=s["q"].device)
    slot = s["table"][s["q_seq"].long()][:, at // page].long().clamp_(min=0) * page + at % page

    def rows(name):
        codes, scales = (s[name + a].view(-1, Hkv, s[name + a].shape[-1])[slot] for a in ("_codes", "_scales"))
        return _values(codes, scales, "nvfp4", TENSOR[name])          # [T, L, Hkv, D]

    w = torch.matmul(s["q"].float().view(T, Hkv, Hq // Hkv, D), rows("k").permute(0, 2, 3, 1)).mul_(D ** -0.5)
    hidden = (at > s["q_pos"][:, None])[:, None, None]
    w.masked_fill_(hidden, -math.inf)
    w = w.sub_(w.amax(-1, keepdim=True).clamp_(min=-1e30)).exp_()     # (an empty place of the batch: no weights)
    o = torch.matmul(w, rows("v").transpose(1, 2)).div_(w.sum(-1, keepdim=True).clamp_(min=1e-30))
    return o.view(T, Hq, D).to(torch.bfloat16)


# ------------------------------------------------------------------------------------ what a pass costs

def work(case):
    if case["op"] == "quant":
        n = case["M"] * case["K"]      # read, and the codes, scales and values written
        return {"bytes": 4 * n + n // 2 + n // BLOCK[case["kind"]], "flops": 4 * n}
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        held = (M + N) * (K // 2 + K // BLOCK[case["kind"]])
        return {"bytes": held + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * M * N * K}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    row = 2 * Hkv * (D // 2 + D // 16)
    if case["op"] == "append":         # (the expanded pages hold the call's own tokens at least)
        T = case["tokens"]
        return {"bytes": T * (2 * (Hq + 2 * Hkv) * D + 2 * Hq * D + row + 4 * Hkv * D + 4 * case["rot"]),
                "flops": 8 * T * (Hq + 2 * Hkv) * D}
    keys = sum(_lengths(case))
    return {"bytes": 4 * case["tokens"] * Hq * D + keys * row, "flops": 4 * Hq * D * keys}


# ------------------------------------------------------------------------------------ in 64 bits

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nearest(x, kind, tensor):
    """The values nearest to x [..., C] (64 bits) that the format holds, by search among the eight magnitudes."""
    size = BLOCK[kind]
    x = x.reshape(*x.shape[:-1], -1, size)
    top = x.abs().amax(-1, keepdim=True)
    if kind == "mxfp4":
        unit = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -120))) - 2)
    else:
        want = (top / (6 * tensor)).clamp(max=448.0)
        step = torch.exp2(torch.floor(torch.log2(want.clamp(min=2.0 ** -6))) - 3)      # E4M3: 3 bits behind the first
        unit = torch.round(want / step) * step * tensor                               # (round: ties to even)
    y = torch.where(unit > 0, x.abs() / unit.clamp(min=2.0 ** -140), 0.0)
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    low = (torch.searchsorted(grid, y.clamp(max=6.0).contiguous(), right=True) - 1).clamp(max=6)
    down, up = grid[low], grid[low + 1]
    mid = (down + up) / 2
    code = torch.where((y > mid) | ((y == mid) & (low % 2 == 1)), up, down)
    return (torch.copysign(code, x) * unit).flatten(-2)


def _held(codes, scales, kind, tensor):
    """64-bit values of packed codes and scale bytes, element by element."""
    grid = torch.tensor(GRID + tuple(-a for a in GRID), dtype=torch.float64, device=codes.device)
    out = torch.empty((*codes.shape[:-1], 2 * codes.shape[-1]), dtype=torch.float64, device=codes.device)
    out[..., 0::2], out[..., 1::2] = grid[codes.long() % 16], grid[torch.div(codes.long(), 16, rounding_mode="floor")]
    b = scales.long()
    if kind == "mxfp4":
        s = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=b.device), b - 127)
    else:
        e, m = torch.div(b, 8, rounding_mode="floor"), (b % 8).double()
        s = torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9) * tensor
    return out * s.repeat_interleave(BLOCK[kind], -1)


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "quant":
        return _nearest(s["x"].double(), case["kind"], _tensor(case))
    if case["op"] == "product":
        def matrix(codes, tiles):
            r = torch.arange(codes.shape[0], device=codes.device)[:, None]
            c = torch.arange(4 * tiles.shape[1], device=codes.device)[None]
            return _held(codes, tiles[r // 128, c // 4, r % 32, r // 32 % 4, c % 4], case["kind"], 1.0)
        return s["alpha"] * (matrix(s["x"], s["sx"]) @ matrix(s["w"], s["sw"]).T)
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    k, v = (_held(s[a + "_codes"], s[a + "_scales"], "nvfp4", TENSOR[a]) for a in ("k", "v"))
    if case["op"] == "append":
        T, rot = case["tokens"], case["rot"]
        x = s["qkv"].double().reshape(T, Hq + 2 * Hkv, D)
        pos = s["q_pos"].long()
        z = torch.complex(s["cos_sin"][pos, :rot // 2].double(), s["cos_sin"][pos, rot // 2:].double())[:, None]

        def head(y, weight):
            if weight is not None:
                y = y * weight.double() / torch.sqrt(torch.mean(y * y, -1, keepdim=True) + EPS)
            y = y.clone()
            if case["pairs"] == "neighbours":
                w = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * z
                y[..., 0:rot:2], y[..., 1:rot:2] = w.real, w.imag
            else:
                w = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * z
                y[..., :rot // 2], y[..., rot // 2:rot] = w.real, w.imag
            return y

        where = s["table"][s["q_seq"].long(), torch.div(pos, page, rounding_mode="floor")].long(), pos % page
        # (the cache takes the keys as bf16 rows of attention: rounded there first)
        k[where] = _nearest(head(x[:, Hq:Hq + Hkv], s.get("gk")).to(torch.bfloat16).double(), "nvfp4", TENSOR["k"])
        v[where] = _nearest(x[:, Hq + Hkv:], "nvfp4", TENSOR["v"])
        return {"q": head(x[:, :Hq], s.get("gq")), "k": k, "v": v}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    G = Hq // Hkv
    for b, n in enumerate(_lengths(case)):
        if n:
            rows = s["table"][b, :-(-n // page)].long()
            keys, values = (a[rows].reshape(-1, Hkv, D)[:n].transpose(0, 1) for a in (k, v))
            z = s["q"][b].double().view(Hkv, G, D) @ keys.transpose(1, 2) / math.sqrt(D)
            out[b] = (torch.softmax(z, -1) @ values).view(Hq, D)
    return out
