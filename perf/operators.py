"""The attention operators around the paged KV cache, in plain torch operations and as the
framework's own calls:

* rope    - the step between the fused projection and attention: queries and keys normalised per
            head, rotated by their positions, keys and values appended to the cache's pages;
* prompt  - causal attention of whole prompts, or of chunks of them behind a cached context,
            packed one after the other with different lengths, grouped heads;
* shared  - one decode step of requests that share a long prefix (a system prompt, samples of one
            prompt), whose pages they have in common.

Shapes: q [T, Hq, D], caches [pages, page, Hkv, D], page tables int32 [requests, pages of one].
"""
import math
import random

import torch

own = False   # True: the framework's calls; False: the plain forms

EPS = 1e-6
HEADS = ((32, 8, 128), (16, 2, 64), (16, 8, 128), (8, 1, 128), (8, 8, 64), (4, 4, 128))
PAGES = (5, 8, 12, 16, 16, 32, 64)


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one generated token of one user: latency alone
        {"name": "rope 1", "op": "rope", "tokens": 1, "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "rot": 128,
         "pairs": "halves", "norm": True, "far": 9000, "mix": 11},
        # a decode step of 64 requests
        {"name": "rope 64", "op": "rope", "tokens": 64, "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "rot": 128,
         "pairs": "halves", "norm": True, "far": 9000, "mix": 12},
        # the packed prompts of one prefill step
        {"name": "rope 8192", "op": "rope", "tokens": 8192, "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "rot": 128,
         "pairs": "halves", "norm": True, "far": 8192, "mix": 13},
        # small heads, half of each rotated in neighbouring pairs, no norms, far positions
        {"name": "rope 5001 partial", "op": "rope", "tokens": 5001, "Hq": 16, "Hkv": 2, "D": 64, "page": 32, "rot": 32,
         "pairs": "neighbours", "norm": False, "far": 120000, "mix": 14},
        # one short question: a prompt smaller than a tile
        {"name": "prompt 1x37", "op": "prompt", "seqs": 1, "shortest": 37, "longest": 37, "context": 0, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 16, "mix": 1},
        # an ordinary prefill step: prompts of all lengths packed
        {"name": "prompt 24 ragged", "op": "prompt", "seqs": 24, "shortest": 1, "longest": 2000, "context": 0, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 16, "mix": 2},
        # chunks of long documents, most of whose positions are cached already; small heads
        {"name": "prompt 3 chunks", "op": "prompt", "seqs": 3, "shortest": 200, "longest": 700, "context": 28000,
         "Hq": 16, "Hkv": 2, "D": 64, "page": 16, "mix": 3},
        # one long document from its first token
        {"name": "prompt 1x16384", "op": "prompt", "seqs": 1, "shortest": 16384, "longest": 16384, "context": 0,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "mix": 4},
        # four samples of one prompt
        {"name": "shared 1x4", "op": "shared", "groups": 1, "per_group": 4, "prefix": 2000, "tail": 300, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 16, "mix": 5},
        # a decode step of 64 users behind one long system prompt
        {"name": "shared 1x64", "op": "shared", "groups": 1, "per_group": 64, "prefix": 8192, "tail": 512, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 16, "mix": 6},
        # rollouts: sixteen prompts, sixteen samples of each, small heads
        {"name": "shared 16x16", "op": "shared", "groups": 16, "per_group": 16, "prefix": 2100, "tail": 700, "Hq": 16,
         "Hkv": 2, "D": 64, "page": 16, "mix": 7},
        # the largest step: 256 requests over one long document, long answers of their own
        {"name": "shared 1x256", "op": "shared", "groups": 1, "per_group": 256, "prefix": 16384, "tail": 1500,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "mix": 8},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    Hq, Hkv, D = rng.choice(HEADS)
    case = {"op": rng.choice(("rope", "prompt", "shared")), "Hq": Hq, "Hkv": Hkv, "D": D, "page": rng.choice(PAGES),
            "mix": rng.randrange(1 << 20)}
    if case["op"] == "rope":
        case["tokens"] = _log(rng, 1, 8192)
        case["rot"] = rng.choice((D, D, D // 2))
        case["pairs"] = rng.choice(("halves", "neighbours"))
        case["norm"] = rng.random() < 0.75
        case["far"] = _log(rng, 10000, 120000)
    elif case["op"] == "prompt":
        case["seqs"] = _log(rng, 1, 32)
        most = min(8192, 16384 // case["seqs"])
        case["longest"] = _log(rng, 1, most)
        case["shortest"] = rng.randint(1, case["longest"])
        case["context"] = rng.choice((0, 0, _log(rng, 100, 16000)))
    else:
        case["groups"] = _log(rng, 1, 16)
        case["per_group"] = _log(rng, 2, max(2, 128 // case["groups"]))
        case["prefix"] = _log(rng, 100, 12000)
        case["tail"] = _log(rng, 1, 1500)
    return case


def _lengths(case):
    """Prompt: [(tokens, context)] of each sequence, the longest given exactly."""
    r = random.Random(case["mix"])
    out = []
    for i in range(case["seqs"]):
        n = case["longest"] if i == 0 else r.randint(case["shortest"], case["longest"])
        out.append((n, r.randint(case["context"] // 2, case["context"]) if case["context"] else 0))
    r.shuffle(out)
    return out


def _tails(case):
    """Shared: each request's own tokens behind the prefix, its new one among them."""
    r = random.Random(case["mix"])
    return [r.randint(1, case["tail"]) for _ in range(case["groups"] * case["per_group"])]


# ------------------------------------------------------------------------------------ inputs

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=g.device, dtype=torch.float32).to(torch.bfloat16)


def _table(g, counts, spare=3):
    """Page tables of requests with `counts` pages each, pages handed out in a random order; -1 behind them."""
    total = sum(counts)
    order = torch.randperm(total + spare, generator=g, device=g.device).to(torch.int32)
    table = torch.full((len(counts), max(counts)), -1, dtype=torch.int32, device=g.device)
    at = 0
    for i, n in enumerate(counts):
        table[i, :n] = order[at:at + n]
        at += n
    return table, total + spare


def _int32(values, device):
    return torch.tensor(values, dtype=torch.int32, device=device)


def _inputs(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7 + 1)
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    s = {"case": case}
    if case["op"] == "rope":
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
        s["qkv"] = _normal(g, T, (Hq + 2 * Hkv) * D)
        if case["norm"]:
            s["gq"] = (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16)
            s["gk"] = (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16)
        half = case["rot"] // 2
        rate = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        angle = torch.arange(case["far"], device=dev, dtype=torch.float64)[:, None] * rate
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
    elif case["op"] == "prompt":
        seqs = _lengths(case)
        s["table"], pages = _table(g, [-(-(n + c) // page) for n, c in seqs])
        starts = [0]
        for n, _ in seqs:
            starts.append(starts[-1] + n)
        s["seqs"], s["starts"] = seqs, starts
        s["q_start"], s["q_pos0"] = _int32(starts, dev), _int32([c for _, c in seqs], dev)
        s["max_pos"] = max(n + c for n, c in seqs) - 1
        s["q"] = _normal(g, starts[-1], Hq, D)
    else:
        tails, per, prefix = _tails(case), case["per_group"], case["prefix"]
        whole = prefix // page     # pages that the whole group has in common; the rest of the prefix is copied
        B = len(tails)
        common, used = _table(g, [max(1, whole)] * case["groups"], 0)
        mine, more = _table(g, [-(-(prefix + t) // page) - whole for t in tails])
        s["table"] = torch.full((B, whole + mine.shape[1]), -1, dtype=torch.int32, device=dev)
        s["table"][:, :whole] = common[:, :whole].repeat_interleave(per, 0)
        s["table"][:, whole:] = torch.where(mine >= 0, mine + used, mine)
        pages = used + more
        s["q_seq"] = torch.arange(B, device=dev, dtype=torch.int32)
        s["q_pos"] = _int32([prefix + t - 1 for t in tails], dev)
        s["max_pos"] = prefix + max(tails) - 1
        s["group_start"] = torch.arange(0, B + 1, per, device=dev, dtype=torch.int32)
        s["group_len"] = torch.full((case["groups"],), whole * page, dtype=torch.int32, device=dev)
        s["q"] = _normal(g, B, Hq, D)
    s["k_cache"], s["v_cache"] = (_normal(g, pages, page, Hkv, D) for _ in range(2))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import invariant_bi_gemm_gb300 as bi
        heads = case["Hq"], case["Hkv"], case["D"], case["page"]
        if case["op"] == "rope":
            s["handle"] = bi.BiQkRope(*heads, rot_dim=case["rot"], eps=EPS, interleaved=case["pairs"] == "neighbours")
        elif case["op"] == "prompt":
            s["handle"] = bi.BiPromptAttention(*heads)
        else:
            s["handle"] = bi.BiAttention(*heads)
    return s


# ------------------------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if op == "rope":
        if own:
            q = s["handle"].run(s["qkv"], s.get("gq"), s.get("gk"), s["cos_sin"], s["q_seq"], s["q_pos"],
                                s["k_cache"], s["v_cache"], s["table"])
        else:
            q = _rope(s)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "prompt":
        if own:
            return s["handle"].run(s["q"], s["q_start"], s["q_pos0"], s["k_cache"], s["v_cache"], s["table"],
                                   s["max_pos"])
        return _prompt(s)
    if own:
        return s["handle"].run_shared(s["q"], s["q_seq"], s["q_pos"], s["k_cache"], s["v_cache"], s["table"],
                                      s["max_pos"], s["group_start"], s["group_len"])
    return _shared(s)


def _rope(s):
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
        co, si = cos[:, None], sin[:, None]
        a, b = a * co - b * si, b * co + a * si
        r = torch.stack((a, b), -1).flatten(-2) if c["pairs"] == "neighbours" else torch.cat((a, b), -1)
        return torch.cat((r, rest), -1).to(torch.bfloat16)

    slot = s["table"][s["q_seq"].long(), pos // page].long() * page + pos % page
    s["k_cache"].view(-1, Hkv, D)[slot] = turned(k, s.get("gk"))
    s["v_cache"].view(-1, Hkv, D)[slot] = v
    return turned(q, s.get("gq"))


def _rows(s, request, length):
    """Keys and values of one request's first positions, [Hkv, length, D] in 32 bits."""
    page = s["case"]["page"]
    at = torch.arange(length, device=s["q"].device)
    slot = s["table"][request, at // page].long() * page + at % page
    return (x.view(-1, *x.shape[2:])[slot].float().transpose(0, 1) for x in (s["k_cache"], s["v_cache"]))


def _prompt(s):
    c = s["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    out = torch.empty_like(s["q"])
    for b, (n, before) in enumerate(s["seqs"]):     # sequences of different lengths
        k, v = _rows(s, b, before + n)
        q = s["q"][s["starts"][b]:s["starts"][b + 1]].float()
        q = q.view(n, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D)
        w = torch.matmul(q, k.transpose(1, 2)).mul_(D ** -0.5).view(Hkv, Hq // Hkv, n, before + n)
        at = torch.arange(before + n, device=q.device)
        w.masked_fill_(at > at[before:, None], -math.inf)
        w = w.sub_(w.amax(-1, keepdim=True)).exp_().view(Hkv, -1, before + n)
        o = torch.matmul(w, v).div_(w.sum(-1, keepdim=True))
        out[s["starts"][b]:s["starts"][b + 1]] = o.view(Hkv, Hq // Hkv, n, D).permute(2, 0, 1, 3).reshape(n, Hq, D)
    return out


def _shared(s):
    c = s["case"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    T, L = s["q"].shape[0], s["max_pos"] + 1
    at = torch.arange(L, device=s["q"].device)
    pages = s["table"][s["q_seq"].long()][:, at // page].long().clamp_(min=0)
    slot = pages * page + at % page
    k = s["k_cache"].view(-1, Hkv, D)[slot].float().permute(0, 2, 3, 1)     # [T, Hkv, D, L]
    w = torch.matmul(s["q"].float().view(T, Hkv, Hq // Hkv, D), k).mul_(D ** -0.5)
    del k
    w.masked_fill_((at > s["q_pos"][:, None])[:, None, None], -math.inf)
    w = w.sub_(w.amax(-1, keepdim=True)).exp_()
    v = s["v_cache"].view(-1, Hkv, D)[slot].float().transpose(1, 2)
    o = torch.matmul(w, v).div_(w.sum(-1, keepdim=True))
    return o.view(T, Hq, D).to(torch.bfloat16)


# ------------------------------------------------------------------------------------ what a pass costs

def work(case):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "rope":
        T = case["tokens"]
        return {"bytes": 4 * T * (Hq + 2 * Hkv) * D + 4 * T * case["rot"], "flops": 8 * T * (Hq + Hkv) * D}
    if case["op"] == "prompt":
        seqs = _lengths(case)
        tokens, keys = sum(n for n, _ in seqs), sum(n + c for n, c in seqs)
        pairs = sum(n * c + n * (n + 1) // 2 for n, c in seqs)
    else:
        tails, prefix = _tails(case), case["prefix"]
        whole = prefix // case["page"] * case["page"]
        tokens, keys = len(tails), case["groups"] * whole + sum(prefix - whole + t for t in tails)
        pairs = sum(prefix + t for t in tails)
    return {"bytes": 4 * tokens * Hq * D + 4 * keys * Hkv * D, "flops": 4 * Hq * D * pairs}


# ------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    G = Hq // Hkv
    if case["op"] == "rope":
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

        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        where = s["table"][s["q_seq"].long(), torch.div(pos, page, rounding_mode="floor")].long(), pos % page
        kc[where] = head(x[:, Hq:Hq + Hkv], s.get("gk"))
        vc[where] = x[:, Hq + Hkv:]
        return {"q": head(x[:, :Hq], s.get("gq")), "k_cache": kc, "v_cache": vc}

    def attend(q, keys, values, last):
        """q [n, D], keys and values [L, D]; row i sees the keys 0..last[i]."""
        z = q @ keys.T / math.sqrt(D)
        z[torch.arange(len(keys), device=z.device)[None] > last[:, None]] = -math.inf
        return torch.softmax(z, 1) @ values

    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    if case["op"] == "prompt":
        spans = [(b, s["starts"][b], s["starts"][b + 1], c) for b, (_, c) in enumerate(s["seqs"])]
    else:
        last = s["q_pos"].tolist()
        spans = [(b, b, b + 1, p) for b, p in enumerate(last)]
    for b, lo, hi, first in spans:
        L = first + hi - lo
        rows = s["table"][b, :-(-L // page)].long()
        keys, values = (x[rows].reshape(-1, Hkv, D)[:L].double() for x in (s["k_cache"], s["v_cache"]))
        for h in range(Hkv):
            q = s["q"][lo:hi, h * G:(h + 1) * G].double().reshape(-1, D)
            seen = torch.arange(first, L, device=q.device).repeat_interleave(G)
            o = [attend(a, keys[:, h], values[:, h], e) for a, e in zip(q.split(8192), seen.split(8192))]
            out[lo:hi, h * G:(h + 1) * G] = torch.cat(o).view(hi - lo, G, D)
    return out
