"""Cases of the operators that take prompts and drafted tokens through a full-attention layer and
score what comes out: norms and rotary positions of queries and keys, attention of chunks of new
tokens over the paged cache, and log probabilities of given tokens with entropy and alternatives.

``own`` false computes each operator in plain torch operations (float32, angles in 64 bits, rounded
once); ``own`` true makes the calls a user makes of the package.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
EPS = 1e-6


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one request between projection and cache: launch latency
        dict(name="rotate-token", op="rotate", N=1, Hq=32, H=8, D=128, rot=128, x="bf16", norm=True, layout="half",
             longest=4096, stretch=1, slack=0),
        # a decode batch at far positions, a quarter of wide heads rotated, neighbouring columns paired
        dict(name="rotate-batch", op="rotate", N=256, Hq=16, H=2, D=256, rot=64, x="f16", norm=False, layout="interleaved",
             longest=1000000, stretch=8, slack=0),
        # prompts taken out of a fused projection (queries, keys and values in one row), odd number of tokens
        dict(name="rotate-prompt", op="rotate", N=32773, Hq=32, H=8, D=128, rot=128, x="bf16", norm=True, layout="half",
             longest=131072, stretch=4, slack=1024),
        # the first prompt of an idle server
        dict(name="chunk-first-prompt", op="chunk", R=1, Hq=32, H=8, D=128, new=17, past=0, page=16, kv="bf16", q="bf16", window=0),
        # drafted tokens of a decode batch verified together, ragged caches
        dict(name="chunk-drafts", op="chunk", R=64, Hq=32, H=8, D=128, new=5, past=4096, page=16, kv="bf16", q="bf16", window=0),
        # prompts of several lengths admitted beside decoding requests, 8-bit cache
        dict(name="chunk-ragged-8bit", op="chunk", R=16, Hq=32, H=4, D=128, new=1000, past=2500, page=32, kv="e4m3", q="bf16",
             window=0),
        # one whole prompt
        dict(name="chunk-prompt", op="chunk", R=1, Hq=32, H=8, D=128, new=8192, past=0, page=64, kv="bf16", q="bf16", window=0),
        # the next chunk of a long document, wide heads
        dict(name="chunk-document", op="chunk", R=1, Hq=16, H=2, D=256, new=512, past=130559, page=64, kv="f16", q="f16",
             window=0),
        # a key-value head for each query head, sliding window, small heads
        dict(name="chunk-window", op="chunk", R=4, Hq=20, H=20, D=64, new=3001, past=2000, page=128, kv="f16", q="f16",
             window=1024),
        # one generated token
        dict(name="logprobs-token", op="logprobs", N=1, V=128000, K=20, x="f32", slack=0),
        # a decode batch, logits inside rows padded to a multiple of 512
        dict(name="logprobs-batch", op="logprobs", N=256, V=64001, K=8, x="bf16", slack=511),
        # a prompt scored, odd rows
        dict(name="logprobs-prompt", op="logprobs", N=2047, V=151001, K=5, x="bf16", slack=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "chunk", "chunk", "logprobs"])
    if op == "rotate":
        D = rng.choice([64, 80, 96, 128, 192, 256])
        H = rng.choice([1, 2, 4, 5, 8])
        Hq = H * rng.choice([1, 2, 3, 4, 8])
        x = rng.choice(["bf16", "f16", "f32"])
        N = min(_log_int(rng, 1, 32768), 32773 * 40 * 128 * 2 // ((Hq + H) * D * SIZE[x]))
        return dict(op=op, N=N, Hq=Hq, H=H, D=D, rot=rng.choice([D, D, D // 2, D // 4 // 2 * 2]), x=x, norm=rng.random() < 0.6,
                    layout=rng.choice(["half", "interleaved"]), longest=_log_int(rng, 16, 1000000),
                    stretch=rng.choice([1, 1, 4, 8]), slack=rng.choice([0, 64, 1024]))
    if op == "chunk":
        D = rng.choice([64, 128, 256])
        H = rng.choice([1, 2, 4, 5, 8])
        G = rng.choice([1, 2, 3, 4, 6, 8])
        R = _log_int(rng, 1, 64)
        new = _log_int(rng, 1, 4096)
        past = rng.choice([0, _log_int(rng, 1, 100000)])
        # scores of the padded plain form and the cache's values stay below those of the largest listed cases
        new = max(1, min(new, math.isqrt(2 ** 30 // (R * G * H))))
        past = max(0, min(past, 2 ** 30 // (R * G * H * new) - new, 2 ** 27 // (R * H * D)))
        kv = rng.choice(["bf16", "f16", "e4m3"])
        return dict(op=op, R=R, Hq=G * H, H=H, D=D, new=new, past=past, page=rng.choice([8, 16, 32, 64, 128]), kv=kv,
                    q=kv if kv != "e4m3" else rng.choice(["bf16", "f16"]), window=rng.choice([0, 0, 0, max(1, (new + past) // 3)]))
    V = _log_int(rng, 100, 262144)
    x = rng.choice(["bf16", "f16", "f32"])
    N = min(_log_int(rng, 1, 2048), 2047 * 151001 // (2 * V))
    return dict(op=op, N=N, V=V, K=rng.choice([0, 1, 5, 20, 64]), x=x, slack=rng.choice([0, 0, 1, 64]))


# ---------------------------------------------------------------------------- inputs
def _lengths(R, longest):
    """Lengths up to `longest`, many short ones: the i-th at the square of its rank."""
    if R == 1:
        return [longest]
    return [round(longest * (i / (R - 1)) ** 2) for i in range(R)]


def _chunks(case):
    """(new tokens, stored tokens before them) of each request: drafts are of one length, prompts ragged."""
    R, new = case["R"], case["new"]
    news = [new] * R if new <= 8 else _lengths(R, new)
    pasts = _lengths(R, case["past"])
    return news, pasts if new <= 8 else pasts[::-1]      # (the long prompts begin, decoding requests have a past)


def _pages(n, page):
    return -(-n // page)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _cache(g, shape, kv):
    """Stored keys or values and, for the 8-bit type, a scale for each stored vector."""
    if kv != "e4m3":
        return _randn(g, *shape, dtype=TYPES[kv]), None
    codes = (_randn(g, *shape, dtype=torch.float16) * 120).clamp(-E4M3_MAX, E4M3_MAX).to(TYPES[kv])
    return codes, (0.5 + torch.rand(shape[:3], generator=g, device="cuda")) / 120


def _frequencies(rot, stretch):
    """Radians a position of each pair of columns; for contexts `stretch` times as long slow pairs (wavelengths over
    8192 positions) turn that much slower, fast ones (under 2048) as before, and those between by both."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if stretch > 1:
        t = ((8192 * f / (2 * math.pi) - 1) / 3).clamp(0, 1)
        f = f * (t + (1 - t) / stretch)
    return f.cuda()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op = case["op"]
    if op == "rotate":
        N, Hq, H, D = case["N"], case["Hq"], case["H"], case["D"]
        rows = _randn(g, N, (Hq + H) * D + case["slack"], dtype=TYPES[case["x"]])      # [queries | keys | other columns]
        s["rows"] = rows
        s["query"] = rows[:, :Hq * D].unflatten(1, (Hq, D))
        s["key"] = rows[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D))
        s["positions"] = torch.randint(0, case["longest"], (N,), generator=g, device="cuda", dtype=torch.int32)
        s["freqs"] = _frequencies(case["rot"], case["stretch"])
        s["magnitude"] = 1.0 if case["stretch"] == 1 else 0.1 * math.log(case["stretch"]) + 1
        s["q_weight"] = (1 + 0.2 * _randn(g, D)).to(TYPES[case["x"]]) if case["norm"] else None
        s["k_weight"] = (1 + 0.2 * _randn(g, D)).to(TYPES[case["x"]]) if case["norm"] else None
        s["q_out"] = torch.empty((N, Hq, D), dtype=TYPES[case["x"]], device="cuda")
        s["k_out"] = torch.empty((N, H, D), dtype=TYPES[case["x"]], device="cuda")
    elif op == "chunk":
        R, page, H, D = case["R"], case["page"], case["H"], case["D"]
        news, pasts = _chunks(case)
        perm = torch.randperm(R, generator=g, device="cuda")
        new = torch.tensor(news, dtype=torch.int32).cuda()[perm]
        lens = new + torch.tensor(pasts, dtype=torch.int32).cuda()[perm]
        s["lens"] = lens
        s["starts"] = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)]).int()
        s["N"], s["longest"] = sum(news), max(a + b for a, b in zip(news, pasts))
        wide = max(1, _pages(s["longest"], page))
        used = (lens.long() + page - 1) // page
        total = sum(_pages(a + b, page) for a, b in zip(news, pasts))
        order = torch.randperm(total + 3, generator=g, device="cuda").int()     # three pages nobody holds
        j = torch.arange(wide, device="cuda")[None, :]
        at = (torch.cumsum(used, 0) - used)[:, None] + j
        s["table"] = torch.where(j < used[:, None], order[at.clamp(max=total + 2)], -1).int().contiguous()
        s["k"], s["k_scale"] = _cache(g, (total + 3, H, page, D), case["kv"])
        s["v"], s["v_scale"] = _cache(g, (total + 3, H, page, D), case["kv"])
        s["query"] = _randn(g, s["N"], case["Hq"], D, dtype=TYPES[case["q"]])
        s["o"] = torch.empty_like(s["query"])
        s["lse"] = torch.empty((s["N"], case["Hq"]), dtype=torch.float32, device="cuda")
    else:
        N, V, K = case["N"], case["V"], case["K"]
        rows = _randn(g, N, V + case["slack"], dtype=TYPES[case["x"]])
        rows *= 3
        s["rows"] = rows
        s["logits"] = rows[:, :V]
        s["logits"][::7, ::3] = -math.inf                                 # rows whose vocabulary a grammar cuts down
        tokens = torch.randint(0, V, (N,), generator=g, device="cuda")
        s["tokens"] = torch.where(torch.arange(N, device="cuda") % 61 == 60, -1, tokens)      # a few of padding
        s["logprob"] = torch.empty(N, dtype=torch.float32, device="cuda")
        s["entropy"] = torch.empty(N, dtype=torch.float32, device="cuda")
        s["top_ids"] = torch.empty((N, min(K, V)), dtype=torch.int32, device="cuda") if K else None
        s["top_logprobs"] = torch.empty((N, min(K, V)), dtype=torch.float32, device="cuda") if K else None
    return s


# ---------------------------------------------------------------------------- plain forms
def _rotated(x, weight, cos, sin, rot, layout):
    """Rows [N, heads, D] in float32, normed where there is a weight, the first `rot` columns turned."""
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(2, keepdim=True) + EPS) * weight.float()
    part, rest = x[..., :rot], x[..., rot:]
    a, b = (part[..., :rot // 2], part[..., rot // 2:]) if layout == "half" else (part[..., 0::2], part[..., 1::2])
    c, d = a * cos - b * sin, a * sin + b * cos
    part = torch.cat([c, d], 2) if layout == "half" else torch.stack([c, d], 3).flatten(2)
    return torch.cat([part, rest], 2)


def _rotate(s):
    angle = s["positions"].double()[:, None] * s["freqs"][None, :]
    cos, sin = ((f(angle) * s["magnitude"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    return {c: _rotated(s[x].float(), s[w], cos, sin, s["rot"], s["layout"]).to(s[x].dtype)
            for c, x, w in (("q", "query", "q_weight"), ("k", "key", "k_weight"))}


def _gathered(s, name):
    """Keys or values of every request in float32, [R, H, T, D] in token order."""
    at = s["table"].clamp(min=0).long()
    x = s[name][at].float()                                     # [R, P, H, page, D]
    if s[name + "_scale"] is not None:
        x = x * s[name + "_scale"][at].unsqueeze(-1)
    return x.transpose(1, 2).reshape(at.shape[0], s["H"], -1, s["D"])


def _chunk(s):
    R, H, D, G = s["R"], s["H"], s["D"], s["Hq"] // s["H"]
    new, lens, starts = torch.diff(s["starts"].long()), s["lens"].long(), s["starts"].long()
    most = s["new"]
    i = torch.arange(most, device="cuda")[None, :]
    row = (starts[:-1, None] + i).clamp(max=s["N"] - 1)                                # [R, most]
    q = s["query"][row].float().view(R, most, H, G, D).permute(0, 2, 3, 1, 4).reshape(R, H, G * most, D)
    scores = torch.matmul(q, _gathered(s, "k").transpose(2, 3).contiguous()).view(R, H, G, most, -1)
    scores /= math.sqrt(D)
    t = torch.arange(scores.shape[4], device="cuda")[None, None, :]
    at = (lens - new)[:, None, None] + i[:, :, None]                                   # position of each new token
    seen = t <= at if not s["window"] else (t <= at) & (t > at - s["window"])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(4, keepdim=True)
    scores -= torch.where(torch.isinf(top), 0.0, top)
    e = scores.exp_()
    total = e.sum(4, keepdim=True)
    o = torch.matmul(e.view(R, H, G * most, -1), _gathered(s, "v")).view(R, H, G, most, D)
    o /= torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total)).squeeze(4)
    r, at = torch.where(i < new[:, None])                                              # in the order of the rows
    return {"o": o.permute(0, 3, 1, 2, 4)[r, at].reshape(-1, s["Hq"], D).to(s["query"].dtype),
            "lse": lse.permute(0, 3, 1, 2)[r, at].reshape(-1, s["Hq"])}


def _logprobs(s):
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    known = (s["tokens"] >= 0) & (s["tokens"] < s["V"])
    at = torch.gather(x, 1, s["tokens"].clamp(0, s["V"] - 1)[:, None])
    out = {"logprob": torch.where(known, (at - lse)[:, 0], math.nan),
           "entropy": (lse - (e * torch.where(e > 0, x, 0.0)).sum(1, keepdim=True) / total)[:, 0]}
    if s["K"]:
        # larger values first, equal ones by their column: one whole number orders both
        bits = (x + 0.0).view(torch.int32).long()
        key = torch.where(bits < 0, -2 ** 31 - bits, bits) * 2 ** 32 + (2 ** 32 - 1 - torch.arange(s["V"], device="cuda"))
        ids = 2 ** 32 - 1 - (torch.topk(key, min(s["K"], s["V"]), dim=1).values & (2 ** 32 - 1))
        out["top_ids"], out["top_logprobs"] = ids.int(), torch.gather(x, 1, ids) - lse
    return out


# ---------------------------------------------------------------------------- one pass
def run(s):
    op = s["op"]
    if not own:
        return {"rotate": _rotate, "chunk": _chunk, "logprobs": _logprobs}[op](s)
    import linear_attn_decode_amd as wb
    if op == "rotate":
        wb.qk_rotate(s["query"], s["key"], s["positions"], s["freqs"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                     interleaved=s["layout"] == "interleaved", magnitude=s["magnitude"], q_out=s["q_out"], k_out=s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "chunk":
        wb.kv_attend_chunk(s["query"], s["k"], s["v"], s["table"], s["lens"], s["starts"], s["o"], window=s["window"],
                           lse=s["lse"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"o": s["o"], "lse": s["lse"]}
    wb.token_logprobs(s["logits"], s["tokens"], s["logprob"], entropy=s["entropy"], top_ids=s["top_ids"],
                      top_logprobs=s["top_logprobs"])
    out = {"logprob": s["logprob"], "entropy": s["entropy"]}
    if s["K"]:
        out["top_ids"], out["top_logprobs"] = s["top_ids"], s["top_logprobs"]
    return out


def _pairs(case):
    """Pairs of a new token and a stored one that it sees."""
    total, w = 0, case["window"]
    for m, p in zip(*_chunks(case)):
        if not w:
            total += m * p + m * (m + 1) // 2
        else:                                                     # positions p .. p + m - 1 see min(position + 1, w)
            short = max(0, min(p + m, w) - p)                     # of them below the window's length
            total += short * p + short * (short + 1) // 2 + (m - short) * w
    return total


def work(case):
    op = case["op"]
    if op == "rotate":
        n = case["N"] * (case["Hq"] + case["H"]) * case["D"]
        return {"bytes": 2 * n * SIZE[case["x"]] + 4 * case["N"] + 4 * case["rot"], "flops": n * (7 if case["norm"] else 3)}
    if op == "chunk":
        news, pasts = _chunks(case)
        w = case["window"]
        stored = sum(m + (min(p, w - 1) if w else p) for m, p in zip(news, pasts) if m)
        vector = case["D"] * SIZE[case["kv"]] + (4 if case["kv"] == "e4m3" else 0)
        rows = sum(news) * case["Hq"]
        return {"bytes": 2 * stored * case["H"] * vector + rows * (2 * case["D"] * SIZE[case["q"]] + 4),
                "flops": 4 * _pairs(case) * case["Hq"] * case["D"]}
    return {"bytes": case["N"] * (case["V"] * SIZE[case["x"]] + 16 + 8 * min(case["K"], case["V"])), "flops": 6 * case["N"] * case["V"]}


# ---------------------------------------------------------------------------- definitions in 64 bits
def _rows_64(x, scale):
    return x.double() if scale is None else x.double() * scale.double().unsqueeze(-1)


def _exact_rotate(s):
    out = {}
    rot = s["rot"]
    at = torch.arange(rot // 2, device="cuda")
    first, second = (at, at + rot // 2) if s["layout"] == "half" else (2 * at, 2 * at + 1)
    turn = torch.polar(torch.full_like(s["freqs"], s["magnitude"]).expand(s["N"], -1), s["positions"].double()[:, None] * s["freqs"])
    for c, x, w in (("q", "query", "q_weight"), ("k", "key", "k_weight")):
        heads = []
        for h in range(s[x].shape[1]):
            y = s[x][:, h].double()
            if s[w] is not None:
                y = y / torch.sqrt((y * y).sum(1, keepdim=True) / s["D"] + EPS) * s[w].double()
            z = torch.complex(y[:, first], y[:, second]) * turn
            y[:, first], y[:, second] = z.real, z.imag
            heads.append(y)
        out[c] = torch.stack(heads, 1)
    return out


def _exact_chunk(s):
    H, D, G, page = s["H"], s["D"], s["Hq"] // s["H"], s["page"]
    o = torch.empty((s["N"], s["Hq"], D), dtype=torch.float64, device="cuda")
    lse = torch.empty((s["N"], s["Hq"]), dtype=torch.float64, device="cuda")
    starts = s["starts"].tolist()
    for r, n in enumerate(s["lens"].tolist()):
        a, b = starts[r], starts[r + 1]
        if a == b:
            continue
        t = torch.arange(n, device="cuda")
        ids, at = s["table"][r].long()[t // page], t % page
        past = n - (b - a)
        for h in range(H):
            k, v = (_rows_64(s[c][ids, h, at], None if s[c + "_scale"] is None else s[c + "_scale"][ids, h, at]) for c in "kv")
            for i in range(a, b, 2048):                            # (rows at a time: scores in 64 bits)
                q = s["query"][i:min(b, i + 2048), h * G:(h + 1) * G].double()
                x = torch.matmul(q.reshape(-1, D), k.t().contiguous()).view(q.shape[0], G, n) / math.sqrt(D)
                where = past + i - a + torch.arange(q.shape[0], device="cuda")[:, None]
                hidden = t > where if not s["window"] else (t > where) | (t <= where - s["window"])
                x.masked_fill_(hidden[:, None], -math.inf)
                total = torch.logsumexp(x, 2)
                lse[i:i + q.shape[0], h * G:(h + 1) * G] = total
                x -= total.unsqueeze(2)
                o[i:i + q.shape[0], h * G:(h + 1) * G] = torch.matmul(x.exp_().view(-1, n), v).view(-1, G, D)
    return {"o": o, "lse": lse}


def _exact_logprobs(s):
    out = {"logprob": [], "entropy": [], "top_logprobs": []}
    for i in range(0, s["N"], 256):                               # (rows at a time)
        x, token = s["logits"][i:i + 256].double(), s["tokens"][i:i + 256]
        p = x - torch.logsumexp(x, 1, keepdim=True)
        own_p = torch.gather(p, 1, token.clamp(0, s["V"] - 1)[:, None])[:, 0]
        out["logprob"].append(torch.where((token >= 0) & (token < s["V"]), own_p, math.nan))
        out["entropy"].append(-torch.special.xlogy(p.exp(), p.exp()).sum(1))
        if s["K"]:
            out["top_logprobs"].append(torch.topk(p, min(s["K"], s["V"]), dim=1).values)
    out = {c: torch.cat(x) for c, x in out.items() if x}
    if s["K"]:
        out["top_ids"] = None
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "chunk": _exact_chunk, "logprobs": _exact_logprobs}[case["op"]](s)
