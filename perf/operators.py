"""The attention layer of a long-context model, measured operator by operator.

The layer normalises every head's query and key and rotates them by their
position (``qk_norm_rope``, trained through ``qk_norm_rope_bwd``), attends over
a causal sliding window plus the sequence's first few tokens, which stay
visible from everywhere ("sinks": ``fwd_sinks`` for prompts and training,
``bwd_sinks`` for the gradient), and answers one token at a time from a
key/value cache under the same mask (``decode_sinks``).

``run`` computes the plain form of each in 32 bits, or, where ``own`` is true,
makes the call a user of this repository makes.  Sizes are those of this
repository's workloads (16 heads of 128, 12 of 64, 8 of 256, sequences of 512
to 16384 tokens, the window of 256) with key/value heads shared by two to
eight query heads, and ragged ones beside them.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
BASE = 10000.0


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the next token of eight sequences, each at its own far position: a
        # launch-bound call of every decoding step
        dict(name="norm-rope token", op="norm_rope", type="bf16", B=8, H=16, Hk=2, N=1, d=128,
             rot=128, interleaved=False, norm=True, packed=True, positions=32768),
        # prompts of the N = 4096 sweep point, read out of the projection's
        # output [B, N, H + 2 Hk, d] and written as attention takes them
        dict(name="norm-rope prompts", op="norm_rope", type="bf16", B=4, H=16, Hk=2, N=4096, d=128,
             rot=128, interleaved=False, norm=True, packed=True, positions=4096),
        # rotation alone, interleaved pairs over half of a 64-wide head, ragged length
        dict(name="rope partial ragged", op="norm_rope", type="fp16", B=3, H=12, Hk=12, N=1537, d=64,
             rot=32, interleaved=True, norm=False, packed=False, positions=1537),
        # the training step's gradient of the second case
        dict(name="norm-rope gradient", op="norm_rope_bwd", type="bf16", B=4, H=16, Hk=2, N=4096,
             d=128, rot=128, interleaved=False, norm=True, packed=True, positions=4096),
        # wide heads, ragged length, partly rotated
        dict(name="norm-rope gradient ragged", op="norm_rope_bwd", type="fp16", B=2, H=8, Hk=8,
             N=1000, d=256, rot=64, interleaved=True, norm=True, packed=False, positions=1000),
        # a short ragged prompt: few tiles, latency counts
        dict(name="sinks prompt short", op="fwd", type="fp16", B=2, H=12, Hk=12, N=333, d=64,
             window=64, sinks=4),
        # the sliding-window workload of the sweep (window 256) with sinks and shared key heads
        dict(name="sinks prompt window 256", op="fwd", type="bf16", B=4, H=16, Hk=2, N=4096, d=128,
             window=256, sinks=4),
        # the longest prompt of the sweep under a wide window
        dict(name="sinks prompt long", op="fwd", type="bf16", B=1, H=16, Hk=2, N=16384, d=128,
             window=4096, sinks=4),
        # training at the N = 4096 point
        dict(name="sinks gradient window 256", op="bwd", type="bf16", B=4, H=16, Hk=2, N=4096,
             d=128, window=256, sinks=4),
        # training on a long ragged sequence
        dict(name="sinks gradient long ragged", op="bwd", type="bf16", B=1, H=16, Hk=4, N=8205,
             d=128, window=2048, sinks=16),
        # one sequence's next token, short cache
        dict(name="sinks token single", op="decode", type="bf16", B=1, H=16, Hk=2, S=1024, d=128,
             len_lo=777, len_hi=777, window=511, sinks=4),
        # a full serving batch with caches of many lengths
        dict(name="sinks token batch", op="decode", type="bf16", B=64, H=16, Hk=2, S=16384, d=128,
             len_lo=100, len_hi=16384, window=8191, sinks=4),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "fwd", "bwd", "decode"])
    case = dict(op=op, type=rng.choice(["bf16", "fp16"]))
    if op in ("norm_rope", "norm_rope_bwd"):
        d = rng.choice([64, 128, 256])
        Hk = rng.choice([1, 2, 4, 8, 12])
        H = Hk * rng.choice([1, 2, 4, 8])
        B = _spread(rng, 1, 16)
        N = _spread(rng, 1, max(1, 2 ** 25 // (B * (H + Hk) * d)))
        case.update(B=B, H=H, Hk=Hk, N=N, d=d, rot=rng.choice([16, 32, d // 2, d]),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.7,
                    packed=rng.random() < 0.5, positions=max(N, rng.choice([1000, 32768])))
    elif op in ("fwd", "bwd"):
        d = rng.choice([64, 128, 256] if op == "fwd" else [64, 128])
        Hk = rng.choice([1, 2, 3, 4, 8])
        H = Hk * rng.choice([1, 2, 4])
        B = _spread(rng, 1, 4)
        most = int(math.sqrt((2 ** 31 if op == "fwd" else 2 ** 29) / (B * H)))
        N = _spread(rng, 1 if op == "fwd" else 60, min(12000, most))
        case.update(B=B, H=H, Hk=Hk, N=N, d=d, window=rng.choice([-1, _spread(rng, 1, 4096)]),
                    sinks=rng.choice([0, 1, 4, 16, 200]))
    else:
        d = rng.choice([64, 128, 256])
        Hk = rng.choice([1, 2, 4, 8])
        H = Hk * rng.choice([1, 3, 4, 8])
        B = _spread(rng, 1, 64)
        S = _spread(rng, 16, min(32768, 2 ** 27 // (B * Hk * d)))
        lo = rng.randint(0, S)
        case.update(B=B, H=H, Hk=Hk, S=S, d=d, len_lo=lo, len_hi=rng.randint(lo, S),
                    window=rng.choice([-1, _spread(rng, 1, 8192)]), sinks=rng.choice([0, 1, 4, 16]))
    return case


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """Cache lengths, evenly over [len_lo, len_hi]."""
    B, lo, hi = case["B"], case["len_lo"], case["len_hi"]
    return [hi if B == 1 else lo + (hi - lo) * b // (B - 1) for b in range(B)]


def _tables(case, device):
    """cos and sin of position x inverse frequency, in 64 bits, kept in 32."""
    rot = case["rot"]
    inv = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    a = torch.arange(case["positions"], dtype=torch.float64, device=device)[:, None] * inv
    return a.cos().float(), a.sin().float()


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    t = TYPES[case["type"]]

    def randn(*shape, dtype=t):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    B, H, Hk, d = case["B"], case["H"], case["Hk"], case["d"]
    s = dict(case)
    if case["op"] in ("norm_rope", "norm_rope_bwd"):
        N = case["N"]
        if case["packed"]:
            # the projection's output: q, k and v heads of a token side by side
            x = randn(B, N, H + 2 * Hk, d)
            s["q"], s["k"] = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hk].transpose(1, 2)
        else:
            s["q"], s["k"] = randn(B, H, N, d), randn(B, Hk, N, d)
        s["cos"], s["sin"] = _tables(case, dev)
        start = torch.randint(0, case["positions"] - N + 1, (B, 1), generator=g, device=dev)
        s["positions"] = (start + torch.arange(N, device=dev)).to(torch.int32)
        s["qw"] = (1 + 0.1 * randn(d, dtype=torch.float32)).to(t) if case["norm"] else None
        s["kw"] = (1 + 0.1 * randn(d, dtype=torch.float32)).to(t) if case["norm"] else None
        if case["op"] == "norm_rope_bwd":
            s["dq"], s["dk"] = randn(B, H, N, d), randn(B, Hk, N, d)
    elif case["op"] in ("fwd", "bwd"):
        N = case["N"]
        s["q"], s["k"], s["v"] = randn(B, H, N, d), randn(B, Hk, N, d), randn(B, Hk, N, d)
        if case["op"] == "bwd":
            # what the forward left, and the gradient that arrives
            s["o"], s["lse"] = _attend(s["q"], s["k"], s["v"], case["window"], case["sinks"])
            s["do"] = randn(B, H, N, d)
    else:
        S = case["S"]
        s["q"], s["k"], s["v"] = randn(B, H, d), randn(B, Hk, S, d), randn(B, Hk, S, d)
        order = torch.randperm(B, generator=g, device=dev)
        s["lens"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)[order]
        unwritten = torch.arange(S, device=dev) >= s["lens"][:, None]
        s["k"].masked_fill_(unwritten[:, None, :, None], 0)
        s["v"].masked_fill_(unwritten[:, None, :, None], 0)
    return s


# -------------------------------------------------------------- plain forms

def _rotate(x, cos, sin, interleaved):
    """Pairs of the first 2 x cos.shape[-1] columns turned by their angle."""
    r = cos.shape[-1]
    turned, rest = x[..., :2 * r], x[..., 2 * r:]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if interleaved else (turned[..., :r], turned[..., r:])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((turned, rest), -1)


def _norm_rope(x, w, cos, sin, interleaved):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
    return _rotate(y, cos, sin, interleaved).to(x.dtype).contiguous()


def _norm_rope_bwd(dy, x, w, cos, sin, interleaved):
    g = _rotate(dy.float(), cos, -sin, interleaved)
    if w is None:
        return g.to(x.dtype).contiguous(), None
    y = x.float()
    r = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
    n, gw = y * r, g * w.float()
    dx = r * (gw - n * (gw * n).mean(-1, keepdim=True))
    dw = (g * n).sum((0, 1, 2))
    return dx.to(x.dtype).contiguous(), dw.to(w.dtype)


def _visible(n, window, sinks, device):
    i = torch.arange(n, device=device)
    back = i[:, None] - i[None, :]
    near = back >= 0
    return near if window < 0 else near & ((back <= window) | (i[None, :] < sinks))


def _scores(q, k, window, sinks):
    """[B, Hk, G, N, N] masked scores in 32 bits."""
    B, H, N, d = q.shape
    q = q.float().view(B, k.shape[1], -1, N, d)
    s = (q @ k.float()[:, :, None].mT) * (1.0 / math.sqrt(d))
    return s.masked_fill_(~_visible(N, window, sinks, q.device), -math.inf)


def _attend(q, k, v, window, sinks):
    s = _scores(q, k, window, sinks)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p @ v.float()[:, :, None]) / l
    return o.reshape(q.shape).to(q.dtype), (m + l.log()).reshape(q.shape[:3])


def _attend_bwd(q, k, v, o, lse, do, window, sinks):
    B, H, N, d = q.shape
    Hk, scale = k.shape[1], 1.0 / math.sqrt(d)
    grouped = (B, Hk, H // Hk, N, d)
    p = _scores(q, k, window, sinks).sub_(lse.view(B, Hk, -1, N, 1)).exp_()
    do = do.float().view(grouped)
    dv = (p.mT @ do).sum(2)
    delta = (do * o.float().view(grouped)).sum(-1, keepdim=True)
    ds = (do @ v.float()[:, :, None].mT).sub_(delta).mul_(p).mul_(scale)
    dq = ds @ k.float()[:, :, None]
    dk = (ds.mT @ q.float().view(grouped)).sum(2)
    return dq.reshape(q.shape).to(q.dtype), dk.to(k.dtype), dv.to(v.dtype)


def _answer(q, k, v, lens, window, sinks):
    """One query per sequence, the last of its lens[b] cached tokens."""
    B, H, d = q.shape
    j = torch.arange(k.shape[2], device=q.device)
    last = lens[:, None] - 1
    seen = j <= last
    if window >= 0:
        seen = seen & ((j >= last - window) | (j < sinks))
    s = (q.float().view(B, k.shape[1], -1, d) @ k.float().mT) * (1.0 / math.sqrt(d))
    s = s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = (s - m.clamp(min=-1e30)).exp()
    l = p.sum(-1, keepdim=True)
    o = (p @ v.float()) / l.clamp(min=1e-30)
    return o.reshape(q.shape).to(q.dtype), (m + l.log()).reshape(B, H)


def run(s):
    if own:
        from exact_attention_154_b200 import fa
    if s["op"] == "norm_rope":
        if own:
            return fa.qk_norm_rope(s["q"], s["k"], s["cos"], s["sin"], positions=s["positions"],
                                   q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                                   interleaved=s["interleaved"])
        at = s["positions"].long()
        cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
        return (_norm_rope(s["q"], s["qw"], cos, sin, s["interleaved"]),
                _norm_rope(s["k"], s["kw"], cos, sin, s["interleaved"]))
    if s["op"] == "norm_rope_bwd":
        if own:
            return fa.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["cos"], s["sin"],
                                       positions=s["positions"], q_weight=s["qw"],
                                       k_weight=s["kw"], eps=EPS, interleaved=s["interleaved"])
        at = s["positions"].long()
        cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
        dq, dqw = _norm_rope_bwd(s["dq"], s["q"], s["qw"], cos, sin, s["interleaved"])
        dk, dkw = _norm_rope_bwd(s["dk"], s["k"], s["kw"], cos, sin, s["interleaved"])
        return dq, dk, dqw, dkw
    if s["op"] == "fwd":
        if own:
            return fa.fwd_sinks(s["q"], s["k"], s["v"], s["window"], s["sinks"])
        return _attend(s["q"], s["k"], s["v"], s["window"], s["sinks"])
    if s["op"] == "bwd":
        if own:
            return fa.bwd_sinks(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["window"],
                                s["sinks"])
        return _attend_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["window"],
                           s["sinks"])
    if own:
        return fa.decode_sinks(s["q"], s["k"], s["v"], s["lens"], s["window"], s["sinks"])
    return _answer(s["q"], s["k"], s["v"], s["lens"], s["window"], s["sinks"])


# -------------------------------------------------------------------- work

def _pairs(n, window, sinks):
    """Visible (query, key) pairs of a sequence of n tokens."""
    if window < 0:
        return n * (n + 1) // 2
    return sum(min(i + 1, window + 1) + min(sinks, max(0, i - window)) for i in range(n))


def work(case):
    B, H, Hk, d = case["B"], case["H"], case["Hk"], case["d"]
    if case["op"] in ("norm_rope", "norm_rope_bwd"):
        N, rot = case["N"], case["rot"]
        rows = B * N * (H + Hk)
        # a table row for each token at most, and each row of the table at most once
        shared = min(B * N, case["positions"]) * rot * 4 + B * N * 4 + (4 * d if case["norm"] else 0)
        if case["op"] == "norm_rope":
            return {"bytes": rows * d * 2 * 2 + shared,
                    "flops": rows * (rot * 3 + (4 * d if case["norm"] else 0))}
        reads = 3 if case["norm"] else 2  # the arriving gradient, x where it is normalised, dx
        return {"bytes": rows * d * 2 * reads + shared + (4 * d if case["norm"] else 0),
                "flops": rows * (rot * 3 + (11 * d if case["norm"] else 0))}
    if case["op"] in ("fwd", "bwd"):
        N = case["N"]
        q, kv, pairs = B * H * N * d * 2, B * Hk * N * d * 2, B * H * _pairs(N, case["window"], case["sinks"])
        if case["op"] == "fwd":
            return {"bytes": 2 * q + 2 * kv + B * H * N * 4, "flops": 4 * d * pairs}
        return {"bytes": 4 * q + 4 * kv + B * H * N * 4, "flops": 10 * d * pairs}
    w, keys = case["window"], 0
    for n in _lengths(case):
        keys += n if w < 0 else min(n, w + 1) + min(case["sinks"], max(0, n - w - 1))
    return {"bytes": keys * Hk * d * 2 * 2 + 2 * B * H * d * 2 + B * H * 4 + B * 4,
            "flops": 4 * d * H * keys}


# ----------------------------------------------------------- 64-bit results

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm_rope", "norm_rope_bwd"):
        return _exact_norm_rope(s)
    if case["op"] == "decode":
        return _exact_answer(s)
    return _exact_attention(s)


def _exact_norm_rope(s):
    """Complex multiplication by exp(i angle), and for the gradient the
    transposed Jacobian of x -> turned(w x / rms(x))."""
    rot, d = s["rot"], s["d"]
    half = torch.arange(rot // 2, device="cuda")
    first = 2 * half if s["interleaved"] else half
    second = first + 1 if s["interleaved"] else half + rot // 2
    freq = torch.exp(-math.log(BASE) * 2.0 * half.double() / rot)
    angle = s["positions"].double()[:, None, :, None] * freq
    unit = torch.polar(torch.ones_like(angle), angle)
    out, weights = [], []
    for x, w, dy in ((s["q"], s["qw"], s.get("dq")), (s["k"], s["kw"], s.get("dk"))):
        x = x.double()
        size = (x.square().sum(-1, keepdim=True) / d + EPS).sqrt()
        w64 = None if w is None else w.double()
        y = (x if w is None else w64 * x / size) if dy is None else dy.double()
        z = torch.complex(y[..., first], y[..., second]) * (unit if dy is None else unit.conj())
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        if dy is not None and w is not None:
            weights.append((y * x / size).sum((0, 1, 2)))
            c = (y * w64 * x).sum(-1, keepdim=True)
            y = y * w64 / size - x * c / (d * size ** 3)
        elif dy is not None:
            weights.append(None)
        out.append(y)
    return tuple(out + weights)


def _exact_attention(s):
    """Softmax and its gradient, one key/value head and a band of query rows
    at a time, over the keys of the definition."""
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    B, H, N, d = q.shape
    Hk, scale, W, A = k.shape[1], d ** -0.5, s["window"], s["sinks"]
    grad = s["op"] == "bwd"
    o, lse = torch.empty_like(q), q.new_empty(B, H, N)
    if grad:
        do = s["do"].double()
        dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b in range(B):
        for h in range(H):
            c = h * Hk // H
            for r in range(0, N, 2048):
                rows = torch.arange(r, min(N, r + 2048), device=q.device)[:, None]
                keys = torch.arange(int(rows[-1]) + 1, device=q.device)[None, :]
                hidden = keys > rows
                if W >= 0:
                    hidden |= (keys < rows - W) & (keys >= A)
                n = keys.shape[1]
                x = torch.einsum("id,jd->ij", q[b, h, rows[:, 0]], k[b, c, :n]) * scale
                x[hidden] = -math.inf
                lse[b, h, rows[:, 0]] = z = torch.logsumexp(x, 1)
                p = torch.exp(x - z[:, None])
                o[b, h, rows[:, 0]] = y = torch.einsum("ij,jd->id", p, v[b, c, :n])
                if grad:
                    e = do[b, h, rows[:, 0]]
                    dv[b, c, :n] += torch.einsum("ij,id->jd", p, e)
                    t = p * (torch.einsum("id,jd->ij", e, v[b, c, :n]) - (e * y).sum(1)[:, None])
                    dq[b, h, rows[:, 0]] = torch.einsum("ij,jd->id", t, k[b, c, :n]) * scale
                    dk[b, c, :n] += torch.einsum("ij,id->jd", t, q[b, h, rows[:, 0]]) * scale
    return (dq, dk, dv) if grad else (o, lse)


def _exact_answer(s):
    q = s["q"].double()
    B, H, d = q.shape
    Hk, W, A = s["k"].shape[1], s["window"], s["sinks"]
    o, lse = torch.zeros_like(q), q.new_full((B, H), -math.inf)
    for b, n in enumerate(s["lens"].tolist()):
        j = torch.arange(n, device=q.device)
        if W >= 0:
            j = j[(j < A) | (j > n - 2 - W)]
        if n == 0:
            continue
        for c in range(Hk):
            heads = slice(c * H // Hk, (c + 1) * H // Hk)
            x = q[b, heads] @ s["k"][b, c, j].double().T / math.sqrt(d)
            lse[b, heads] = torch.logsumexp(x, -1)
            o[b, heads] = torch.softmax(x, -1) @ s["v"][b, c, j].double()
    return o, lse
