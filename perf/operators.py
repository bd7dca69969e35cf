"""The operators of an adapted layer with an 8-bit base weight, as they are measured.

Three operators, each with its plain form (elementary torch operations) and the
calls a user makes of the library:

  i8       y = (s_x q_x) (s_w q_w)^T: the tokens are quantised row by row (scale
           max|x| / 127), the product runs in 8-bit integers, and each output is
           scaled by its token and its channel.  The weight is quantised already.
  adapted  the same product with the multi-LoRA delta of each token's segment,
           y += scale * B[a] (A[a] x), x unquantised.
  rope     rotary positions on the heads of q and k: pairs (j, j + rot/2) ("half")
           or (2j, 2j + 1) ("interleaved") of the first rot dimensions of a head are
           turned by pos * freq[j]; `inverse` is the gradient (the turn back).

A case is a dict of plain values; `prepare` makes its inputs from the seed alone.
"""
import math
from types import SimpleNamespace

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence decoding: a 4096 x 4096 projection of one token
        dict(name="i8_token", op="i8", n=1, d_in=4096, d_out=4096, x="bf16", y="bf16"),
        # a decode batch of 37 sequences, narrow output (grouped keys), half precision
        dict(name="i8_decode_kv", op="i8", n=37, d_in=4096, d_out=1024, x="fp16", y="fp16"),
        # a decode step of 256 requests
        dict(name="i8_decode", op="i8", n=256, d_in=4096, d_out=4096, x="bf16", y="bf16"),
        # a chunk of a long prompt through an MLP's down projection, kept in fp32
        dict(name="i8_chunk_down", op="i8", n=2011, d_in=14336, d_out=4096, x="fp32", y="fp32"),
        # 16 images of 4096 tokens in a diffusion transformer's projection
        dict(name="i8_diffusion", op="i8", n=65536, d_in=1280, d_out=1280, x="bf16", y="bf16"),
        # 32 prompts through an MLP's up projection, no adapters
        dict(name="i8_prefill_up", op="i8", n=17389, d_in=4096, d_out=14336, x="bf16", y="bf16"),
        # the same with 64 adapters of rank 64, heavy-tailed over the prompts
        dict(name="adapted_prefill_up", op="adapted", n=17389, n_seg=32, adapters=64, lo_rank=64, hi_rank=64,
             none=0, d_in=4096, d_out=14336),
        # a short mixed batch: every rank from 8 to 128, requests without an adapter,
        # requests of one token
        dict(name="adapted_mixed_kv", op="adapted", n=1535, n_seg=23, adapters=16, lo_rank=8, hi_rank=128,
             none=4, d_in=4096, d_out=1024),
        # a decode step of 256 requests at far positions, frequencies stretched by bands
        dict(name="rope_decode", op="rope", n=256, heads_q=32, heads_k=8, dim=128, rot=128, t="bf16",
             interleaved=False, fused=True, far=131072, scaling="bands", inverse=False),
        # 32 prompts, q and k as slices of one fused projection
        dict(name="rope_prefill", op="rope", n=17389, heads_q=32, heads_k=8, dim=128, rot=128, t="bf16",
             interleaved=False, fused=True, far=8192, scaling="none", inverse=False),
        # part of the head, neighbouring pairs, a stretched context
        dict(name="rope_partial", op="rope", n=2011, heads_q=20, heads_k=20, dim=80, rot=40, t="fp16",
             interleaved=True, fused=False, far=1 << 20, scaling="yarn", inverse=False),
        # the gradient of a training batch in fp32
        dict(name="rope_grad", op="rope", n=8190, heads_q=32, heads_k=8, dim=128, rot=128, t="fp32",
             interleaved=False, fused=False, far=8192, scaling="ntk", inverse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["i8", "i8", "adapted", "rope", "rope"])
    cap = 17389 * 4096 * 14336
    if op == "rope":
        dim = rng.choice([32, 64, 72, 80, 96, 128, 256])
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        rot -= rot % 2
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 2, 4])
        n = min(_log(rng, 1, 20000), 17389 * 40 * 128 // ((hq + hk) * dim))
        return dict(op="rope", n=max(n, 1), heads_q=hq, heads_k=hk, dim=dim, rot=rot,
                    t=rng.choice(["bf16", "bf16", "fp16", "fp32"]), interleaved=rng.random() < 0.5,
                    fused=rng.random() < 0.5, far=_log(rng, 1024, 1 << 20),
                    scaling=rng.choice(["none", "linear", "ntk", "bands", "yarn"]), inverse=rng.random() < 0.4)
    d_in = 8 * _log(rng, 16, 1792)
    d_out = 8 * _log(rng, 8, 1792)
    if op == "i8":
        n = max(1, min(_log(rng, 1, 65536), cap // (d_in * d_out)))
        return dict(op="i8", n=n, d_in=d_in, d_out=d_out, x=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    y=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    n = max(1, min(_log(rng, 16, 17389), cap // (d_in * d_out)))
    lo = 8 * rng.randint(1, 16)
    hi = 8 * rng.randint(lo // 8, 16)
    n_seg = rng.randint(1, max(1, min(32, n // 2)))
    return dict(op="adapted", n=n, n_seg=n_seg, adapters=rng.randint(1, 64), lo_rank=lo, hi_rank=hi,
                none=rng.randint(0, n_seg // 4), d_in=d_in, d_out=d_out)


# ----------------------------------------------------------------------- inputs
def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _weight(case, g):
    """Rows of N(0, 1/d_in) rounded to 127 steps of their own largest value."""
    d_in, d_out = case["d_in"], case["d_out"]
    W = torch.randn(d_out, d_in, generator=g, device="cuda") / math.sqrt(d_in)
    Sw = W.abs().amax(1) / 127
    Wq = torch.round(W / Sw[:, None]).clamp_(-127, 127).to(torch.int8)
    return Wq, Sw


def _tokens(n, d, t, g):
    """Activations: unit normal with a few channels ten times as large, as layers show them."""
    X = torch.randn(n, d, generator=g, device="cuda")
    X[:, torch.randperm(d, generator=g, device="cuda")[:max(1, d // 256)]] *= 10
    return X.to(TYPES[t])


def _lengths(case, seed):
    """n_seg lengths that add up to n: every seventh is a single token, the rest vary eightfold."""
    g = _gen(seed + 1, "cpu")
    n, k = case["n"], case["n_seg"]
    w = torch.rand(k, generator=g) * 7 + 1
    w[3::7] = 0
    if float(w.sum()) == 0:
        w[:] = 1
    lens = torch.ones(k, dtype=torch.int64)
    lens += ((n - k) * w / w.sum()).floor().long()
    lens[int(w.argmax())] += n - int(lens.sum())
    return lens


def _segments(case, seed):
    """Segment bounds, one adapter each (heavy-tailed, grouped as a router leaves them); -1: none."""
    g = _gen(seed + 2, "cpu")
    lens = _lengths(case, seed)
    p = 1.0 / torch.arange(1, case["adapters"] + 1, dtype=torch.float64) ** 1.1
    ad = torch.multinomial(p, case["n_seg"], replacement=True, generator=g)
    ad[:case["none"]] = -1
    ad = ad.sort().values
    off = torch.zeros(case["n_seg"] + 1, dtype=torch.int64)
    off[1:] = lens.cumsum(0)
    return off, ad


def _pool(case, seed, g):
    """Adapters packed back to back: A [r, d_in] ~ N(0, 1/d_in), B [d_out, r] ~ N(0, 1/r)."""
    c = _gen(seed + 3, "cpu")
    lo, hi = case["lo_rank"] // 8, case["hi_rank"] // 8
    rank = 8 * torch.randint(lo, hi + 1, (case["adapters"],), generator=c)
    d_in, d_out = case["d_in"], case["d_out"]
    total = int(rank.sum())
    A = (torch.randn(total * d_in, generator=g, device="cuda") / math.sqrt(d_in)).bfloat16()
    per_row = (1 / rank.double().sqrt()).float().repeat_interleave(rank * d_out).cuda()
    B = (torch.randn(total * d_out, generator=g, device="cuda") * per_row).bfloat16()
    start = torch.zeros_like(rank)
    start[1:] = rank.cumsum(0)[:-1]
    return SimpleNamespace(A=A, B=B, A_off=(start * d_in).cuda(), B_off=(start * d_out).cuda(),
                           rank=rank.int().cuda(), d_in=d_in, d_out=d_out, max_rank=int(rank.max()),
                           start=start.tolist(), ranks=rank.tolist())


SCALINGS = {  # keyword arguments of the long-context forms, as configurations carry them
    "none": dict(base=10000.0),
    "linear": dict(base=10000.0, factor=4.0),
    "ntk": dict(base=10000.0, factor=4.0),
    "bands": dict(base=500000.0, factor=8.0, low=1.0, high=4.0, original=8192),
    "yarn": dict(base=10000.0, factor=16.0, low=1.0, high=32.0, original=4096),
}


def _freqs(rot, scaling):
    """Radians per position of each pair, and the factor on the rotated values."""
    a = SCALINGS[scaling]
    j = torch.arange(rot // 2, dtype=torch.float64)
    base, m = a["base"], 1.0
    if scaling == "ntk" and rot > 2:
        base = base * a["factor"] ** (rot / (rot - 2))
    f = base ** (-2 * j / rot)
    if scaling == "linear":
        f = f / a["factor"]
    if scaling == "bands":       # short waves stay, long ones stretch, a ramp between
        turns = a["original"] * f / (2 * math.pi)
        keep = ((turns - a["low"]) / (a["high"] - a["low"])).clamp(0, 1)
        f = f * (keep + (1 - keep) / a["factor"])
    if scaling == "yarn":        # a ramp over the pair's index
        def index(turns):
            return rot * math.log(a["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo = max(math.floor(index(a["high"])), 0)
        hi = min(math.ceil(index(a["low"])), rot - 1)
        ramp = ((j - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * (1 - ramp + ramp / a["factor"])
        m = 0.1 * math.log(a["factor"]) + 1
    return f, m


def prepare(case, seed):
    g = _gen(seed)
    s = SimpleNamespace(case=case)
    if case["op"] == "rope":
        n, hq, hk, d = case["n"], case["heads_q"], case["heads_k"], case["dim"]
        t = TYPES[case["t"]]
        if case["fused"]:        # q | k | v columns of one projection's output
            qkv = torch.randn(n, (hq + 2 * hk) * d, generator=g, device="cuda").to(t)
            q, k = qkv[:, :hq * d].view(n, hq, d), qkv[:, hq * d:(hq + hk) * d].view(n, hk, d)
        else:
            q = torch.randn(n, hq, d, generator=g, device="cuda").to(t)
            k = torch.randn(n, hk, d, generator=g, device="cuda").to(t)
        s.x = [q, k]
        s.pos = torch.randint(0, case["far"], (n,), generator=g, device="cuda")
        if own:
            import adapter_gemv_sgmv_b200 as L
            f, s.m = L.lora_rope_freqs(case["rot"], scaling=case["scaling"], **SCALINGS[case["scaling"]])
            s.y = [torch.empty(v.shape, dtype=t, device="cuda") for v in s.x]
        else:
            f, s.m = _freqs(case["rot"], case["scaling"])
        s.freqs = f.cuda()
        return s
    adapted = case["op"] == "adapted"
    x, y = ("bf16", "bf16") if adapted else (case["x"], case["y"])
    s.X = _tokens(case["n"], case["d_in"], x, g)
    s.Wq, s.Sw = _weight(case, g)
    if adapted:
        s.pool = _pool(case, seed, g)
        off, ad = _segments(case, seed)
        s.off, s.ad = off.tolist(), ad.tolist()
        s.seg_off, s.seg_ad, s.scale = off.int().cuda(), ad.int().cuda(), 0.5
    if own:
        s.Q = torch.empty(case["n"], (case["d_in"] + 15) // 16 * 16, dtype=torch.int8, device="cuda")[:, :case["d_in"]]
        if case["d_in"] % 16:    # rows of 8-bit matrices start on 16-byte boundaries
            W = torch.zeros(case["d_out"], (case["d_in"] + 15) // 16 * 16, dtype=torch.int8, device="cuda")
            W[:, :case["d_in"]] = s.Wq
            s.Wq = W[:, :case["d_in"]]
        s.Sx = torch.empty(case["n"], dtype=torch.float32, device="cuda")
        s.Y = torch.empty(case["n"], case["d_out"], dtype=TYPES[y], device="cuda")
    return s


# ------------------------------------------------------------------- plain forms
def _quantised(X):
    """Whole numbers of x / (max|x| / 127), ties to even, and the scales.  64 bits: a
    quotient next to a half has to fall on its side."""
    Xd = X.double()
    top = Xd.abs().amax(1, keepdim=True)
    q = torch.round(Xd * 127 / torch.where(top > 0, top, torch.ones_like(top)))
    return q.float(), (top[:, 0].float() / 127)


def _product(q, Wq):
    """Sums of integer products: 1024 of them stay below 2**24, where fp32 is exact."""
    acc = torch.zeros(q.shape[0], Wq.shape[0], dtype=torch.float64, device=q.device)
    for k in range(0, q.shape[1], 1024):
        acc += q[:, k:k + 1024] @ Wq[:, k:k + 1024].float().t()
    return acc.float()


def _plain_product(s):
    q, Sx = _quantised(s.X)
    y = _product(q, s.Wq)
    y *= Sx[:, None]
    y *= s.Sw
    return y


def _plain_rope(s):
    c = s.case
    rot, half = c["rot"], c["rot"] // 2
    angle = s.pos.double()[:, None] * s.freqs
    cos, sin = (torch.cos(angle) * s.m).float()[:, None], (torch.sin(angle) * s.m).float()[:, None]
    if c["inverse"]:
        sin = -sin
    out = []
    for x in s.x:
        v = x.float()
        a, b = (v[..., 0:rot:2], v[..., 1:rot:2]) if c["interleaved"] else (v[..., :half], v[..., half:rot])
        y = v.clone()
        ra, rb = a * cos - b * sin, b * cos + a * sin
        if c["interleaved"]:
            y[..., 0:rot:2], y[..., 1:rot:2] = ra, rb
        else:
            y[..., :half], y[..., half:rot] = ra, rb
        out.append(y.to(x.dtype))
    return out


def run(s):
    c = s.case
    if own:
        import adapter_gemv_sgmv_b200 as L
        if c["op"] == "rope":
            L.lora_rope(s.x, s.y, s.pos, s.freqs, interleaved=c["interleaved"], mscale=s.m, inverse=c["inverse"])
            return s.y
        L.lora_quant_i8(s.X, s.Q, s.Sx)
        if c["op"] == "i8":
            L.lora_linear_i8(s.Q, s.Sx, s.Wq, s.Sw, s.Y)
        else:
            L.lora_linear_i8_sgmv(s.Q, s.Sx, s.X, s.Wq, s.Sw, s.Y, s.pool, s.seg_off, s.seg_ad, s.scale)
        return s.Y
    if c["op"] == "rope":
        return _plain_rope(s)
    y = _plain_product(s)
    if c["op"] == "i8":
        return y.to(TYPES[c["y"]])
    p = s.pool
    for k, a in enumerate(s.ad):
        if a >= 0:
            r, a0, b0 = p.ranks[a], p.start[a] * p.d_in, p.start[a] * p.d_out
            A = p.A[a0:a0 + r * p.d_in].view(r, p.d_in).float()
            B = p.B[b0:b0 + p.d_out * r].view(p.d_out, r).float()
            rows = slice(s.off[k], s.off[k + 1])
            y[rows] += s.scale * ((s.X[rows].float() @ A.t()) @ B.t())
    return y.bfloat16()


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        f, m = _freqs(case["rot"], case["scaling"])
        turn = torch.polar(torch.full((case["n"], case["rot"] // 2), m, dtype=torch.float64, device="cuda"),
                           s.pos.double()[:, None] * f.cuda() * (-1 if case["inverse"] else 1))
        out = []
        for x in s.x:
            v = x.double()
            body, rest = v[..., :case["rot"]], v[..., case["rot"]:]
            n, h = v.shape[:2]
            if case["interleaved"]:
                z = torch.view_as_complex(body.reshape(n, h, -1, 2).contiguous()) * turn[:, None]
                body = torch.view_as_real(z).reshape(n, h, -1)
            else:
                z = torch.complex(*body.reshape(n, h, 2, -1).unbind(2)) * turn[:, None]
                body = torch.cat([z.real, z.imag], -1)
            out.append(torch.cat([body, rest], -1))
        return out
    y = torch.empty(case["n"], case["d_out"], dtype=torch.float64, device="cuda")
    W = s.Wq.double().t()
    for r in range(0, case["n"], 4096):
        X = s.X[r:r + 4096].double()
        step = X.abs().max(dim=1, keepdim=True).values / 127
        q = X / step.clamp_min(1e-300)
        near = (q - q.floor() - 0.5).abs() < 1e-9          # halves go to the even neighbour
        q = torch.where(near, 2 * ((q.floor() + 1) / 2).floor(), (q + 0.5).floor())
        y[r:r + 4096] = (q @ W) * step * s.Sw.double()
    if case["op"] == "adapted":
        p = s.pool
        for k, a in enumerate(s.ad):
            if a >= 0:
                i, o, r = p.start[a], s.off[k], p.ranks[a]
                A = p.A.view(-1, p.d_in)[i:i + r].double()
                B = p.B[i * p.d_out:(i + r) * p.d_out].view(p.d_out, r).double()
                x = s.X[o:s.off[k + 1]].double()
                y[o:s.off[k + 1]] += torch.einsum("nr,or->no", torch.einsum("ni,ri->nr", x, A), B) * s.scale
    return y


# ------------------------------------------------------------------------- work
def work(case):
    n = case["n"]
    if case["op"] == "rope":
        e = n * (case["heads_q"] + case["heads_k"]) * case["dim"]
        pairs = n * (case["heads_q"] + case["heads_k"]) * case["rot"] // 2
        return dict(bytes=2 * e * BYTES[case["t"]] + 8 * n + 4 * case["rot"], flops=6 * pairs)
    d_in, d_out = case["d_in"], case["d_out"]
    x, y = ("bf16", "bf16") if case["op"] == "adapted" else (case["x"], case["y"])
    b = n * d_in * BYTES[x] + d_out * d_in + 4 * d_out + n * d_out * BYTES[y]
    f = 2 * n * d_in * d_out
    if case["op"] == "adapted":
        r = (case["lo_rank"] + case["hi_rank"]) / 2
        b += 2 * r * (d_in + d_out) * min(case["adapters"], case["n_seg"] - case["none"])
        f += 2 * r * (d_in + d_out) * n * (1 - case["none"] / case["n_seg"])
    return dict(bytes=int(b), flops=int(f))
