"""Cases of the operators of an attention block beside the Gaussians: layer norm, cross attention between
Gaussians and the tokens of their views (or the other way round), and dropout whose mask is drawn from a counter.

With own = False `run` computes them from elementary torch operations in float32; with own = True it makes
the framework's calls.

A case's "op":
  norm       y = (x - mean) / sqrt(var + eps) w + b of every row
  norm back  dx, dw, db of that from dy
  attn       softmax(scale q k^T) v of every batch item and head
  attn train the same, then dq, dk and dv from the output's gradient
  drop       x keep / (1 - p) + residual, with keep from (seed, offset, row, column)
  drop back  dy keep / (1 - p) with the same keep
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5

# No listed or drawn case asks more than the largest listed ones of its kind: bytes of the row-wise operators, products
# and scores of attention (a training pass weighs three times).
MOST_BYTES, MOST_FLOPS, MOST_SCORES = 1.6e9, 4.3e11, 8.3e8


def rowwise(name, op, rows, n, dtype, affine=True, residual=False, p=0.1, pad=0):
    return {"name": name, "op": op, "rows": rows, "n": n, "dtype": dtype, "affine": affine, "residual": residual,
            "p": p, "pad": pad}


def attention(name, op, batch, nq, nk, heads, kv_heads, d, dtype, ragged=False, seen=1.0, packed=False):
    return {"name": name, "op": op, "batch": batch, "nq": nq, "nk": nk, "heads": heads, "kv_heads": kv_heads, "d": d,
            "dtype": dtype, "ragged": ragged, "seen": seen, "packed": packed}


def listed():
    return [
        # the features of the 1M-Gaussian scene before their attention
        rowwise("norm 1M", "norm", 1_000_000, 128, "bf16"),
        # one row: an appearance code, latency
        rowwise("norm one view", "norm", 1, 512, "f32"),
        # the backward over the 100k-Gaussian scene, an odd width in float32
        rowwise("norm 100k back", "norm back", 100_000, 333, "f32"),
        # the 1M-Gaussian scene's backward; features are columns of a wider buffer
        rowwise("norm 1M back", "norm back", 1_000_000, 128, "f16", pad=64),
        # one view's code reads the scene's tokens while rendering: latency
        attention("one view", "attn", 1, 1, 256, 8, 8, 64, "bf16"),
        # every Gaussian of the 1M scene reads 64 appearance tokens; keys and values from one projection
        attention("1M read 64", "attn", 1, 1_000_000, 64, 4, 4, 32, "f16", packed=True),
        # 100k Gaussians read 8 views of 128 tokens, two heads of keys for eight of queries
        attention("100k read 1024", "attn", 1, 100_000, 1024, 8, 2, 64, "bf16"),
        # eight view codes gather over the Gaussians of the 1M scene that they see
        attention("8 read 1M", "attn", 1, 8, 1_000_000, 8, 8, 32, "bf16", seen=0.7),
        # a batch of scenes of unlike sizes, trained in float32, an odd head
        attention("ragged train", "attn train", 4, 5_003, 333, 4, 4, 40, "f32", ragged=True),
        # 65536 Gaussians of a scene read 1024 tokens, trained
        attention("64k read 1024 train", "attn train", 1, 65_536, 1024, 4, 4, 128, "bf16"),
        # the attention's output dropped into the residual stream, the 1M-Gaussian scene
        rowwise("drop 1M", "drop", 1_000_000, 128, "bf16", residual=True),
        # the backward of a wide hidden layer's dropout, odd rows
        rowwise("drop 100k back", "drop back", 100_000, 509, "f32", p=0.25),
    ]


def spread(rng, low, high):
    """A whole number from low to high, even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("norm", "norm back", "attn", "attn", "attn train", "attn train", "drop", "drop back"))
    dtype = rng.choice(("f32", "f16", "bf16"))
    if not op.startswith("attn"):
        c = rowwise("", op, rng.choice((rng.randint(1, 8), spread(rng, 1, 3_000_000), spread(rng, 20_000, 3_000_000))),
                    spread(rng, 3, 4096), dtype, rng.random() < 0.8, op == "drop" and rng.random() < 0.6,
                    rng.choice((0.05, 0.1, 0.25, 0.5)), rng.choice((0, 0, 1, 8, 13, 64)))
        over = work(c)["bytes"] / MOST_BYTES
        if over > 1:
            c["rows"] = max(1, int(c["rows"] / over * 0.98))
        return {k: v for k, v in c.items() if k != "name"}
    kv_heads = rng.choice((1, 2, 4, 8))
    d = rng.choice((32, 64, 128, 8 * rng.randint(1, 16), rng.randint(5, 160), spread(rng, 16, 256)))
    # Gaussians read tokens, view codes gather over Gaussians, sets of like sizes
    few, many = rng.choice((rng.randint(1, 16), spread(rng, 1, 4096))), spread(rng, 500, 1_000_000)
    nq, nk = rng.choice(((few, many), (many, few), (many, few), (spread(rng, 1, 20_000), spread(rng, 1, 20_000))))
    c = attention("", op, rng.choice((1, 1, 2, rng.randint(2, 8))), nq, nk, kv_heads * rng.choice((1, 1, 2, 4)),
                  kv_heads, d, dtype, rng.random() < 0.3, rng.choice((1.0, 1.0, 0.8, 0.4)), rng.random() < 0.5)
    for _ in range(60):
        if cost(c) <= 1:
            break
        longest = "nq" if c["nq"] >= c["nk"] else "nk"
        c[longest] = max(1, int(c[longest] * max(0.5, min(0.95, 1 / cost(c)))))
    return {k: v for k, v in c.items() if k != "name"}


def cost(c):
    w, scores = work(c), c["batch"] * c["heads"] * c["nq"] * c["nk"]
    return max(w["bytes"] / MOST_BYTES, w["flops"] / MOST_FLOPS,
               scores * (3 if c["op"] == "attn train" else 1) / MOST_SCORES)


def work(c):
    size = TYPES[c["dtype"]].itemsize
    if not c["op"].startswith("attn"):
        cells = c["rows"] * c["n"]
        if c["op"] == "norm":
            return {"bytes": size * (2 * cells + 2 * c["n"] * c["affine"]), "flops": 7 * cells}
        if c["op"] == "norm back":
            return {"bytes": size * (3 * cells + 3 * c["n"] * c["affine"]), "flops": 15 * cells}
        return {"bytes": size * cells * (2 + c["residual"]), "flops": 2 * cells}
    q, kv = (c["batch"] * n * h * c["d"] for n, h in ((c["nq"], c["heads"]), (c["nk"], c["kv_heads"])))
    products = 2 * c["nk"] * q
    if c["op"] == "attn":
        return {"bytes": size * (2 * q + 2 * kv), "flops": 2 * products}
    # q, k, v and dout read, out, dq, dk and dv written; the weights themselves are too large to keep, but
    # the four products of the backward have no other way
    return {"bytes": size * (4 * q + 4 * kv), "flops": 6 * products}


def normal(gen, shape, scale, dtype):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t = TYPES[c["dtype"]]
    if not c["op"].startswith("attn"):
        rows, n = c["rows"], c["n"]
        s = {"c": c, "x": normal(gen, (rows, n + c["pad"]), 1.0, t)[:, c["pad"]:]}
        if c["op"].startswith("norm"):
            # features with a mean of their own and channels of unlike size
            s["x"] += normal(gen, (rows, 1), 0.5, t)
            s["x"] *= 0.5 + torch.rand(n, generator=gen, device="cuda").to(t)
            s["w"] = 1 + normal(gen, (n,), 0.2, t) if c["affine"] else None
            s["b"] = normal(gen, (n,), 0.2, t) if c["affine"] else None
            s["dy"] = normal(gen, (rows, n), 0.1, t) if c["op"] == "norm back" else None
        else:
            s["residual"] = normal(gen, (rows, n), 1.0, t) if c["residual"] else None
            s["seed"], s["offset"] = (int(torch.randint(1 << 62, (1,), generator=gen, device="cuda")) for _ in range(2))
        return s
    batch, nq, nk, heads, kv_heads, d = (c[k] for k in ("batch", "nq", "nk", "heads", "kv_heads", "d"))
    s = {"c": c, "q": normal(gen, (batch, nq, heads, d), 1.0, t), "mask": None, "q_lengths": None, "k_lengths": None}
    if c["packed"]:
        kv = normal(gen, (batch, nk, 2, kv_heads, d), 1.0, t)
        s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
    else:
        s["k"], s["v"] = (normal(gen, (batch, nk, kv_heads, d), 1.0, t) for _ in range(2))
    s["k"] *= 1.5
    if c["seen"] < 1:
        s["mask"] = torch.rand((batch, nk), generator=gen, device="cuda") < c["seen"]
    if c["ragged"]:
        for key, n in (("q_lengths", nq), ("k_lengths", nk)):
            part = torch.rand(batch, generator=gen, device="cuda").clamp(min=0.25)
            part[0] = 1.0
            s[key] = (part * n).ceil().to(torch.int32)
    if c["op"] == "attn train":
        s["dout"] = normal(gen, (batch, nq, heads, d), 0.2, t)
    return s


# The plain forms: elementary operations in float32, rounded once.

def plain_moments(s):
    x = s["x"].float()
    centred = x - x.mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt((centred * centred).mean(1, keepdim=True) + EPS)
    return centred * rstd, rstd


def plain_norm(s):
    y, _ = plain_moments(s)
    if s["w"] is not None:
        y = y * s["w"].float() + s["b"].float()
    return y.to(s["x"].dtype)


def plain_norm_back(s):
    xh, rstd = plain_moments(s)
    dy = s["dy"].float()
    g = dy if s["w"] is None else dy * s["w"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    got = {"dx": dx}
    if s["w"] is not None:
        got["dw"], got["db"] = (dy * xh).sum(0), dy.sum(0)
    return {k: v.to(s["x"].dtype) for k, v in got.items()}


def plain_allowed(s):
    """[batch, 1, 1, nk] and [batch, 1, nq, 1]: the keys and queries that count; None where all do."""
    nq, nk, device = s["q"].shape[1], s["k"].shape[1], s["q"].device
    keys, queries = s["mask"], None
    if s["k_lengths"] is not None:
        inside = torch.arange(nk, device=device) < s["k_lengths"][:, None]
        keys = inside if keys is None else keys & inside
    if s["q_lengths"] is not None:
        queries = (torch.arange(nq, device=device) < s["q_lengths"][:, None])[:, None, :, None]
    return None if keys is None else keys[:, None, None], queries


def by_head(t, heads):
    """[batch, n, h, d] as float32 [batch, heads, n, d]: a head of keys for each head of queries."""
    t = t.float().transpose(1, 2)
    group = heads // t.shape[1]
    return t.repeat_interleave(group, 1) if group > 1 else t.contiguous()


def plain_attn(s):
    c, train = s["c"], s["c"]["op"] == "attn train"
    heads, scale = c["heads"], 1.0 / math.sqrt(c["d"])
    q, k, v = (by_head(s[n], heads) for n in ("q", "k", "v"))
    scores = torch.matmul(q * scale, k.transpose(2, 3).contiguous())
    keys, queries = plain_allowed(s)
    if keys is not None:
        scores = scores.masked_fill(~keys, -math.inf)
        v = v.masked_fill(~keys.transpose(2, 3), 0.0)
    peak = scores.amax(3, keepdim=True).clamp(min=-3e38)
    p = torch.exp(scores - peak)
    total = p.sum(3, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    if queries is not None:
        p = p * queries
    t = s["q"].dtype
    got = {"out": torch.matmul(p, v).transpose(1, 2).to(t).contiguous()}
    if not train:
        return got
    dout = by_head(s["dout"], heads)
    ds = torch.matmul(dout, v.transpose(2, 3).contiguous())
    ds = p * (ds - (p * ds).sum(3, keepdim=True)) * scale
    got["dq"] = torch.matmul(ds, k).transpose(1, 2).to(t).contiguous()
    for name, weights, rows in (("dk", ds, q), ("dv", p, dout)):
        g = torch.matmul(weights.transpose(2, 3).contiguous(), rows)
        g = g.view(g.shape[0], c["kv_heads"], -1, g.shape[2], g.shape[3]).sum(2)
        got[name] = g.transpose(1, 2).to(t).contiguous()
    return got


def low_high(a, b):
    """Low and high 32 bits of the product of a 32-bit constant and 32-bit numbers held in int64."""
    a_low, a_high = a & 0xFFFF, a >> 16
    b_low, b_high = b & 0xFFFF, b >> 16
    low = a_low * b_low
    mid = a_high * b_low + (low >> 16)
    cross = a_low * b_high + (mid & 0xFFFF)
    return ((cross & 0xFFFF) << 16) | (low & 0xFFFF), a_high * b_high + (mid >> 16) + (cross >> 16)


def plain_keep(s):
    """[rows, n] of keep, and the factor 1 / (1 - p): ten rounds of Philox4x32 (Salmon, Moraes, Dror and Shaw,
    "Parallel random numbers: as easy as 1, 2, 3", 2011) of the counter (column / 8, row, offset), keyed by the seed;
    a column takes 16 of the 128 bits."""
    c, device = s["c"], s["x"].device
    blocks = (c["n"] + 7) // 8
    x0 = torch.arange(blocks, device=device)[None].expand(c["rows"], blocks)
    x1 = torch.arange(c["rows"], device=device)[:, None].expand(c["rows"], blocks)
    x2, x3 = (torch.full_like(x0, w) for w in (s["offset"] & 0xFFFFFFFF, s["offset"] >> 32))
    k0, k1 = s["seed"] & 0xFFFFFFFF, s["seed"] >> 32
    for _ in range(10):
        low0, high0 = low_high(0xD2511F53, x0)
        low1, high1 = low_high(0xCD9E8D57, x2)
        x0, x1, x2, x3 = high1 ^ x1 ^ k0, low1, high0 ^ x3 ^ k1, low0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack([h for w in (x0, x1, x2, x3) for h in (w & 0xFFFF, w >> 16)], 2)
    threshold = round(c["p"] * 65536)
    return words.view(c["rows"], -1)[:, :c["n"]] >= threshold, 65536.0 / (65536 - threshold)


def plain_drop(s):
    keep, factor = plain_keep(s)
    y = torch.where(keep, s["x"].float() * factor, 0.0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


# The framework's calls.

def own_run(s):
    from differentiable_gaussian_splatting_dgs_amd import network
    c = s["c"]
    if c["op"] == "norm":
        return network.layer_norm(s["x"], s["w"], s["b"], eps=EPS)
    if c["op"] == "norm back":
        dx, dw, db = network.layer_norm_backward(s["dy"], s["x"], s["w"], s["b"], eps=EPS)
        return {"dx": dx} if dw is None else {"dx": dx, "dw": dw, "db": db}
    if c["op"] == "drop":
        return network.dropout(s["x"], c["p"], s["seed"], s["offset"], residual=s["residual"])
    if c["op"] == "drop back":
        return network.dropout_backward(s["x"], c["p"], s["seed"], s["offset"])
    inputs = s["q"], s["k"], s["v"]
    valid = {k: s[k] for k in ("mask", "q_lengths", "k_lengths")}
    if c["op"] == "attn":
        return {"out": network.cross_attention(*inputs, **valid)}
    out, lse = network.cross_attention_forward(*inputs, **valid)
    dq, dk, dv = network.cross_attention_backward(s["dout"], *inputs, out, lse, **valid)
    return {"out": out, "dq": dq, "dk": dk, "dv": dv}


PLAIN = {"norm": plain_norm, "norm back": plain_norm_back, "attn": plain_attn, "attn train": plain_attn,
         "drop": plain_drop, "drop back": plain_drop}


def run(s):
    return own_run(s) if own else PLAIN[s["c"]["op"]](s)


# The definition in 64 bits.

def exact_norm(s, back):
    x = s["x"].double()
    n = x.shape[1]
    w = torch.ones_like(x[0]) if s["w"] is None else s["w"].double()
    d = x - (x.sum(1) / n)[:, None]
    sigma = torch.sqrt(d.square().sum(1) / n + EPS)[:, None]
    if not back:
        return d / sigma * w if s["b"] is None else torch.addcmul(s["b"].double(), d / sigma, w)
    dy = s["dy"].double()
    g = dy * w
    along = (g * d).sum(1, keepdim=True) / (n * sigma * sigma)
    answer = {"dx": (g - g.sum(1, keepdim=True) / n - d * along) / sigma}
    if s["w"] is not None:
        answer["dw"], answer["db"] = (dy * d / sigma).sum(0), dy.sum(0)
    return answer


def exact_attn(c, s):
    """A batch item and a head at a time, from the rows and keys that count, in slices of the queries."""
    batch, nq, heads, d = s["q"].shape
    train, group = c["op"] == "attn train", heads // c["kv_heads"]
    zeros = {k: torch.zeros(s[v].shape, dtype=torch.float64, device="cuda")
             for k, v in (("out", "q"), ("dq", "q"), ("dk", "k"), ("dv", "v")) if train or k == "out"}
    for b in range(batch):
        count = nq if s["q_lengths"] is None else int(s["q_lengths"][b])
        last = s["k"].shape[1] if s["k_lengths"] is None else int(s["k_lengths"][b])
        which = torch.arange(last, device="cuda")
        if s["mask"] is not None:
            which = which[s["mask"][b, :last]]
        if which.numel() == 0:
            continue
        step = max(1, 100_000_000 // which.numel())
        for h in range(heads):
            k, v = (s[n][b, which, h // group].double() for n in ("k", "v"))
            for i in range(0, count, step):
                rows = slice(i, min(i + step, count))
                q = s["q"][b, rows, h].double()
                z = (q @ k.t().contiguous()).mul_(d ** -0.5)
                norm = torch.logsumexp(z, 1)
                weights = z.sub_(norm[:, None]).exp_()
                out = weights @ v
                zeros["out"][b, rows, h] = out
                if train:
                    g = s["dout"][b, rows, h].double()
                    zeros["dv"][b, :, h // group].index_add_(0, which, weights.t().contiguous() @ g)
                    dz = (g @ v.t().contiguous()).sub_((g * out).sum(1)[:, None]).mul_(weights).mul_(d ** -0.5)
                    zeros["dq"][b, rows, h] = dz @ k
                    zeros["dk"][b, :, h // group].index_add_(0, which, dz.t().contiguous() @ q)
    return {k: zeros[k] for k in ("out", "dq", "dk", "dv") if k in zeros}


def exact_drop(c, s):
    """The generator's state as one [rows, blocks, 4] tensor; products wrap in 64 bits, which leaves both halves."""
    low = 0xFFFFFFFF
    blocks = -(-c["n"] // 8)
    state = torch.empty(c["rows"], blocks, 4, dtype=torch.int64, device="cuda")
    state[..., 0], state[..., 1] = torch.arange(blocks, device="cuda"), torch.arange(c["rows"], device="cuda")[:, None]
    state[..., 2], state[..., 3] = s["offset"] % 2 ** 32, s["offset"] // 2 ** 32
    multiply = torch.tensor([0xD2511F53, 0xCD9E8D57], device="cuda")
    for i in range(10):
        key = [(k + i * step) & low for k, step in zip((s["seed"] & low, s["seed"] >> 32), (0x9E3779B9, 0xBB67AE85))]
        product = state[..., ::2] * multiply
        high = (product >> 32 & low).flip(-1) ^ state[..., 1::2] ^ torch.tensor(key, device="cuda")
        state = torch.stack([high, (product & low).flip(-1)], 3).flatten(2)
    drawn = torch.stack([state & 0xFFFF, state >> 16], 3).flatten(1)[:, :c["n"]]
    least = round(c["p"] * 2 ** 16)
    y = s["x"].double() * (drawn >= least) / (1 - least / 2 ** 16)
    return y if s["residual"] is None else y + s["residual"].double()


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"].startswith("norm"):
        return exact_norm(s, c["op"] == "norm back")
    if c["op"].startswith("attn"):
        return exact_attn(c, s)
    return exact_drop(c, s)
