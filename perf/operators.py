"""Latent attention over the paged pool: the operators' plain forms, and the framework's calls.

A latent cache holds one row a token, shared by every head: a latent vector c of R values
and a position key r of P values.  Three operators work on it.

  write     c' = c * rsqrt(mean(c^2) + eps) * w and r' = the pairs of r turned by the token's
            angles, stored at the token's block and slot; the heads' position queries are
            turned by the same angles.
  absorbed  out[i, h] = sum_t p[i, h, t] c_t with p = softmax_t(scale * (ql[i, h] . c_t +
            qr[i, h] . r_t)): the queries were multiplied by the key projection before the
            call, so every head reads the latent rows themselves.
  expanded  k[t, h] = (Wk[h] c_t, r_t), v[t, h] = Wv[h] c_t and ordinary attention over them.

Query i of a sequence's n_q newest tokens sees the tokens [0, len - n_q + i].
"""
import math
import random

import torch

own = False

BLOCK = 32   # tokens a block
D = 128      # values of a head's expanded key (without its position part) and value
P = 64       # values of the position key
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _write(name, n, heads, latent, interleaved, norm=True):
    return dict(name=name, op="write", tokens=n, heads=heads, latent=latent, interleaved=interleaved, norm=norm)


def _attend(op, name, batch, n_q, heads, latent, lo, hi):
    """Sequence lengths are spread over [lo, hi] by the case alone; the last one is hi."""
    return dict(name=name, op=op, batch=batch, n_q=n_q, heads=heads, latent=latent, lo=lo, hi=hi)


def listed():
    return [
        # one decode step of a few sequences: the write's latency
        _write("write a step of 8", 8, 16, 512, True),
        # the prompts of one scheduler step, an odd number of tokens, rotation by halves
        _write("write 4999 prompt tokens", 4999, 16, 512, False),
        # a long prompt at the full head count, where the position queries are most of the bytes
        _write("write 16384 tokens 128 heads", 16384, 128, 512, True),
        # a single short conversation: the decode call's latency
        _attend("absorbed", "decode 1 x 1000", 1, 1, 16, 512, 1000, 1000),
        # a ragged batch on a few heads of each device, one sequence of it empty
        _attend("absorbed", "decode 64 ragged 16 heads", 64, 1, 16, 512, 0, 8192),
        # every head on one device
        _attend("absorbed", "decode 8 x 4096 128 heads", 8, 1, 128, 512, 4096, 4096),
        # long contexts
        _attend("absorbed", "decode 16 x 16384 32 heads", 16, 1, 32, 512, 16384, 16384),
        # drafted tokens checked together, the narrower latent
        _attend("absorbed", "verify 4 drafted x 33", 33, 4, 16, 256, 100, 4096),
        # a short prompt: the prefill call's latency
        _attend("expanded", "prompt of 100", 1, 100, 4, 512, 100, 100),
        # a chunk of 1000 new tokens behind contexts of different lengths
        _attend("expanded", "chunk of 1000 x 4 ragged", 4, 1000, 16, 512, 1000, 4096),
        # a whole prompt
        _attend("expanded", "prompt of 4096 32 heads", 1, 4096, 32, 512, 4096, 4096),
        # the longest prompt
        _attend("expanded", "prompt of 8192 16 heads", 1, 8192, 16, 512, 8192, 8192),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("write", "absorbed", "absorbed", "expanded"))
    latent = rng.choice((256, 512, 512))
    heads = rng.choice((1, 2, 3, 5, 8, 12, 16, 20, 32, 40, 64, 96, 128))
    if op == "write":
        n = _spread(rng, 1, 16384)
        return dict(op=op, tokens=n, heads=heads, latent=latent, interleaved=rng.random() < 0.5, norm=rng.random() < 0.8)
    if op == "absorbed":
        n_q = rng.choice((1, 1, 1, 2, 3, 4, 7, 8))
        hi = _spread(rng, n_q, 16384)
        batch = _spread(rng, 1, max(1, min(128, 262144 // hi, 32768 // (heads * n_q))))
        return dict(op=op, batch=batch, n_q=n_q, heads=heads, latent=latent, lo=rng.choice((n_q, max(n_q, hi // 2), hi)), hi=hi)
    hi = _spread(rng, 16, 8192)
    n_q = _spread(rng, 1, hi)
    heads = min(heads, 32)
    batch = _spread(rng, 1, max(1, min(16, (1 << 29) // (heads * n_q * hi), 32768 // hi)))
    return dict(op=op, batch=batch, n_q=n_q, heads=heads, latent=latent, lo=rng.choice((n_q, max(n_q, hi // 2), hi)), hi=hi)


def _lens(case):
    rng = random.Random(case["batch"] * 7919 + case["hi"])
    lens = [rng.randint(max(case["lo"], case["n_q"]), case["hi"]) for _ in range(case["batch"])]
    lens[-1] = case["hi"]
    if case["lo"] == 0:
        lens[0] = 0
    return lens


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _tables(positions):
    """cos and sin of every position's P / 2 angles, the angles taken in 64 bits."""
    freq = 10000.0 ** (-torch.arange(P // 2, dtype=torch.float64, device="cuda") / (P // 2))
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat((a.cos(), a.sin()), 1).float()


def _pool(latent, blocks, cache=None):
    """A one-layer latent pool; with `cache` its only slab is that tensor's memory."""
    import paged_kv_cache_split_gb300 as pkv
    if cache is None:
        pool = pkv.Pool(1, 1, latent, "latent", rope_dim=P, max_slabs=blocks // 32 + 1)
    else:
        alloc = pkv.Allocator(pkv.ALLOC_FN(lambda ctx, n, stream: cache.data_ptr()),
                              pkv.RELEASE_FN(lambda ctx, ptr, stream: None), None)
        pool = pkv.Pool(1, 1, latent, "latent", rope_dim=P, slab_blocks=blocks, max_slabs=1, allocator=alloc)
    pool.reserve_rows(blocks)
    return pool


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda").bfloat16()  # noqa: E731
    R, W, H = case["latent"], case["latent"] + P, case["heads"]
    if case["op"] == "write":
        n = case["tokens"]
        blocks = -(-n // BLOCK) + 1
        # a little behind the data: the pool keeps its copy descriptors there
        memory = torch.zeros(blocks * BLOCK * W + 4096, dtype=torch.bfloat16, device="cuda")
        pool = _pool(R, blocks, memory) if own else None
        cache = memory[:blocks * BLOCK * W].view(blocks, BLOCK, W)
        cache.copy_(normal(blocks, BLOCK, W))
        place = torch.randperm(blocks * BLOCK, generator=g, device="cuda")[:n].int()  # tokens of many sequences
        q = normal(n, H, D + P)
        return dict(case=case, pool=pool, memory=memory, cache=cache, rows=place // BLOCK, slots=place % BLOCK,
                    kv=normal(n, W) * 3, weight=1 + 0.1 * normal(R) if case["norm"] else None,
                    positions=torch.randint(0, 131072, (n,), generator=g, device="cuda").int(), tables=_tables(131072),
                    q=q[..., D:], q_out=torch.empty(n, H, P, dtype=torch.bfloat16, device="cuda"))
    lens, n_q, B = _lens(case), case["n_q"], case["batch"]
    need = [-(-x // BLOCK) for x in lens]
    blocks, width = sum(need), max(need)
    cache = normal(blocks, BLOCK, W)
    order = torch.randperm(blocks, generator=g, device="cuda").int()
    table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    for b, first in enumerate(sum(need[:b]) for b in range(B)):
        table[b, :need[b]] = order[first:first + need[b]]
    s = dict(case=case, cache=cache, table=table, ctx=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             longest=max(lens), scale=(D + P) ** -0.5)
    if case["op"] == "absorbed":
        s["q"] = normal(B, n_q, H, W)
    else:
        s["q"] = normal(B, n_q, H, D + P)
        s["wk"] = (normal(H, D, R).float() * R ** -0.5).bfloat16()
        s["wv"] = (normal(H, D, R).float() * R ** -0.5).bfloat16()
    if own:
        pool = s["pool"] = _pool(R, blocks)
        pool.import_blocks(pool.config(), torch.arange(blocks, dtype=torch.int32, device="cuda"),
                           s.pop("cache").view(torch.uint8).reshape(blocks, -1))
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _turn(x, cos, sin, interleaved):
    """The pairs (2 j, 2 j + 1), or (j, j + P / 2), of x turned by the j-th angle."""
    x = x.float()
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :P // 2], x[..., P // 2:])
    y = (a * cos - b * sin, a * sin + b * cos)
    return torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)


def _plain_write(s):
    R, il = s["case"]["latent"], s["case"]["interleaved"]
    t = s["tables"][s["positions"].long()]
    cos, sin = t[:, :P // 2], t[:, P // 2:]
    c = s["kv"][:, :R].float()
    if s["weight"] is not None:
        c = c * torch.rsqrt((c * c).mean(1, keepdim=True) + EPS) * s["weight"].float()
    row = torch.cat((c, _turn(s["kv"][:, R:], cos, sin, il)), 1)
    s["cache"][s["rows"].long(), s["slots"].long()] = row.bfloat16()
    s["q_out"].copy_(_turn(s["q"], cos[:, None], sin[:, None], il))
    return {"cache": s["cache"], "q": s["q_out"]}


def _visible(s, T):
    """[B, n_q, T]: whether query i of a sequence sees token t."""
    n_q = s["case"]["n_q"]
    last = s["ctx"][:, None] - n_q + torch.arange(n_q, device="cuda")
    return torch.arange(T, device="cuda") <= last[..., None]


def _weights(x, seen):
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.masked_fill(m == -math.inf, 0))
    return p / p.sum(-1, keepdim=True).clamp_min(1e-30)


def _plain_absorbed(s):
    R, B, n_q, H = s["case"]["latent"], s["case"]["batch"], s["case"]["n_q"], s["case"]["heads"]
    kv = s["cache"][s["table"].long()].flatten(1, 2).float()
    x = torch.matmul(s["q"].flatten(1, 2).float(), kv.transpose(1, 2)) * s["scale"]
    p = _weights(x.view(B, n_q, H, -1), _visible(s, kv.shape[1])[:, :, None])
    return torch.matmul(p.flatten(1, 2), kv[..., :R]).view(B, n_q, H, R).bfloat16()


def _plain_expanded(s):
    R, B, H = s["case"]["latent"], s["case"]["batch"], s["case"]["heads"]
    kv = s["cache"][s["table"].long()].flatten(1, 2).float()
    T = kv.shape[1]
    k = torch.matmul(kv[..., :R], s["wk"].float().view(H * D, R).t()).view(B, T, H, D).transpose(1, 2)
    v = torch.matmul(kv[..., :R], s["wv"].float().view(H * D, R).t()).view(B, T, H, D).transpose(1, 2)
    q = s["q"].float().transpose(1, 2)
    x = torch.matmul(q[..., :D], k.transpose(2, 3))
    x += torch.matmul(q[..., D:], kv[:, None, :, R:].transpose(2, 3))
    x *= s["scale"]
    p = _weights(x, _visible(s, T)[:, None])
    return torch.matmul(p, v).transpose(1, 2).bfloat16().contiguous()


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op, R = s["case"]["op"], s["case"]["latent"]
    if not own:
        return {"write": _plain_write, "absorbed": _plain_absorbed, "expanded": _plain_expanded}[op](s)
    pool = s["pool"]
    if op == "write":
        pool.write_latent(0, s["rows"], s["slots"], s["kv"], s["positions"], s["tables"], norm_weight=s["weight"],
                          eps=EPS, interleaved=s["case"]["interleaved"], q_rope=s["q"], q_out=s["q_out"])
        return {"cache": s["cache"], "q": s["q_out"]}
    if op == "absorbed":
        q = s["q"]
        return pool.paged_latent_attention(0, q[..., :R], q[..., R:], s["table"], s["ctx"], s["scale"],
                                           max_ctx=s["longest"])
    return pool.latent_prefill_attention(0, s["q"], s["wk"], s["wv"], s["table"], s["ctx"], s["scale"],
                                         max_ctx=s["longest"])


def work(case):
    R, W, H = case["latent"], case["latent"] + P, case["heads"]
    if case["op"] == "write":
        n = case["tokens"]
        return {"bytes": n * (2 * 2 * W + 2 * 2 * H * P + 4 * P + 12) + 2 * R * case["norm"],
                "flops": n * (4 * R * case["norm"] + 3 * P * (H + 1))}
    lens, n_q = _lens(case), case["n_q"]
    rows = case["batch"] * n_q * H
    tokens, pairs = sum(lens), sum(sum(max(0, x - n_q + i + 1) for i in range(n_q)) for x in lens)
    small = sum(-(-x // BLOCK) for x in lens) * 4 + 4 * case["batch"]
    if case["op"] == "absorbed":
        return {"bytes": 2 * tokens * W + 2 * rows * (W + R) + small, "flops": 2 * pairs * H * (W + R)}
    return {"bytes": 2 * tokens * W + 2 * rows * (D + P + D) + 2 * 2 * H * D * R + small,
            "flops": 2 * tokens * R * H * 2 * D + 2 * pairs * H * (D + P + D)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, a sequence and a head at a time
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    R, H = case["latent"], case["heads"]
    if case["op"] == "write":
        half = P // 2
        ang = s["tables"].double()[s["positions"].long()]
        z = torch.complex(ang[:, :half], ang[:, half:])  # a turn is a product of complex numbers

        def turned(x, z):
            x = x.double()
            x = x.reshape(*x.shape[:-1], half, 2) if case["interleaved"] else x.reshape(*x.shape[:-1], 2, half).transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(x.contiguous()) * z)
            return (y if case["interleaved"] else y.transpose(-1, -2)).reshape(*y.shape[:-2], P)

        lat = s["kv"][:, :R].double()
        if s["weight"] is not None:
            lat = lat / (lat.square().sum(1, keepdim=True) / R + EPS).sqrt() * s["weight"].double()
        flat = s["cache"].double().view(-1, R + P)
        flat[s["rows"].long() * BLOCK + s["slots"].long()] = torch.cat((lat, turned(s["kv"][:, R:], z)), 1)
        return {"cache": flat.view(s["cache"].shape), "q": turned(s["q"], z[:, None])}
    lens, n_q = _lens(case), case["n_q"]
    out = torch.zeros(case["batch"], n_q, H, R if case["op"] == "absorbed" else D, dtype=torch.float64, device="cuda")
    for b, L in enumerate(lens):
        if L == 0:
            continue
        kv = s["cache"][s["table"][b, :-(-L // BLOCK)].long()].view(-1, R + P)[:L].double()
        hidden = torch.ones(n_q, L, dtype=torch.bool, device="cuda").triu(L - n_q + 1)
        for h in range(H):
            q = s["q"][b, :, h].double()
            if case["op"] == "absorbed":
                keys, values = kv, kv[:, :R]
            else:
                keys = torch.cat((kv[:, :R] @ s["wk"][h].double().t(), kv[:, R:]), 1)
                values = kv[:, :R] @ s["wv"][h].double().t()
            logits = (q @ keys.t()).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
            out[b, :, h] = torch.softmax(logits, -1) @ values
    return out
