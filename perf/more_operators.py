"""Drafted trees over a paged cache: the operators' plain forms, and the framework's calls.

A serving step that verifies drafted tokens makes three calls on the pool:

  rotate   the new tokens' keys (and the heads' queries) are normalised where the model does
           so, turned by the angles of their positions, and stored with the values at the
           tokens' blocks and slots; a packed pool quantises them on the way.
  tree     out[i, h] = sum_t p[i, h, t] v_t with p = softmax_t(scale * q[i, h] . k_t): query
           i of a sequence's n_q drafted tokens, its last ones, sees every token before
           them and the drafted ones that its row of a bit mask names (its ancestors).
  accept   the drafted tokens on the accepted path move, in every layer, to the places
           behind the tokens before them.
"""
import math
import random

import torch

own = False

BLOCK = 32   # tokens a block
EPS = 1e-6
SEED = 0x5EED  # of a packed pool's basis
BITS = {"bf16": (16, 16), "k4v4": (4, 4), "k8v4": (8, 4), "k8v8": (8, 8)}
GROUP = 32   # values a group of a packed format


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _rotate(name, n, kv_heads, heads, dim, rot, interleaved=False, norm=True, fmt="bf16"):
    return dict(name=name, op="rotate", tokens=n, kv_heads=kv_heads, heads=heads, dim=dim, rot=rot,
                interleaved=interleaved, norm=norm, fmt=fmt)


def _tree(name, batch, n_q, kv_heads, heads, dim, lo, hi, fmt="bf16"):
    """Sequence lengths, drafted tokens among them, are spread over [lo, hi]; the last is hi."""
    return dict(name=name, op="tree", batch=batch, n_q=n_q, kv_heads=kv_heads, heads=heads, dim=dim, lo=lo, hi=hi, fmt=fmt)


def _accept(name, batch, n_q, kv_heads, dim, layers, lo, hi):
    return dict(name=name, op="accept", batch=batch, n_q=n_q, kv_heads=kv_heads, dim=dim, layers=layers, lo=lo, hi=hi)


def listed():
    return [
        # one decode step of a few sequences: latency
        _rotate("rotate a step of 8", 8, 8, 16, 128, 128),
        # the prompts of one scheduler step, heads of 64, an odd number of tokens
        _rotate("rotate 5001 tokens dim 64", 5001, 8, 32, 64, 64, norm=False),
        # the drafted trees of 24 sequences into a packed pool
        _rotate("rotate 24 trees k4v4", 24 * 63, 8, 16, 128, 128, norm=False, fmt="k4v4"),
        # long prompts, half of each head turned, pairs side by side
        _rotate("rotate 16384 tokens", 16384, 8, 32, 128, 64, interleaved=True),
        # a short tree behind a short context: latency
        _tree("tree of 8 behind 1000", 1, 8, 8, 16, 128, 1008, 1008),
        # small trees, many sequences of different lengths, heads of 64
        _tree("tree of 13 x 48 ragged", 48, 13, 8, 32, 64, 13, 4096),
        # one long conversation, heads of 256
        _tree("tree of 31 x 2 dim 256", 2, 31, 4, 8, 256, 9000, 12001),
        # wide trees, long contexts
        _tree("tree of 64 x 16 x 16384", 16, 64, 8, 16, 128, 16384, 16384),
        # a packed pool
        _tree("tree of 24 x 16 k4v4", 16, 24, 8, 16, 128, 8192, 16384, "k4v4"),
        # a packed pool with heads of 64, ragged
        _tree("tree of 16 x 33 k8v8", 33, 16, 8, 32, 64, 500, 6000, "k8v8"),
        # a step's accepted paths
        _accept("accept of 16 x 8", 8, 16, 8, 128, 28, 40, 400),
        # many sequences, wide trees
        _accept("accept of 64 x 64", 64, 64, 8, 128, 28, 64, 300),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("rotate", "tree", "tree", "tree", "accept"))
    dim = rng.choice((64, 128, 128, 256))
    kv_heads = rng.choice((1, 2, 4, 8, 8) if dim < 256 else (1, 2, 4))
    heads = kv_heads * rng.choice((1, 2, 2, 4, 8))
    fmt = rng.choice(("bf16", "bf16", "bf16", "k4v4", "k8v4", "k8v8"))
    if op == "rotate":
        n = _spread(rng, 1, 16384 * 40 * 128 // ((2 * kv_heads + heads) * dim) if fmt == "bf16" else 4096)
        return dict(op=op, tokens=min(n, 32768), kv_heads=kv_heads, heads=heads, dim=dim, rot=rng.choice((dim, dim, dim // 2)),
                    interleaved=rng.random() < 0.4, norm=fmt == "bf16" and rng.random() < 0.5, fmt=fmt)
    if op == "tree":
        n_q = _spread(rng, 1, 96)
        hi = _spread(rng, n_q, 16384)
        room = min((1 << 28) // (hi * heads * n_q), (1 << 28) // (hi * kv_heads * dim))
        batch = _spread(rng, 1, max(1, min(64, room)))
        return dict(op=op, batch=batch, n_q=n_q, kv_heads=kv_heads, heads=heads, dim=dim,
                    lo=rng.choice((n_q, max(n_q, hi // 2), hi)), hi=hi, fmt=fmt)
    n_q = _spread(rng, 1, 96)
    return dict(op=op, batch=_spread(rng, 1, 48), n_q=n_q, kv_heads=kv_heads, dim=dim, layers=rng.choice((1, 4, 16, 28)),
                lo=n_q, hi=n_q + _spread(rng, 1, 200))


def _lens(case):
    rng = random.Random(case["batch"] * 7919 + case["hi"])
    lens = [rng.randint(max(case["lo"], case["n_q"]), case["hi"]) for _ in range(case["batch"])]
    lens[-1] = case["hi"]
    return lens


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _tables(positions, rot):
    """cos and sin of every position's rot / 2 angles, the angles taken in 64 bits."""
    freq = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") / (rot // 2))
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat((a.cos(), a.sin()), 1).float()


def _signs(dim):
    """The signs of a packed pool's basis: the top bit of splitmix64(seed + i)."""
    m, out = (1 << 64) - 1, []
    for i in range(dim):
        z = (SEED + i + 0x9E3779B97F4A7C15) & m
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & m
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & m
        out.append(-1.0 if (z ^ (z >> 31)) >> 63 else 1.0)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def _basis(dim):
    """[dim, dim]: row i is sign i times row i of the Hadamard matrix, over sqrt(dim)."""
    h = torch.ones(1, 1, dtype=torch.float64, device="cuda")
    while h.shape[0] < dim:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)))
    return _signs(dim)[:, None] * h * dim ** -0.5


def _parts(case, blocks):
    """Shapes of a layer's stored tensors, as bytes: K, V and, packed, their scales and offsets."""
    kb, vb = BITS[case.get("fmt", "bf16")]
    lead = (blocks, BLOCK, case["kv_heads"])
    shapes = [lead + (case["dim"] * kb // 8,), lead + (case["dim"] * vb // 8,)]
    return shapes if kb == 16 else shapes + [lead + (case["dim"] // GROUP * 8,)] * 2


def _views(memory, case, blocks, layers=1):
    """The stored tensors of a pool whose one slab is `memory`: of each kind, [layers, ...] bytes."""
    shapes = _parts(case, blocks)
    sizes = [math.prod(s) for s in shapes]
    whole = memory[:layers * sum(sizes)].view(layers, -1)
    out, at = [], 0
    for shape, size in zip(shapes, sizes):
        out.append(whole[:, at:at + size].view(layers, *shape))
        at += size
    return out


def _pool(case, blocks, memory=None, layers=1):
    """A pool; with `memory` its only slab is that tensor's."""
    import paged_kv_cache_split_gb300 as pkv
    kw = dict(hadamard_seed=SEED, max_slabs=blocks // 32 + 1)
    if memory is not None:
        kw = dict(hadamard_seed=SEED, slab_blocks=blocks, max_slabs=1,
                  allocator=pkv.Allocator(pkv.ALLOC_FN(lambda ctx, n, stream: memory.data_ptr()),
                                          pkv.RELEASE_FN(lambda ctx, ptr, stream: None), None))
    pool = pkv.Pool(layers, case["kv_heads"], case["dim"], case.get("fmt", "bf16"), **kw)
    pool.reserve_rows(blocks)
    return pool


def _memory(case, blocks, layers=1):
    """Memory of a pool's one slab; a little behind the data is the pool's own."""
    return torch.zeros(layers * sum(math.prod(s) for s in _parts(case, blocks)) + layers * 4096 + 4096,
                       dtype=torch.uint8, device="cuda")


def _quantise(x, bits):
    """fp32 [..., dim] to codes (as bytes) and (scale, offset) of each group of 32."""
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    lo, top = g.amin(-1, keepdim=True), float((1 << bits) - 1)
    scale = (g.amax(-1, keepdim=True) - lo) / top
    c = torch.round((g - lo) / torch.where(scale == 0, torch.ones_like(scale), scale)).clamp(0, top)
    c = torch.where(scale == 0, torch.zeros_like(c), c).to(torch.uint8).reshape(x.shape)
    if bits == 4:
        c = c[..., 0::2] | (c[..., 1::2] << 4)
    return c, torch.cat((scale, lo), -1).reshape(*x.shape[:-1], -1)


def _values(codes, meta, dim, dtype=torch.float32):
    """What stored codes stand for (meta: bytes or fp32)."""
    if meta.dtype == torch.uint8:
        meta = meta.contiguous().view(torch.float32)
    if codes.shape[-1] * 2 == dim:
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    meta = meta.to(dtype).unflatten(-1, (-1, 2))
    v = codes.to(dtype).unflatten(-1, (-1, GROUP)) * meta[..., :1] + meta[..., 1:]
    return v.flatten(-2)


def _trees(batch, n_q, seed):
    """Random trees, parents before children: [batch, n_q, words] int32, each node's ancestors and itself."""
    rng = random.Random(seed)
    words = -(-n_q // 32)
    out = []
    for _ in range(batch):
        seen = []
        for i in range(n_q):
            # drafts branch near their ends: a parent among the last few nodes, or the root
            p = -1 if i == 0 or rng.random() < 0.1 else rng.randint(max(0, i - 6), i - 1)
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        out.append([[(s >> 32 * w & 0xFFFFFFFF) - ((s >> 32 * w + 31 & 1) << 32) for w in range(words)] for s in seen])
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _table(lens, g):
    """Block table over shuffled blocks, and how many there are."""
    need = [-(-x // BLOCK) for x in lens]
    order = torch.randperm(sum(need), generator=g, device="cuda").int()
    table = torch.zeros(len(lens), max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, at


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda").bfloat16()  # noqa: E731
    Hk, D = case["kv_heads"], case["dim"]
    if case["op"] == "rotate":
        n, H = case["tokens"], case["heads"]
        blocks = -(-n // BLOCK) + 1
        memory = _memory(case, blocks)
        pool = _pool(case, blocks, memory) if own else None
        place = torch.randperm(blocks * BLOCK, generator=g, device="cuda")[:n].int()  # tokens of many sequences
        qkv = normal(n, H + 2 * Hk, D)  # one projection's output
        weight = [1 + 0.1 * normal(D) for _ in range(2)] if case["norm"] else [None, None]
        return dict(case=case, pool=pool, memory=memory, cache=_views(memory, case, blocks), rows=place // BLOCK,
                    slots=place % BLOCK, q=qkv[:, :H], k=qkv[:, H:H + Hk], v=qkv[:, H + Hk:], q_norm=weight[0],
                    k_norm=weight[1], positions=torch.randint(0, 40000, (n,), generator=g, device="cuda").int(),
                    tables=_tables(40000, case["rot"]), basis=None if case["fmt"] == "bf16" else _basis(D),
                    q_out=torch.empty(n, H, D, dtype=torch.bfloat16, device="cuda"))
    lens, n_q, B = _lens(case), case["n_q"], case["batch"]
    table, blocks = _table(lens, g)
    s = dict(case=case, table=table, ctx=torch.tensor(lens, dtype=torch.int32, device="cuda"), longest=max(lens))
    if case["op"] == "accept":
        rng = random.Random(seed)
        n = [rng.randint(0, min(n_q, 9)) for _ in range(B)]  # accepted paths are short
        path = [sorted(rng.sample(range(min(n_q, 6 * x) if x else 1), x)) + [0] * (min(n_q, 9) - x) for x in n]
        memory = _memory(case, blocks, case["layers"])
        pool = _pool(case, blocks, memory, case["layers"]) if own else None
        cache = [x.view(torch.bfloat16) for x in _views(memory, case, blocks, case["layers"])]
        for x in cache:
            x.normal_(generator=g)
        s.update(pool=pool, memory=memory, cache=cache, path=torch.tensor(path, dtype=torch.int32, device="cuda"),
                 path_lens=torch.tensor(n, dtype=torch.int32, device="cuda"),
                 new_lens=torch.empty(B, dtype=torch.int32, device="cuda"))
        return s
    s.update(scale=D ** -0.5, q=normal(B, n_q, case["heads"], D), mask=_trees(B, n_q, seed))
    k, v = normal(blocks, BLOCK, Hk, D), normal(blocks, BLOCK, Hk, D)
    if case["fmt"] == "bf16":
        s["cache"] = [k.view(torch.uint8), v.view(torch.uint8)]
    else:
        kb, vb = BITS[case["fmt"]]
        (kc, km), (vc, vm) = _quantise(k.float(), kb), _quantise(v.float(), vb)
        s["cache"] = [kc, vc, km.view(torch.uint8), vm.view(torch.uint8)]
        s["basis"] = _basis(D)
    if own:
        pool = s["pool"] = _pool(case, blocks)
        records = torch.cat([x.reshape(blocks, -1) for x in s.pop("cache")], 1)
        pool.import_blocks(pool.config(), torch.arange(blocks, dtype=torch.int32, device="cuda"), records)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _turn(x, cos, sin, case):
    """The first `rot` values of x turned: pairs (2 j, 2 j + 1), or (j, j + rot / 2), by the j-th angle."""
    r = case["rot"]
    t, rest = x[..., :r], x[..., r:]
    a, b = (t[..., 0::2], t[..., 1::2]) if case["interleaved"] else (t[..., :r // 2], t[..., r // 2:])
    y = (a * cos - b * sin, a * sin + b * cos)
    y = torch.stack(y, -1).flatten(-2) if case["interleaved"] else torch.cat(y, -1)
    return torch.cat((y, rest), -1)


def _normed(x, weight):
    return x if weight is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.to(x.dtype)


def _stored(s):
    """What a packed pool holds for the tokens just written, as the values it stands for."""
    at = (s["rows"].long(), s["slots"].long())
    kc, vc, km, vm = (x[0][at] for x in s["cache"])
    return {"k": _values(kc, km, s["case"]["dim"]), "v": _values(vc, vm, s["case"]["dim"]), "q": s["q_out"]}


def _plain_rotate(s):
    case, r = s["case"], s["case"]["rot"]
    at = (s["rows"].long(), s["slots"].long())
    t = s["tables"][s["positions"].long()][:, None]
    s["q_out"].copy_(_turn(_normed(s["q"].float(), s["q_norm"]), t[..., :r // 2], t[..., r // 2:], case))
    if case["fmt"] == "bf16":
        k = _turn(_normed(s["k"].float(), s["k_norm"]), t[..., :r // 2], t[..., r // 2:], case)
        for cache, x in zip(s["cache"], (k, s["v"])):
            cache.view(torch.bfloat16)[0][at] = x.bfloat16()
        return {"k": s["cache"][0].view(torch.bfloat16), "v": s["cache"][1].view(torch.bfloat16), "q": s["q_out"]}
    # a code's border may lie anywhere: 64 bits up to the quantiser's input
    t = t.double()
    k = _turn(_normed(s["k"].double(), s["k_norm"]), t[..., :r // 2], t[..., r // 2:], case)
    k = torch.matmul(k, s["basis"]).float()
    kb, vb = BITS[case["fmt"]]
    (kc, km), (vc, vm) = _quantise(k, kb), _quantise(s["v"].float(), vb)
    for cache, x in zip(s["cache"], (kc, vc, km.view(torch.uint8), vm.view(torch.uint8))):
        cache[0][at] = x
    return _stored(s)


def _seen(s, T):
    """[B, n_q, T]: whether query i of a sequence sees token t."""
    n_q = s["case"]["n_q"]
    bits = torch.arange(n_q, device="cuda")
    tree = (s["mask"].long()[..., bits // 32] >> bits % 32 & 1).bool()  # [B, n_q, n_q]
    t = torch.arange(T, device="cuda") - (s["ctx"].long()[:, None] - n_q)  # [B, T]: the drafted token there
    drafted = (t >= 0) & (t < n_q)
    tree = torch.gather(tree, 2, t.clamp(0, n_q - 1)[:, None].expand(-1, n_q, -1))
    return (t < 0)[:, None] | (drafted[:, None] & tree)


def _context(s, kind, dtype=torch.float32):
    """[B, T, kv_heads, dim]: the sequences' keys (0) or values (1), a packed pool's keys in its basis."""
    at = s["table"].long()
    x = s["cache"][kind][at].flatten(1, 2)
    if s["case"]["fmt"] == "bf16":
        return x.view(torch.bfloat16).to(dtype)
    return _values(x, s["cache"][kind + 2][at].flatten(1, 2), s["case"]["dim"], dtype)


def _plain_tree(s):
    case = s["case"]
    B, n_q, Hk, D, H = case["batch"], case["n_q"], case["kv_heads"], case["dim"], case["heads"]
    q = s["q"].float()
    if case["fmt"] != "bf16":
        q = torch.matmul(q, s["basis"].float())
    q = q.view(B, n_q, Hk, H // Hk, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, D)
    k = _context(s, 0)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]
    T = k.shape[1]
    del k
    x = x.view(B, Hk, H // Hk, n_q, T).masked_fill(~_seen(s, T)[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.masked_fill(m == -math.inf, 0))
    del x
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    y = torch.matmul(p.flatten(2, 3), _context(s, 1).transpose(1, 2))
    return y.view(B, H, n_q, D).transpose(1, 2).bfloat16().contiguous()


def _plain_accept(s):
    n_q = s["case"]["n_q"]
    first = s["ctx"].long() - n_q
    k = torch.arange(s["path"].shape[1], device="cuda")
    move = k < s["path_lens"][:, None]                       # [B, path]
    b = torch.arange(len(first), device="cuda")[:, None].expand_as(move)[move]
    src, dst = (first[:, None] + s["path"])[move], (first[:, None] + k)[move]
    rs, rd = s["table"][b, src // BLOCK].long(), s["table"][b, dst // BLOCK].long()
    for cache in s["cache"]:
        cache[:, rd, dst % BLOCK] = cache[:, rs, src % BLOCK]
    s["new_lens"].copy_(first + s["path_lens"])
    return {"k": s["cache"][0], "v": s["cache"][1], "lens": s["new_lens"]}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if not own:
        return {"rotate": _plain_rotate, "tree": _plain_tree, "accept": _plain_accept}[case["op"]](s)
    pool = s["pool"]
    if case["op"] == "rotate":
        pool.write_rotated(0, s["rows"], s["slots"], s["k"], s["v"], s["positions"], s["tables"], q=s["q"],
                           k_norm=s["k_norm"], q_norm=s["q_norm"], eps=EPS, interleaved=case["interleaved"],
                           q_out=s["q_out"])
        if case["fmt"] != "bf16":
            return _stored(s)
        return {"k": s["cache"][0].view(torch.bfloat16), "v": s["cache"][1].view(torch.bfloat16), "q": s["q_out"]}
    if case["op"] == "tree":
        return pool.paged_tree_attention(0, s["q"], s["mask"], s["table"], s["ctx"], s["scale"], max_ctx=s["longest"])
    pool.accept_drafts(s["path"], s["path_lens"], s["table"], s["ctx"], case["n_q"], new_lens=s["new_lens"])
    return {"k": s["cache"][0], "v": s["cache"][1], "lens": s["new_lens"]}


def _token_bytes(case):
    """Stored bytes of a token of one layer."""
    return sum(math.prod(x[1:]) for x in _parts(case, 1)) // BLOCK


def work(case):
    Hk, D = case["kv_heads"], case["dim"]
    if case["op"] == "rotate":
        n, H, r = case["tokens"], case["heads"], case["rot"]
        return {"bytes": n * (2 * D * (2 * Hk + 2 * H) + _token_bytes(case) + 4 * r + 12) + 4 * D * case["norm"],
                "flops": n * (H + Hk) * (3 * r + 4 * D * case["norm"])
                + (0 if case["fmt"] == "bf16" else n * Hk * D * (2 * 4 + int(math.log2(D))))}
    lens, n_q = _lens(case), case["n_q"]
    if case["op"] == "tree":
        H, words = case["heads"], -(-n_q // 32)
        rows, tokens = case["batch"] * n_q * H, sum(lens)
        pairs = H * sum(n_q * (x - n_q) + n_q * (n_q + 1) // 2 for x in lens)
        return {"bytes": tokens * _token_bytes(case) + 2 * 2 * rows * D + 4 * case["batch"] * n_q * words
                + sum(-(-x // BLOCK) for x in lens) * 4 + 4 * case["batch"], "flops": 4 * pairs * D}
    # about half of the longest path is accepted
    moved = case["batch"] * (1 + min(n_q, 9)) // 2
    return {"bytes": 2 * moved * case["layers"] * _token_bytes(case) + 4 * case["batch"] * (min(n_q, 9) + 3), "flops": 0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rotate(s):
    case, D = s["case"], s["case"]["dim"]
    half = case["rot"] // 2
    ang = s["tables"].double()[s["positions"].long()][:, None]
    z = torch.complex(ang[..., :half], ang[..., half:])  # a turn is a product of complex numbers

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = x / (x.square().sum(-1, keepdim=True) / D + EPS).sqrt() * weight.double()
        t = x[..., :2 * half]
        t = t.unflatten(-1, (half, 2)) if case["interleaved"] else t.unflatten(-1, (2, half)).transpose(-1, -2)
        y = torch.view_as_real(torch.view_as_complex(t.contiguous()) * z)
        y = y.flatten(-2) if case["interleaved"] else y.transpose(-1, -2).flatten(-2)
        return torch.cat((y, x[..., 2 * half:]), -1)

    k, q = turned(s["k"], s["k_norm"]), turned(s["q"], s["q_norm"])
    at = (s["rows"].long(), s["slots"].long())
    if case["fmt"] == "bf16":
        out = {"q": q}
        for name, cache, x in (("k", s["cache"][0], k), ("v", s["cache"][1], s["v"].double())):
            whole = cache.view(torch.bfloat16)[0].double()
            whole[at] = x
            out[name] = whole[None]
        return out
    i = torch.arange(D, device="cuda")
    odd = i[:, None] & i  # the sign of entry (i, j) is the parity of the bits that i and j share
    for shift in (4, 2, 1):
        odd = odd ^ odd >> shift
    h = 1.0 - 2.0 * (odd & 1).double()
    k = (k * _signs(D)) @ h / math.sqrt(D)

    def held(x, bits):
        # the quantiser works on fp32 values, and its scale and offset are fp32
        x = x.float().unflatten(-1, (-1, GROUP))
        lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
        scale = (hi - lo) / float(2 ** bits - 1)
        code = ((x - lo) / scale).round().nan_to_num(0.0)
        return (code.double() * scale.double() + lo.double()).flatten(-2)

    kb, vb = BITS[case["fmt"]]
    return {"k": held(k, kb), "v": held(s["v"].double(), vb), "q": q}


def exact(case, seed):
    if case["op"] == "accept":
        return None  # copies
    s = prepare(case, seed)
    if case["op"] == "rotate":
        return _exact_rotate(s)
    lens, n_q, Hk, D, H = _lens(case), case["n_q"], case["kv_heads"], case["dim"], case["heads"]
    out = torch.zeros(case["batch"], n_q, H, D, dtype=torch.float64, device="cuda")
    words = s["mask"].cpu().tolist()
    for b, L in enumerate(lens):
        hidden = torch.zeros(n_q, L, dtype=torch.bool)
        for i in range(n_q):
            hidden[i, L - n_q:] = torch.tensor([not words[b][i][j // 32] >> j % 32 & 1 for j in range(n_q)])
        hidden = hidden.cuda()
        at = s["table"][b, :-(-L // BLOCK)].long()
        kv = []
        for kind in (0, 1):
            x = s["cache"][kind][at].flatten(0, 1)[:L]
            if case["fmt"] == "bf16":
                kv.append(x.view(torch.bfloat16).double())
            else:
                kv.append(_values(x, s["cache"][kind + 2][at].flatten(0, 1)[:L], D, torch.float64))
        if case["fmt"] != "bf16":
            kv[0] = kv[0] @ s["basis"].t()  # back to the heads' own coordinates
        for h in range(H):
            k, v = (x[:, h // (H // Hk)] for x in kv)
            logits = (s["q"][b, :, h].double() @ k.t()).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
            out[b, :, h] = torch.softmax(logits, -1) @ v
    return out
