"""The drafted-token operators through the C ABI: the rotated cache write, attention for trees
of drafted tokens, and the move of accepted tokens, each against a plain statement of its
formula in 64 bits, and a run of them together.

Tolerances count the roundings each operator documents (u = 2^-8 is half a bf16 step
relative to the value, h = 2^-11 half an fp16 one):
  write, bf16    one rounding of a value computed in fp32: u |y|, plus 2^-16 of the row's
                 largest value for the fp32 steps (a few roundings of 2^-24 each, and the mean
                 of squares of 256 values);
  write, packed  the scale and offset are fp32 values of a row known to 2^-22 of its largest
                 value (2^-36 without the norm); a code is the nearest one of a quotient off by
                 the 2^-22 of top steps that the fp32 subtraction and division may lose;
  tree           u |y| for the output, u sum p |v| for the probabilities' rounding to 16 bits
                 (bf16: u; fp16, packed pools: less), 2 d sum p |v| for the logits, d being D 2^-23
                 scale sum |q k| for the fp32 sums.  A packed value is c s + o with s and o rounded to
                 fp16 and one rounding more: off by h (|c s| + |o| + |c s + o|) <= h (2 M + M + M) =
                 4 h M, M the largest magnitude of its group, as c s is at most the group's range.  So
                 values add 4 h sum p M and keys 4 h scale sum |q| M to d, the queries' own rounding h
                 scale sum |q| |k|.  The operands lie under a power of two by tile (64 tokens) whose
                 largest is 2^13 to 2^14: fp16 drops at most 2^-25 of it, 2^-38 of the tile's largest
                 magnitude T a value (keys: 2^-38 scale D |q| T; values: 2^-38 T), and at most 2^-25
                 of P, whose largest is 2^-1 at least: L 2^-24 of the largest p T over L tokens.
The elementwise bounds are worst cases; a relative L2 bound holds the average: each
rounding contributes at most u / sqrt(3) in the mean square, at most four of them with
logits of unit size, so 2 u < 1e-2."""
import ctypes
import math

import numpy as np
import pytest

import paged_kv_cache_split_gb300 as pkv
from paged_kv_cache_split_gb300 import workloads as wl
from tests.harness import bf16_dev_to_f64, to_dev_bf16  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -8
H16 = 2.0 ** -11
BITS = {"bf16": (16, 16), "k4v4": (4, 4), "k8v4": (8, 4), "k8v8": (8, 8)}
SEED = 0xABCD


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def tables(n, rot):
    f = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") / (rot // 2))
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat((a.cos(), a.sin()), 1).float()


def splitmix_signs(D, seed=SEED):
    m, out = (1 << 64) - 1, []
    for i in range(D):
        z = (seed + i + 0x9E3779B97F4A7C15) & m
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & m
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & m
        out.append(-1.0 if (z ^ (z >> 31)) >> 63 else 1.0)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def basis(D):
    h = torch.ones(1, 1, dtype=torch.float64, device="cuda")
    while h.shape[0] < D:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)))
    return splitmix_signs(D)[:, None] * h * D ** -0.5


def make_pool(fmt, Hk, D, rows, layers=1, group=32, slab_blocks=32):
    p = pkv.Pool(layers, Hk, D, fmt, hadamard_seed=SEED, group_size=group, slab_blocks=slab_blocks,
                 max_slabs=rows // slab_blocks + 4)
    p.reserve_rows(rows)
    return p


def unpack(codes, bits):
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2) if bits == 4 else codes


def stored(pool, rows, layer=0):
    """Per kind, what blocks `rows` hold of `layer`: codes [n, 32, Hk, D] and, packed, fp32
    [n, 32, Hk, D / group, 2]; bf16 values for a bf16 pool."""
    n, Hk, D = rows.numel(), pool.n_kv_heads, pool.head_dim
    rec = pool.export_blocks(rows).view(n, pool.n_layers, -1)[:, layer]
    out, at = [], 0
    kb, vb = BITS[pool.format]
    for kind, rb in enumerate(pool.row_bytes):
        x = rec[:, at:at + 32 * Hk * rb].reshape(n, 32, Hk, rb)
        at += 32 * Hk * rb
        if kind >= 2:
            out.append(x.contiguous().view(torch.float32).unflatten(-1, (-1, 2)))
        elif kb == 16:
            out.append(x.contiguous().view(torch.bfloat16))
        else:
            out.append(unpack(x, (kb, vb)[kind]))
    return out


def values(codes, meta):
    g = codes.shape[-1] // meta.shape[-2]
    return (codes.double().unflatten(-1, (-1, g)) * meta[..., :1].double() + meta[..., 1:].double()).flatten(-2)


def turned(x, pos, tab, interleaved, weight=None, eps=1e-6):
    """The rotated write's formula in 64 bits."""
    x = x.double()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    rot = tab.shape[1]
    t = tab.double()[pos.long()][:, None]
    c, s = t[..., :rot // 2], t[..., rot // 2:]
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    y = (a * c - b * s, a * s + b * c)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat((y, x[..., rot:]), -1)


def check(got, ref, tol, what):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert worst <= 1, f"{what}: {worst:.2f} times the bound"


def check_bf16_rows(got, ref, what):
    check(got, ref, U * ref.abs() + 2.0 ** -16 * ref.abs().amax(-1, keepdim=True) + 1e-30, what)


def check_packed_rows(codes, meta, x, bits, known, what):
    """codes and (scale, offset) of rows whose true values are x, known to `known` of a row's largest."""
    g, top = x.shape[-1] // meta.shape[-2], 2 ** bits - 1
    xg = x.unflatten(-1, (-1, g))
    off = known * x.abs().amax(-1, keepdim=True)[..., None] + 2.0 ** -24 * xg.abs().amax(-1, keepdim=True) + 1e-44
    scale, lo = meta[..., :1].double(), meta[..., 1:].double()
    assert ((lo - xg.amin(-1, keepdim=True)).abs() <= off).all(), f"{what}: offsets"
    want = (xg.amax(-1, keepdim=True) - xg.amin(-1, keepdim=True)) / top
    assert ((scale - want).abs() <= 2 * off / top + 2.0 ** -22 * want).all(), f"{what}: scales"
    c = codes.double().unflatten(-1, (-1, g))
    q = (xg - lo) / scale
    slack = top * 2.0 ** -22 + 2 * off / scale
    near = ((c - q).abs() <= 0.5 + slack) | (scale == 0) & (c == 0)
    assert near.all(), f"{what}: codes, {(~near).sum().item()} are not the nearest"


# ---------------------------------------------------------------------------
# write_rotated
# ---------------------------------------------------------------------------
def write_case(fmt, D, Hk, Hq, n, rot, interleaved, norm, group=32, seed=0, positions=5000):
    g = gen(seed + n + D + Hk)
    blocks = -(-n // 32) + 1
    pool = make_pool(fmt, Hk, D, blocks, group=group)
    place = torch.randperm(blocks * 32, generator=g, device="cuda")[:n].int()
    rows, slots = place // 32, place % 32
    qkv = normal(g, n, Hq + 2 * Hk, D)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    kn, qn = ((1 + 0.1 * normal(g, D)).bfloat16() if norm else None for _ in range(2))
    pos = torch.randint(0, positions, (n,), generator=g, device="cuda").int()
    tab = tables(positions, rot)
    before = stored(pool, torch.arange(blocks, dtype=torch.int32, device="cuda"))
    out = pool.write_rotated(0, rows, slots, k, v, pos, tab, q=q if Hq else None, k_norm=kn, q_norm=qn if Hq else None,
                             interleaved=interleaved)
    assert pool.check_errors() == 0
    after = stored(pool, torch.arange(blocks, dtype=torch.int32, device="cuda"))
    at = (rows.long(), slots.long())
    if Hq:
        check_bf16_rows(out, turned(q, pos, tab, interleaved, qn), "queries")
    else:
        assert out is None
    want = turned(k, pos, tab, interleaved, kn)
    if fmt == "bf16":
        check_bf16_rows(after[0][at], want, "keys")
        assert torch.equal(after[1][at].view(torch.int16), v.contiguous().view(torch.int16)), "values are copied"
    else:
        kb, vb = BITS[fmt]
        check_packed_rows(after[0][at], after[2][at], want @ basis(D), kb, 2.0 ** -22 if norm else 2.0 ** -36, "keys")
        check_packed_rows(after[1][at], after[3][at], v.double(), vb, 0.0, "values")
    # slots that no token names keep what they held
    for a, b in zip(after, before):
        rest = torch.ones(blocks, 32, dtype=torch.bool, device="cuda")
        rest[at] = False
        assert torch.equal(a[rest], b[rest])


@pytest.mark.parametrize("fmt,D,group", [("bf16", 64, 32), ("bf16", 128, 32), ("bf16", 256, 32), ("k4v4", 64, 32),
                                         ("k4v4", 128, 64), ("k8v4", 128, 32), ("k8v8", 256, 32), ("k4v4", 256, 64),
                                         ("k8v8", 64, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_write_rotated(fmt, D, group, interleaved, norm):
    write_case(fmt, D, 8 if D < 256 else 4, 16, 77, D, interleaved, norm, group)


@pytest.mark.parametrize("fmt", ["bf16", "k4v4", "k8v8"])
@pytest.mark.parametrize("D,Hk,Hq,n,rot", [(64, 1, 1, 1, 64), (64, 1, 0, 3, 32), (64, 3, 9, 65, 64), (128, 1, 8, 2, 32),
                                           (128, 5, 5, 33, 96), (128, 8, 64, 31, 64), (256, 1, 2, 9, 256),
                                           (256, 7, 7, 40, 128), (256, 8, 64, 5, 160), (64, 8, 32, 4500, 64),
                                           (128, 2, 127, 12, 128)])
def test_write_rotated_shapes(fmt, D, Hk, Hq, n, rot):
    for il in (False, True):
        write_case(fmt, D, Hk, Hq, n, rot, il, n % 2 == 1)


@pytest.mark.parametrize("fmt,D,group", [("bf16", 128, 32), ("k4v4", 128, 32), ("k4v4", 128, 64), ("k8v4", 64, 32),
                                         ("k8v8", 256, 32)])
def test_write_rotated_by_nothing_is_write_block(fmt, D, group):
    """Angles of zero and no norm: what write_block stores.  Bit for bit but for the scales of
    packed groups, which may be an ulp apart; a code then differs where a value lies on a border."""
    g = gen(3)
    a, b = (make_pool(fmt, 4, D, 8, group=group) for _ in range(2))
    n = 201
    place = torch.randperm(256, generator=g, device="cuda")[:n].int()
    k = (torch.randn(n, 4, D, generator=g, device="cuda") * torch.exp(torch.randn(n, 4, 1, generator=g, device="cuda") * 3)).bfloat16()
    v = normal(g, n, 4, D)
    k[7] = 0  # groups of one value: a scale of 0
    v[8] = 1.5
    tab = torch.cat((torch.ones(4, D // 2), torch.zeros(4, D // 2)), 1).cuda()
    a.write_rotated(0, place // 32, place % 32, k, v, place % 4, tab)
    b.write_block(0, place // 32, place % 32, k, v)
    x, y = (stored(p, torch.arange(8, dtype=torch.int32, device="cuda")) for p in (a, b))
    if fmt == "bf16":
        assert torch.equal(x[0].view(torch.int16), y[0].view(torch.int16))
        assert torch.equal(x[1].view(torch.int16), y[1].view(torch.int16))
        return
    for kind in (0, 1):
        s, t = x[kind + 2].double(), y[kind + 2].double()
        assert torch.equal(s[..., 1], t[..., 1]), "offsets"
        assert ((s[..., 0] - t[..., 0]).abs() <= 2.0 ** -22 * t[..., 0]).all(), "scales"
        apart = (x[kind].int() - y[kind].int()).abs()
        # bf16 values over a group's range: a border is met by less than one value in 16
        assert apart.max() <= 1 and apart.double().mean() < 1 / 16, "codes"


@pytest.mark.parametrize("fmt", ["k4v4", "k8v8"])
@pytest.mark.parametrize("mag", [2.0 ** -60, 2.0 ** -20, 2.0 ** 16, 2.0 ** 60])
def test_write_rotated_packed_magnitudes(fmt, mag):
    """Rows of any magnitude, with an outlier in each: the turned keys keep their bits."""
    g = gen(4)
    D, n = 128, 64
    pool = make_pool(fmt, 2, D, 2)
    k = torch.randn(n, 2, D, generator=g, device="cuda")
    k[torch.arange(n), :, torch.arange(n) % D] *= 2.0 ** 9
    k, v = (k * mag).bfloat16(), (torch.randn(n, 2, D, generator=g, device="cuda") * mag).bfloat16()
    t = torch.arange(n, dtype=torch.int32, device="cuda")
    tab = tables(n, D)
    pool.write_rotated(0, t // 32, t % 32, k, v, t, tab)
    kc, vc, km, vm = (x.flatten(0, 1) for x in stored(pool, i32([0, 1])))
    kb, vb = BITS[fmt]
    check_packed_rows(kc, km, turned(k, t, tab, False) @ basis(D), kb, 2.0 ** -36, "keys")
    check_packed_rows(vc, vm, v.double(), vb, 0.0, "values")


def test_write_rotated_in_place_and_strided():
    g = gen(5)
    n, Hk, Hq, D = 50, 2, 6, 128
    for fmt in ("bf16", "k4v4"):
        pool = make_pool(fmt, Hk, D, 4)
        t = torch.arange(n, dtype=torch.int32, device="cuda")
        tab = tables(n, D)
        kv = normal(g, n, Hk, 2 * D + 8)
        q = normal(g, Hq, n, D)  # heads first
        want = turned(q.transpose(0, 1), t, tab, False)
        got = pool.write_rotated(0, t // 32, t % 32, kv[..., :D], kv[..., D + 8:], t, tab, q=q.transpose(0, 1),
                                 q_out=q.transpose(0, 1))
        assert got.data_ptr() == q.data_ptr()
        check_bf16_rows(q.transpose(0, 1), want, "in place")
        if fmt == "bf16":
            k, v = (x.flatten(0, 1)[:n] for x in stored(pool, i32([0, 1])))
            check_bf16_rows(k, turned(kv[..., :D], t, tab, False), "keys")
            assert torch.equal(v, kv[..., D + 8:])
        # one key for every head: a stride of zero
        one = normal(g, n, 1, D).expand(n, Hk, D)
        pool.write_rotated(0, t // 32, t % 32, one, one, t, tab)
        x = stored(pool, i32([0, 1]))
        for y in x:
            assert torch.equal(y[:, :, 0], y[:, :, 1])
        assert pool.check_errors() == 0


@pytest.mark.parametrize("fmt", ["bf16", "k8v4"])
@pytest.mark.parametrize("bad,word", [("row", pkv.ERR_ROW), ("row-", pkv.ERR_ROW), ("slot", pkv.ERR_SLOT),
                                      ("slot-", pkv.ERR_SLOT), ("pos", pkv.ERR_POS), ("pos-", pkv.ERR_POS)])
def test_write_rotated_out_of_range(fmt, bad, word):
    g = gen(6)
    n, D = 40, 64
    pool = make_pool(fmt, 2, D, 32)
    t = torch.arange(n, dtype=torch.int32, device="cuda")
    rows, slots, pos = t // 32, t % 32, t.clone()
    {"row": rows, "slot": slots, "pos": pos}[bad.rstrip("-")][5] = -1 if bad[-1] == "-" else {"r": 32, "s": 32, "p": n}[bad[0]]
    q = normal(g, n, 4, D)
    mark = torch.full_like(q, 7.0)
    tab = tables(n, D)
    pool.write_rotated(0, rows, slots, normal(g, n, 2, D), normal(g, n, 2, D), pos, tab, q=q, q_out=mark)
    assert pool.check_errors() == word
    for x in stored(pool, i32([0, 1])):
        flat = x.flatten(0, 1)
        assert not flat[5].any() and flat[4].any() and flat[6].any()
    if bad.startswith("pos"):
        assert (mark[5] == 7).all()
    else:
        check_bf16_rows(mark, turned(q, t, tab, False), "queries")


def test_write_rotated_refusals():
    pool = make_pool("bf16", 2, 64, 4)
    t = torch.arange(4, dtype=torch.int32, device="cuda")
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16, device="cuda")
    call = lambda **kw: pool.write_rotated(**{**dict(layer=0, rows=t, slots=t, k=x, v=x, positions=t,  # noqa: E731
                                                     cos_sin=tables(4, 64)), **kw})
    call()
    for kw in (dict(layer=1), dict(cos_sin=tables(4, 16)), dict(cos_sin=tables(4, 128)), dict(cos_sin=tables(4, 48)),
               dict(q=q, q_out=q.transpose(0, 1)[:, :1].expand(4, 4, 64)), dict(k_norm=x[0, 0], eps=-1.0),
               dict(k_norm=x[0, 0], eps=math.inf)):
        with pytest.raises(pkv.PkvError) as e:
            call(**kw)
        assert e.value.status == pkv.PKV_ERR_INVALID
    odd = torch.zeros(4, 2, 70, dtype=torch.bfloat16, device="cuda")
    shifted = torch.zeros(4 * 128 + 8, dtype=torch.bfloat16, device="cuda")[1:513].view(4, 2, 64)
    for kw in (dict(k=odd[..., :64]), dict(v=shifted), dict(q=q, q_out=q.as_strided((4, 4, 64), (64, 64, 1)))):
        with pytest.raises(pkv.PkvError):
            call(**kw)
    for kw in (dict(k=x[:3]), dict(k=x.float()), dict(q_out=q), dict(q_norm=x[0, 0]), dict(positions=t.long()),
               dict(q=q[0]), dict(k=x.cpu())):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    latent = pkv.Pool(1, 1, 256, "latent", max_slabs=2)
    with pytest.raises(pkv.PkvError) as e:
        latent.write_rotated(0, t, t, torch.zeros(4, 1, 256, dtype=torch.bfloat16, device="cuda"),
                             torch.zeros(4, 1, 256, dtype=torch.bfloat16, device="cuda"), t, tables(4, 64))
    assert e.value.status == pkv.PKV_ERR_FORMAT
    none = t[:0]
    assert pool.write_rotated(0, none, none, x[:0], x[:0], none, tables(4, 64), q=q[:0]).shape == (0, 4, 64)


# ---------------------------------------------------------------------------
# paged_tree_attention
# ---------------------------------------------------------------------------
class Case:
    """A pool whose sequences hold seeded tokens in shuffled blocks.  Slots past a sequence's
    length hold stale bytes."""

    def __init__(self, fmt, D, Hk, lens, seed=0, group=32, layers=1, layer=0, stale=True, mag_k=1.0, mag_v=1.0, extra=0,
                 slab_blocks=32, shape_kv=None):
        g = gen(seed)
        self.fmt, self.D, self.Hk, self.lens, self.layer = fmt, D, Hk, list(lens), layer
        need = [-(-max(x, 0) // 32) for x in lens]
        n = max(1, sum(need))
        self.pool = make_pool(fmt, Hk, D, n + 3, layers, group, slab_blocks)
        order = torch.randperm(n + 3, generator=g, device="cuda")[:n].int()
        self.table = torch.zeros(len(lens), max(1, max(need) + extra), dtype=torch.int32, device="cuda")
        live = torch.zeros(n, 32, dtype=torch.bool, device="cuda")
        at = 0
        for b, L in enumerate(lens):
            self.table[b, :need[b]] = order[at:at + need[b]]
            live[at:at + need[b]].view(-1)[:max(L, 0)] = True
            at += need[b]
        k = torch.randn(n, 32, Hk, D, generator=g, device="cuda") * mag_k
        v = torch.randn(n, 32, Hk, D, generator=g, device="cuda") * mag_v
        if shape_kv:
            k, v = shape_kv(k, v)
        t = torch.arange(n * 32, dtype=torch.int32, device="cuda")
        self.order = order
        self.pool.write_block(layer, order[(t // 32).long()], t % 32, k.bfloat16().view(-1, Hk, D), v.bfloat16().view(-1, Hk, D))
        self.live, self.need = live, need
        if stale:
            self.spoil(~live)
        self.ctx = i32(list(lens))

    def spoil(self, where):
        """NaN (or the bytes 0xFF: NaN metadata) into the slots `where` [n, 32] of the blocks in order."""
        rec = self.pool.export_blocks(self.order)
        n, Hk = rec.shape[0], self.Hk
        one = rec.view(n, self.pool.n_layers, -1)[:, self.layer]
        at = 0
        for rb in self.pool.row_bytes:
            one[:, at:at + 32 * Hk * rb].view(n, 32, Hk * rb)[where] = 0xFF
            at += 32 * Hk * rb
        self.pool.import_blocks(self.pool.config(), self.order, rec)

    def kv(self, b):
        """[L, Hk, D] keys and values of sequence b in 64 bits, and for a packed pool the largest
        magnitude of each value's group; its keys are in the pool's basis."""
        L = self.lens[b]
        rows = self.table[b, :-(-L // 32)].contiguous()
        x = stored(self.pool, rows, self.layer)
        if self.fmt == "bf16":
            return [y.flatten(0, 1)[:L].double() for y in x] + [None, None]
        k, v = (values(x[i], x[i + 2]).flatten(0, 1)[:L] for i in (0, 1))
        return [k, v] + [y.abs().unflatten(-1, (x[2].shape[-2], -1)).amax(-1, keepdim=True).expand(
            *y.shape[:-1], x[2].shape[-2], y.shape[-1] // x[2].shape[-2]).flatten(-2) for y in (k, v)]


def random_tree(B, n_q, seed):
    rng = np.random.default_rng(seed)
    parents = np.full((B, n_q), -1, np.int64)
    for i in range(1, n_q):
        parents[:, i] = np.where(rng.random(B) < 0.15, -1, rng.integers(max(0, i - 5), i, B))
    return parents


def bits_of(mask, n_q):
    """[..., n_q, words] words to booleans [..., n_q, n_q]."""
    j = torch.arange(n_q, device=mask.device)
    return (mask.long()[..., j // 32] >> j % 32 & 1).bool()


def tile_largest(x):
    """[L]: the largest of x [L, D] in each token's tile of 64."""
    m = x.amax(-1)
    m = torch.nn.functional.pad(m, (0, -m.shape[0] % 64)).view(-1, 64).amax(-1)
    return m.repeat_interleave(64)[:x.shape[0]]


def reference(case, b, q, seen, scale):
    """(out, tolerance) of sequence b; q [n_q, Hq, D], seen [n_q, n_q]."""
    n_q, Hq, D = q.shape
    L, G = case.lens[b], Hq // case.Hk
    k, v, km, vm = case.kv(b)
    qd = q.double() if km is None else q.double() @ basis(D)
    vis = torch.ones(n_q, L, dtype=torch.bool, device="cuda")
    vis[:, L - n_q:] = seen
    unseen = ~vis.any(0)
    for x in (k, v, km, vm):
        if x is not None:
            x[unseen] = 0
    outs, tols = [], []
    for h in range(Hq):
        qh, kh, vh = qd[:, h], k[:, h // G], v[:, h // G]
        x = (qh @ kh.t() * scale).masked_fill(~vis, -math.inf)
        p = torch.softmax(x, -1).nan_to_num(0.0)
        out, mag = p @ vh, p @ vh.abs()
        size = qh.abs() @ kh.abs().t()
        d = D * 2.0 ** -23 * size
        extra = 0.0
        if km is not None:
            d = d + H16 * size + 4 * H16 * (qh.abs() @ km[:, h // G].t())
            tk, tv = (tile_largest(y[:, h // G]) for y in (km, vm))
            d = d + 2.0 ** -38 * D * qh.abs().amax(-1, keepdim=True) * tk
            extra = 4 * H16 * (p @ vm[:, h // G]) + 2.0 ** -38 * tv.max() + L * 2.0 ** -24 * (p * tv).amax(-1, keepdim=True)
        d = (abs(scale) * d).masked_fill(~vis, 0).amax(-1, keepdim=True)
        outs.append(out)
        tols.append(U * out.abs() + (U + 2 * d) * mag + extra + 1e-30)
    return torch.stack(outs, 1), torch.stack(tols, 1)


def run_tree(case, n_q, Hq, seed=0, scale=None, mask=None, q=None, l2=True, **kw):
    B = len(case.lens)
    scale = case.D ** -0.5 if scale is None else scale
    q = normal(gen(seed + 17), B, n_q, Hq, case.D) if q is None else q
    if mask is None:
        mask = torch.from_numpy(pkv.tree_masks(random_tree(B, n_q, seed))[0]).cuda()
    out = case.pool.paged_tree_attention(case.layer, q, mask, case.table, case.ctx, scale, **kw)
    torch.cuda.synchronize()
    seen = bits_of(mask if mask.dim() == 3 else mask.expand(B, *mask.shape), n_q)
    for b, L in enumerate(case.lens):
        if L < n_q:
            assert not out[b].any(), f"sequence {b} has no tokens"
            continue
        ref, tol = reference(case, b, q[b], seen[b], scale)
        check(out[b], ref, tol, f"sequence {b} of length {L}")
        if l2 and ref.norm() > 0:
            assert ((out[b].double() - ref).norm() / ref.norm()).item() <= 1e-2
    return out


FORMATS = [("bf16", 64, 32), ("bf16", 128, 32), ("bf16", 256, 32), ("k4v4", 64, 32), ("k4v4", 128, 32), ("k4v4", 128, 64),
           ("k8v4", 128, 32), ("k8v8", 64, 32), ("k8v8", 128, 32), ("k4v4", 256, 64), ("k8v8", 256, 32)]


@pytest.mark.parametrize("fmt,D,group", FORMATS)
@pytest.mark.parametrize("n_q,G", [(1, 1), (1, 8), (7, 2), (16, 4), (33, 2), (64, 2), (70, 4)])
def test_tree_attention(fmt, D, group, n_q, G):
    lens = [n_q, n_q + 1, 96, 127, 128, 129, 161, 700, 0, 1201]
    lens = [max(x, n_q) if x else 0 for x in lens]
    case = Case(fmt, D, 2, lens, seed=n_q + G, group=group)
    run_tree(case, n_q, 2 * G, seed=n_q)
    assert case.pool.check_errors() == 0


@pytest.mark.parametrize("fmt,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("k4v4", 128), ("k8v8", 256), ("k8v4", 64)])
@pytest.mark.parametrize("Hk,Hq,n_q", [(1, 1, 5), (1, 3, 11), (3, 15, 9), (5, 5, 40), (8, 16, 24), (7, 49, 20), (8, 64, 17),
                                       (1, 16, 130), (2, 2, 300)])
def test_tree_attention_heads(fmt, D, Hk, Hq, n_q):
    case = Case(fmt, D, Hk, [n_q + 40, n_q, 0, n_q + 333], seed=Hq)
    run_tree(case, n_q, Hq, seed=Hq)
    assert case.pool.check_errors() == 0


@pytest.mark.parametrize("fmt,D", [("bf16", 128), ("k4v4", 128), ("bf16", 64), ("bf16", 256)])
@pytest.mark.parametrize("ctas", [1, 2, 7, 40, 152, 400])
def test_tree_attention_any_split(fmt, D, ctas):
    """Any number of CTAs, with bit-identical repeats."""
    case = Case(fmt, D, 4, [900, 12, 0, 4000, 260, 33], seed=9)
    case.pool.decode_set_ctas(ctas)
    a = run_tree(case, 12, 8, seed=2)
    for _ in range(3):
        assert torch.equal(a, case.pool.paged_tree_attention(
            0, normal(gen(19), 6, 12, 8, D), torch.from_numpy(pkv.tree_masks(random_tree(6, 12, 2))[0]).cuda(), case.table,
            case.ctx, D ** -0.5))


def test_a_chain_is_the_causal_prefill():
    n_q = 16
    for fmt, D in (("bf16", 128), ("k4v4", 128), ("k8v8", 64)):
        case = Case(fmt, D, 4, [16, 300, 1025], seed=3)
        q = normal(gen(4), 3, n_q, 8, D)
        mask = torch.from_numpy(pkv.tree_masks(np.arange(n_q) - 1)[0]).cuda()
        a = case.pool.paged_tree_attention(0, q, mask, case.table, case.ctx, D ** -0.5)
        b = case.pool.paged_prefill_attention(0, q, case.table, case.ctx, D ** -0.5)
        assert ((a.double() - b.double()).norm() / b.double().norm()).item() < 1e-2


@pytest.mark.parametrize("fmt,D", [("bf16", 128), ("bf16", 64), ("bf16", 256), ("k4v4", 128), ("k8v8", 64)])
def test_rows_that_see_nothing_are_zero(fmt, D):
    """No prefix and an empty mask row; a prefix and an empty mask row."""
    n_q = 40
    case = Case(fmt, D, 2, [n_q, n_q + 31, n_q + 200], seed=5)
    mask = torch.from_numpy(pkv.tree_masks(random_tree(3, n_q, 1))[0]).cuda()
    mask[:, ::3] = 0
    out = run_tree(case, n_q, 4, mask=mask)
    assert not out[0, ::3].any() and out[1, ::3].any()
    mask[:] = 0
    out = run_tree(case, n_q, 4, mask=mask)
    assert not out[0].any()


@pytest.mark.parametrize("fmt,D", [("bf16", 128), ("bf16", 256), ("k4v4", 128), ("k8v8", 64)])
def test_any_mask(fmt, D):
    """Masks that are no trees: any bits, bits past n_q set, one for all sequences."""
    n_q = 45
    case = Case(fmt, D, 2, [n_q + 19, n_q + 1000, n_q], seed=6)
    g = gen(1)
    mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (3, n_q, 2), generator=g, device="cuda").int()
    run_tree(case, n_q, 6, mask=mask)
    run_tree(case, n_q, 6, mask=mask[1].contiguous())


@pytest.mark.parametrize("fmt,D", [("bf16", 128), ("bf16", 64), ("bf16", 256), ("k4v4", 128), ("k8v8", 64), ("k8v4", 256)])
def test_unseen_drafts_may_hold_anything(fmt, D):
    """A sequence with fewer drafts than the batch: its unused places hold NaN and no mask names them."""
    n_q = 24
    lens = [n_q + 100, n_q + 31, n_q, n_q + 500]
    case = Case(fmt, D, 2, lens, seed=8)
    used = [24, 5, 10, 17]
    mask = pkv.tree_masks(random_tree(4, n_q, 3))[0]
    where, at = torch.zeros_like(case.live), 0
    for b, u in enumerate(used):
        mask[b, u:] = 0
        flat = where[at:at + case.need[b]].view(-1)
        flat[lens[b] - n_q + u:lens[b]] = True
        at += case.need[b]
    # a row of an unused draft sees the prefix alone
    case.spoil(where)
    mask = torch.from_numpy(mask).cuda()
    q = normal(gen(2), 4, n_q, 8, D)
    out = run_tree(case, n_q, 8, mask=mask, q=q)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("fmt,D", [("bf16", 128), ("bf16", 256), ("k4v4", 128), ("k8v8", 128)])
def test_results_hang_on_the_sequence_alone(fmt, D):
    """Other sequences' queries, the queries of unused slots and stale bytes change no bit."""
    n_q = 20
    lens = [n_q + 700, 0, n_q + 55, n_q + 1500]
    outs = []
    q = normal(gen(3), 4, n_q, 4, D)
    mask = torch.from_numpy(pkv.tree_masks(random_tree(4, n_q, 3))[0]).cuda()
    for stale, junk in ((True, float("nan")), (False, 3e38), (True, 0.0)):
        case = Case(fmt, D, 2, lens, seed=4, stale=stale)
        q[1] = junk
        outs.append(case.pool.paged_tree_attention(0, q, mask, case.table, case.ctx, D ** -0.5))
    for o in outs[1:]:
        assert torch.equal(outs[0], o)


@pytest.mark.parametrize("fmt,D", [("bf16", 128), ("bf16", 64), ("bf16", 256), ("k4v4", 128), ("k8v8", 128)])
def test_logits_of_any_size(fmt, D):
    """Rising and falling logits (every tile moves the reference, or none), huge ones, scales of 0
    and below."""
    n_q = 9

    def rising(sign):
        def f(k, v):
            n = k.shape[0] * 32
            ramp = torch.linspace(0, 1, n, device="cuda").view(-1, 32, 1, 1) * sign
            return k * 0.1 + ramp * 4, v
        return f

    for sign in (1, -1):
        case = Case(fmt, D, 1, [900], seed=7, shape_kv=rising(sign))
        q = torch.ones(1, n_q, 2, D, dtype=torch.bfloat16, device="cuda")
        for scale in (D ** -0.5, 0.0, -D ** -0.5):
            run_tree(case, n_q, 2, scale=scale, q=q, l2=False)
    case = Case(fmt, D, 1, [400, 64], seed=7)
    for scale in (30.0, -30.0, 1e-8):
        run_tree(case, n_q, 2, scale=scale, l2=False)


@pytest.mark.parametrize("fmt,D", [("bf16", 128), ("k4v4", 128), ("k8v8", 64), ("k8v4", 256)])
@pytest.mark.parametrize("mk,mv", [(2.0 ** -20, 1.0), (2.0 ** 16, 1.0), (1.0, 2.0 ** -50), (1.0, 2.0 ** 40)])
def test_magnitudes(fmt, D, mk, mv):
    case = Case(fmt, D, 2, [300, 41], seed=8, mag_k=mk, mag_v=mv)
    run_tree(case, 10, 4, scale=D ** -0.5 / mk)
    # and the magnitude in the queries instead of the scale
    q = (torch.randn(2, 10, 4, D, generator=gen(1), device="cuda") / mk).bfloat16()
    run_tree(case, 10, 4, q=q)


def test_uneven_magnitudes():
    """Tokens 2^20 apart within a tile: each keeps the accuracy of its own size."""
    def f(k, v):
        big = torch.arange(32, device="cuda").view(1, 32, 1, 1) % 5 == 0
        return torch.where(big, k * 2.0 ** -12, k), torch.where(big, v, v * 2.0 ** -12)
    for fmt in ("k4v4", "k8v8", "bf16"):
        run_tree(Case(fmt, 128, 2, [333, 64], seed=2, shape_kv=f), 8, 4)


def test_tree_attention_layers_slabs_and_wide_tables():
    case = Case("bf16", 128, 2, [65, 400], seed=1, layers=3, layer=2, extra=5, slab_blocks=5)
    run_tree(case, 4, 4)
    case = Case("k4v4", 64, 8, [65, 400], seed=1, layers=3, layer=1, extra=5, slab_blocks=3)
    run_tree(case, 4, 16)


@pytest.mark.parametrize("fmt", ["bf16", "k4v4"])
def test_tree_attention_lengths_out_of_range(fmt):
    case = Case(fmt, 128, 2, [200, 3, 100, 64], seed=2)
    for bad in (-1, 7, 200 + 33, 2 ** 31 - 1):
        case.ctx = i32([200, bad, 100, 64])
        case.lens[1] = 0
        run_tree(case, 8, 4)
        assert case.pool.check_errors() == pkv.ERR_CTX
    case.ctx = i32([200, 0, 100, 64])
    case.table[2, 1] = 10 ** 6
    out = case.pool.paged_tree_attention(0, normal(gen(0), 4, 8, 4, 128), torch.zeros(4, 8, 1, dtype=torch.int32, device="cuda") - 1,
                                         case.table, case.ctx, 0.1)
    assert case.pool.check_errors() == pkv.ERR_ROW
    assert torch.isfinite(out[[0, 1, 3]]).all()


def test_tree_attention_many_sequences():
    """More sequences than CTAs, some unused; a batch of 4096."""
    lens = [8 + (i * 37) % 90 if i % 7 else 0 for i in range(500)]
    run_tree(Case("bf16", 64, 1, lens, seed=1), 8, 2)
    case = Case("bf16", 64, 1, [9, 0, 40], seed=1)
    table = case.table.repeat(1366, 1)[:4096].contiguous()
    ctx = case.ctx.repeat(1366)[:4096].contiguous()
    q = normal(gen(0), 3, 2, 2, 64)
    mask = torch.full((2, 1), 3, dtype=torch.int32, device="cuda")
    out = case.pool.paged_tree_attention(0, q.repeat(1366, 1, 1, 1)[:4096].contiguous(), mask, table, ctx, 0.125)
    for b in range(3):
        assert (out[b::3] == out[b]).all()
    case.lens = [9, 0, 40]
    run_tree(case, 2, 2, q=q, mask=mask)


def test_tree_attention_streams_and_graphs():
    """A call on another stream; two captured graphs replayed at once."""
    case = Case("bf16", 128, 2, [1500, 900], seed=1)
    packed = Case("k8v8", 128, 2, [1500, 900], seed=1)
    q = normal(gen(0), 2, 10, 4, 128)
    mask = torch.from_numpy(pkv.tree_masks(random_tree(2, 10, 3))[0]).cuda()
    for c in (case, packed):
        call = lambda **kw: c.pool.paged_tree_attention(0, q, mask, c.table, c.ctx, 0.1, **kw)  # noqa: E731
        want = call()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        got = call(stream=s1)
        s1.synchronize()
        assert torch.equal(want, got)
        graphs = []
        for s in (s1, s2):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                call()
                gr = torch.cuda.CUDAGraph()
                with torch.cuda.graph(gr, stream=s):
                    o = call()
                graphs.append((gr, o, s))
        torch.cuda.synchronize()
        for gr, o, s in graphs:
            o.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            for gr, o, s in graphs:
                with torch.cuda.stream(s):
                    gr.replay()
        torch.cuda.synchronize()
        for gr, o, s in graphs:
            assert torch.equal(want, o)


def test_tree_attention_refusals():
    case = Case("bf16", 64, 2, [100, 50], seed=1)
    q = normal(gen(0), 2, 8, 4, 64)
    mask = torch.ones(2, 8, 1, dtype=torch.int32, device="cuda")
    ok = dict(layer=0, q=q, tree_mask=mask, block_table=case.table, ctx_lens=case.ctx, scale=0.1)
    call = lambda **kw: case.pool.paged_tree_attention(**{**ok, **kw})  # noqa: E731
    call()
    small = torch.empty(case.pool.tree_workspace_bytes(2, 8, 4) - 1, dtype=torch.uint8, device="cuda")
    shifted = torch.empty(case.pool.tree_workspace_bytes(2, 8, 4) + 512, dtype=torch.uint8, device="cuda")[16:]
    for kw in (dict(layer=1), dict(layer=-1), dict(scale=math.nan), dict(scale=math.inf), dict(scale=3e38),
               dict(q=normal(gen(0), 2, 8, 3, 64)), dict(workspace=small), dict(workspace=shifted)):
        with pytest.raises(pkv.PkvError) as e:
            call(**kw)
        assert e.value.status == pkv.PKV_ERR_INVALID
    for kw in (dict(q=q[0]), dict(tree_mask=mask[:1]), dict(tree_mask=mask.long()), dict(q=q.float()),
               dict(q=normal(gen(0), 2, 8, 4, 128)), dict(block_table=case.table[:1]), dict(ctx_lens=case.ctx[:1]),
               dict(q=q.transpose(1, 2)), dict(out=q[:1]), dict(tree_mask=torch.ones(2, 8, 2, dtype=torch.int32, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    with pytest.raises(pkv.PkvError):
        case.pool.tree_workspace_bytes(4097, 1, 2)
    with pytest.raises(pkv.PkvError):
        case.pool.tree_workspace_bytes(1, 1025, 2)
    assert call(q=q[:0], tree_mask=mask[:0], block_table=case.table[:0], ctx_lens=case.ctx[:0]).shape == (0, 8, 4, 64)
    latent = pkv.Pool(1, 1, 256, "latent", max_slabs=2)
    with pytest.raises(pkv.PkvError) as e:
        latent.tree_workspace_bytes(1, 1, 1)
    assert e.value.status == pkv.PKV_ERR_FORMAT


# ---------------------------------------------------------------------------
# accept_drafts
# ---------------------------------------------------------------------------
def fill_random(pool, rows, seed):
    rec = torch.randint(0, 256, (rows.numel(), pool.block_record_bytes()), generator=gen(seed), device="cuda").to(torch.uint8)
    pool.import_blocks(pool.config(), rows, rec)
    return rec


def moved(pool, rec, table, lens, n_q, paths):
    """The records after the accepted paths moved (host loops over bytes)."""
    out = rec.clone()
    L, Hk = pool.n_layers, pool.n_kv_heads
    at = 0
    per_layer = sum(32 * Hk * rb for rb in pool.row_bytes)
    tab = table.cpu().numpy()
    for layer in range(L):
        at = layer * per_layer
        for rb in pool.row_bytes:
            w = Hk * rb
            for b, p in enumerate(paths):
                first = lens[b] - n_q
                for k, j in enumerate(p):
                    s, d = first + j, first + k
                    out[tab[b, d // 32], at + d % 32 * w:at + (d % 32 + 1) * w] = \
                        rec[tab[b, s // 32], at + s % 32 * w:at + (s % 32 + 1) * w]
            at += 32 * w
    return out


@pytest.mark.parametrize("fmt,D,Hk,layers", [("bf16", 128, 8, 3), ("k4v4", 64, 1, 2), ("k4v4", 128, 8, 2), ("k8v8", 256, 4, 1),
                                             ("latent", 512, 1, 2), ("bf16", 64, 1, 1), ("k8v4", 128, 3, 2)])
def test_accept_drafts(fmt, D, Hk, layers):
    pool = pkv.Pool(layers, Hk, D, fmt, max_slabs=40, slab_blocks=7)
    n_q, lens = 70, [70, 101, 300, 0, 150, 96, 230]
    paths = [[0, 1, 2], [5, 9, 11, 40, 69], list(range(70)), [], [], [69], list(range(1, 70, 2))]
    need = [-(-x // 32) for x in lens]
    rows = torch.arange(sum(need), dtype=torch.int32, device="cuda")
    pool.reserve_rows(sum(need))
    order = torch.randperm(sum(need), generator=gen(1), device="cuda").int()
    table = torch.zeros(len(lens), max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, x in enumerate(need):
        table[b, :x] = order[at:at + x]
        at += x
    rec = fill_random(pool, rows, 2)
    path = torch.full((len(lens), 70), -5, dtype=torch.int32, device="cuda")
    for b, p in enumerate(paths):
        path[b, :len(p)] = i32(p)
    new = pool.accept_drafts(path, i32([len(p) for p in paths]), table, i32(lens), n_q)
    assert pool.check_errors() == 0
    assert new.tolist() == [x - n_q + len(p) if x else 0 for x, p in zip(lens, paths)]
    want = moved(pool, rec, table, lens, n_q, paths)
    assert torch.equal(pool.export_blocks(rows), want)


@pytest.mark.parametrize("path,n,word,new", [([3, 3, 4], 3, pkv.ERR_PATH, 92), ([4, 2, 5], 3, pkv.ERR_PATH, 92),
                                             ([0, 1, 8], 3, pkv.ERR_PATH, 92), ([-1, 1, 2], 3, pkv.ERR_PATH, 92),
                                             ([0, 1, 2], 4, pkv.ERR_PATH, 92), ([0, 1, 2], -1, pkv.ERR_PATH, 92),
                                             ([1, 2, 8], 2, 0, 94), ([7, 0, 0], 1, 0, 93)])
def test_accept_drafts_bad_paths(path, n, word, new):
    pool = make_pool("bf16", 2, 64, 32, layers=2)
    every = torch.arange(32, dtype=torch.int32, device="cuda")
    rec = fill_random(pool, every, 1)
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
    good = [2, 5, 7]
    p = i32([good, path, good])
    got = pool.accept_drafts(p, i32([3, n, 3]), table, i32([100, 100, 64]), 8)
    assert pool.check_errors() == word
    assert got.tolist() == [95, new, 59]
    want = moved(pool, rec, table, [100, 100, 64], 8, [good, [] if word else path[:n], good])
    assert torch.equal(pool.export_blocks(every), want)


def test_accept_drafts_lengths_and_rows_out_of_range():
    pool = make_pool("bf16", 2, 64, 32)
    every = torch.arange(32, dtype=torch.int32, device="cuda")
    rec = fill_random(pool, every, 1)
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
    p, n = i32([[2, 5]] * 3), i32([2, 2, 2])
    for bad in (-3, 5, 129):
        assert pool.accept_drafts(p, n, table, i32([0, bad, 0]), 8).tolist() == [0, 0, 0]
        assert pool.check_errors() == pkv.ERR_CTX
    table[1, 3] = 40
    pool.accept_drafts(p, n, table, i32([0, 104, 0]), 8)
    assert pool.check_errors() == pkv.ERR_ROW
    assert torch.equal(pool.export_blocks(every), rec)


def test_accept_drafts_refusals():
    pool = make_pool("bf16", 2, 64, 4)
    table, ctx = i32([[0, 1]]), i32([40])
    path, n = i32([[1]]), i32([1])
    for kw in (dict(n_q=0), dict(n_q=1025), dict(new_lens=ctx), dict(new_lens=n)):
        with pytest.raises(pkv.PkvError) as e:
            pool.accept_drafts(**{**dict(path=path, path_lens=n, block_table=table, ctx_lens=ctx, n_q=8), **kw})
        assert e.value.status == pkv.PKV_ERR_INVALID
    for kw in (dict(path=path[0]), dict(path=path.long()), dict(ctx_lens=i32([1, 2])), dict(block_table=table[0])):
        with pytest.raises((ValueError, TypeError)):
            pool.accept_drafts(**{**dict(path=path, path_lens=n, block_table=table, ctx_lens=ctx, n_q=8), **kw})
    none = i32([])
    assert pool.accept_drafts(none.view(0, 3), none, none.view(0, 2), none, 8).numel() == 0
    assert pool.accept_drafts(none.view(1, 0), i32([0]), table, ctx, 8).tolist() == [32]


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["bf16", "k4v4", "k8v8"])
def test_a_step_of_verification(fmt):
    """A prompt, a tree verified, its path accepted, and the next token decoded: as if the
    accepted tokens had been written one after another."""
    g = gen(11)
    B, n_q, Hk, Hq, D, L0 = 3, 13, 4, 8, 128, [70, 33, 128]
    tab = tables(400, D)
    pool, plain = (make_pool(fmt, Hk, D, 40) for _ in range(2))
    width = 8
    table = torch.from_numpy(pool.alloc_rows(B * width)).cuda().view(B, width)
    plain.alloc_rows(B * width)
    parents = random_tree(B, n_q, 5)
    masks, depths = pkv.tree_masks(parents)

    def place(b, t):
        return table[b, t // 32], t % 32

    def write(pool, where, k, v, pos, **kw):
        rows, slots = (torch.stack(x).int() for x in zip(*((r, torch.tensor(s, device="cuda")) for r, s in where)))
        return pool.write_rotated(0, rows, slots, k, v, i32(pos), tab, **kw)

    prompt = [(b, t) for b in range(B) for t in range(L0[b])]
    k, v = normal(g, len(prompt), Hk, D), normal(g, len(prompt), Hk, D)
    for p in (pool, plain):
        write(p, [place(*x) for x in prompt], k, v, [t for _, t in prompt])
    dk, dv, dq = normal(g, B, n_q, Hk, D), normal(g, B, n_q, Hk, D), normal(g, B, n_q, Hq, D)
    drafts = [(b, L0[b] + j) for b in range(B) for j in range(n_q)]
    pos = [L0[b] + int(depths[b, j]) for b in range(B) for j in range(n_q)]
    q = write(pool, [place(*x) for x in drafts], dk.flatten(0, 1), dv.flatten(0, 1), pos, q=dq.flatten(0, 1))
    ctx = i32([x + n_q for x in L0])
    out = pool.paged_tree_attention(0, q.view(B, n_q, Hq, D), torch.from_numpy(masks).cuda(), table, ctx, D ** -0.5)
    # the deepest token's path is accepted
    paths = []
    for b in range(B):
        j, path = int(depths[b].argmax()), []
        while j >= 0:
            path.append(j)
            j = int(parents[b, j])
        paths.append(path[::-1])
    most = max(map(len, paths))
    new = pool.accept_drafts(i32([p + [0] * (most - len(p)) for p in paths]), i32([len(p) for p in paths]), table, ctx, n_q)
    assert new.tolist() == [x + len(p) for x, p in zip(L0, paths)]
    # the same tokens, written in order
    for b, p in enumerate(paths):
        write(plain, [place(b, L0[b] + i) for i in range(len(p))], dk[b, p], dv[b, p], [L0[b] + i for i in range(len(p))])
    for b in range(B):
        L = int(new[b])
        for x, y in zip(pool.gather_visible(0, table[b].contiguous(), L), plain.gather_visible(0, table[b].contiguous(), L)):
            assert torch.equal(x, y)
        # the last accepted token's output is that of a decode of its prefix
        last = plain.paged_decode_attention(0, q.view(B, n_q, Hq, D)[b:b + 1, paths[b][-1]].contiguous(),
                                            table[b:b + 1].contiguous(), new[b:b + 1].contiguous(), D ** -0.5)
        got = out[b, paths[b][-1]].double()
        assert ((got - last[0].double()).norm() / got.norm()).item() < 1e-2
    nq = normal(g, B, Hq, D)
    assert torch.equal(pool.paged_decode_attention(0, nq, table, new, D ** -0.5),
                       plain.paged_decode_attention(0, nq, table, new, D ** -0.5))
    assert pool.check_errors() == 0 and plain.check_errors() == 0


def test_concurrent_writes_on_two_streams():
    """Two layers written from two streams at once."""
    g = gen(1)
    pool = make_pool("k8v8", 4, 128, 130, layers=2)
    n = 4096
    t = torch.arange(n, dtype=torch.int32, device="cuda")
    k, v = normal(g, 2, n, 4, 128), normal(g, 2, n, 4, 128)
    tab = tables(n, 128)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for layer, s in enumerate(streams):
        pool.write_rotated(layer, t // 32, t % 32, k[layer], v[layer], t, tab, stream=s)
    torch.cuda.synchronize()
    one = make_pool("k8v8", 4, 128, 130, layers=2)
    for layer in range(2):
        one.write_rotated(layer, t // 32, t % 32, k[layer], v[layer], t, tab)
    every = torch.arange(128, dtype=torch.int32, device="cuda")
    assert torch.equal(pool.export_blocks(every), one.export_blocks(every))
