"""The latent-pool operators through the C ABI: the cache write (norm, rotation, store),
the absorbed attention and the expanded attention, each against a plain statement of its
formula in 64 bits.

Tolerances count the roundings each operator documents (u = 2^-8 is half a bf16 step
relative to the value):
  write      one rounding of a value computed in fp32: u |y|, plus 2^-16 of the row's
             largest value for the fp32 steps (a few roundings of 2^-24 each, and the
             mean of squares of 512 values);
  absorbed   u |y| for the output, u sum p |c| for the probabilities' rounding, and
             2 d sum p |c| for the logits, d the fp32 error of a dot product of W terms,
             W 2^-23 scale sum |q k| (the bound of any summation order, truncating or not);
  expanded   u |y| for the output, 2 h sum p |v| for the probabilities' and the values'
             rounding to fp16 (h = 2^-11; values far below the largest of their 128 tokens
             lose at most 2^-25 of that), the logits as above, with the keys' rounding, u
             scale sum |q k|, inside d.
The elementwise bounds are worst cases; a relative L2 bound holds the average: each
rounding contributes at most u / sqrt(3) in the mean square, at most four of them with
logits of unit size, so 2 u < 1e-2."""
import ctypes
import math

import numpy as np
import pytest

import paged_kv_cache_split_gb300 as pkv

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -8
H16 = 2.0 ** -11
P, DH = 64, 128


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


def tables(n):
    f = 10000.0 ** (-torch.arange(P // 2, dtype=torch.float64, device="cuda") / (P // 2))
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat((a.cos(), a.sin()), 1).float()


class Case:
    """A one-layer (or more) pool whose sequences hold seeded rows in shuffled blocks.  Slots
    past a sequence's length hold `stale` bytes."""

    def __init__(self, lens, R=512, seed=0, extra=0, n_layers=1, layer=0, stale=0x7FC0, scale_kv=1.0, slab_blocks=32,
                 shuffle=True):
        g = gen(seed)
        self.lens, self.R, self.layer, self.W = list(lens), R, layer, R + P
        need = [-(-x // 32) for x in lens]
        n = max(1, sum(need))
        self.pool = pkv.Pool(n_layers, 1, R, "latent", rope_dim=P, max_slabs=n // slab_blocks + 4,
                             slab_blocks=slab_blocks)
        self.pool.reserve_rows(n + 3)
        self.rows = normal(g, n * 32, self.W)
        if scale_kv != 1.0:
            self.rows = (self.rows.float() * scale_kv).bfloat16()
        order = torch.randperm(n + 3, generator=g, device="cuda")[:n].int()
        if not shuffle:
            order = torch.arange(n, dtype=torch.int32, device="cuda")
        self.width = max(1, max(need) + extra)
        self.table = torch.full((len(lens), self.width), 0, dtype=torch.int32, device="cuda")
        blocks = torch.full((n, 32, self.W), 0, dtype=torch.bfloat16, device="cuda")
        blocks.view(torch.int16).fill_(stale if stale < 0x8000 else stale - 0x10000)
        self.seq = []
        at = 0
        for b, L in enumerate(lens):
            self.table[b, :need[b]] = order[at:at + need[b]]
            own = self.rows[at * 32:at * 32 + L]
            self.seq.append(own)
            blocks[at:at + need[b]].view(-1, self.W)[:L] = own
            at += need[b]
        rec = torch.zeros((n, n_layers, 32 * self.W * 2), dtype=torch.uint8, device="cuda")
        rec[:, layer] = blocks.view(torch.uint8).reshape(n, -1)
        self.pool.import_blocks(self.pool.config(), order, rec)
        self.ctx = i32(list(lens))


def softmax_ref(x, hidden):
    x = x.masked_fill(hidden, -math.inf)
    return torch.softmax(x, -1)


def hidden_for(n_q, L):
    return torch.ones(n_q, L, dtype=torch.bool, device="cuda").triu(L - n_q + 1)


def absorbed_ref(case, q, b, scale):
    """(out, tolerance) of sequence b, q [n_q, Hq, W]."""
    kv = case.seq[b].double()
    n_q, L = q.shape[0], case.lens[b]
    qd = q.double().transpose(0, 1)
    p = softmax_ref(qd @ kv.t() * scale, hidden_for(n_q, L))
    out = p @ kv[:, :case.R]
    mag = p @ kv[:, :case.R].abs()
    seen = (~hidden_for(n_q, L)).double()
    d = case.W * 2.0 ** -23 * scale * ((qd.abs() @ kv.abs().t()) * seen).amax(-1, keepdim=True)
    return out.transpose(0, 1), (U * out.abs() + (U + 2 * d) * mag + 1e-30).transpose(0, 1)


def expanded_ref(case, q, wk, wv, b, scale):
    kv = case.seq[b].double()
    n_q, L, H = q.shape[0], case.lens[b], q.shape[1]
    outs, tols = [], []
    for h in range(H):
        k = torch.cat((kv[:, :case.R] @ wk[h].double().t(), kv[:, case.R:]), 1)
        v = kv[:, :case.R] @ wv[h].double().t()
        qh = q[:, h].double()
        p = softmax_ref(qh @ k.t() * scale, hidden_for(n_q, L))
        seen = (~hidden_for(n_q, L)).double()
        d = (U + (DH + P) * 2.0 ** -23) * scale * ((qh.abs() @ k.abs().t()) * seen).amax(-1, keepdim=True)
        out, mag = p @ v, p @ v.abs()
        outs.append(out)
        tols.append(U * out.abs() + (2 * H16 + 2 * d) * mag + 2.0 ** -24 * v.abs().max() + 1e-30)
    return torch.stack(outs, 1), torch.stack(tols, 1)


def check(got, ref, tol, what):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst = (err / tol).max().item()
    assert worst <= 1, f"{what}: {worst:.2f} times the bound"
    rel = ((got.double() - ref).norm() / ref.norm().clamp_min(1e-300)).item()
    assert rel <= 1e-2, f"{what}: relative L2 {rel:.2e}"


def check_absorbed(case, out, q, scale, seqs=None):
    for b in (range(len(case.lens)) if seqs is None else seqs):
        if case.lens[b] == 0:
            assert not out[b].any()
        else:
            check(out[b], *absorbed_ref(case, q[b], b, scale), f"sequence {b} of {case.lens[b]}")


def absorbed(case, q, scale, **kw):
    return case.pool.paged_latent_attention(case.layer, q[..., :case.R], q[..., case.R:], case.table, case.ctx, scale,
                                            **kw)


SCALE = (DH + P) ** -0.5


# ---------------------------------------------------------------------------
# write
# ---------------------------------------------------------------------------
def write_ref(kv, R, pos, tab, w, eps, il, q):
    t = tab.double()[pos.long()]
    cos, sin = t[:, :P // 2], t[:, P // 2:]

    def turn(x, c, s):
        x = x.double()
        a, b = (x[..., 0::2], x[..., 1::2]) if il else (x[..., :P // 2], x[..., P // 2:])
        y0, y1 = a * c - b * s, a * s + b * c
        return torch.stack((y0, y1), -1).flatten(-2) if il else torch.cat((y0, y1), -1)

    c = kv[:, :R].double()
    if w is not None:
        c = c / (c.square().mean(1, keepdim=True) + eps).sqrt() * w.double()
    return torch.cat((c, turn(kv[:, R:], cos, sin)), 1), None if q is None else turn(q, cos[:, None], sin[:, None])


def write_tol(ref):
    return U * ref.abs() + 2.0 ** -16 * ref.abs().amax(-1, keepdim=True) + 1e-30


def pool_rows(pool, n_rows, W, layer=0):
    """[n_rows, 32, W] bf16 of one layer, read back through export_blocks."""
    rec = pool.export_blocks(torch.arange(n_rows, dtype=torch.int32, device="cuda"))
    per = 32 * W * 2
    return rec[:, layer * per:(layer + 1) * per].contiguous().view(torch.bfloat16).view(n_rows, 32, W)


@pytest.mark.parametrize("R", [256, 512])
@pytest.mark.parametrize("il", [True, False])
@pytest.mark.parametrize("n,H,norm", [(1, 1, True), (1, 0, False), (7, 16, True), (65, 33, False), (300, 128, True),
                                      (2000, 5, True)])
def test_write_matches_the_formula(R, il, n, H, norm):
    g = gen(R + n + H)
    W = R + P
    blocks = -(-n // 32) + 2
    pool = pkv.Pool(2, 1, R, "latent", max_slabs=blocks // 32 + 2)
    pool.reserve_rows(blocks)
    before = normal(g, blocks, 2, 32, W)
    pool.import_blocks(pool.config(), torch.arange(blocks, dtype=torch.int32, device="cuda"),
                       before.view(torch.uint8).reshape(blocks, -1))
    wide = normal(g, n, W + 40)
    kv = wide[:, 16:16 + W] * 1  # contiguous
    kv_view = wide[:, 16:16 + W]
    pos = torch.randint(0, 131072, (n,), generator=g, device="cuda").int()
    pos[0], pos[-1] = 0, 131071
    tab = tables(131072)
    w = (1 + 0.2 * normal(g, R)) if norm else None
    place = torch.randperm(blocks * 32, generator=g, device="cuda")[:n].int()
    rows, slots = place // 32, place % 32
    q = normal(g, n, H, DH + P)[..., DH:] if H else None
    got_q = pool.write_latent(1, rows, slots, kv_view, pos, tab, norm_weight=w, eps=1e-5, interleaved=il, q_rope=q)
    ref, qref = write_ref(kv, R, pos, tab, w, 1e-5, il, q)
    cache = pool_rows(pool, blocks, W, 1)
    got = cache.view(-1, W)[place.long()]
    assert ((got.double() - ref).abs() <= write_tol(ref)).all()
    if not norm:
        assert torch.equal(got[:, :R].view(torch.int16), kv[:, :R].contiguous().view(torch.int16))
    if H:
        assert ((got_q.double() - qref).abs() <= write_tol(qref)).all()
    else:
        assert got_q is None
    untouched = torch.ones(blocks * 32, dtype=torch.bool, device="cuda")
    untouched[place.long()] = False
    assert torch.equal(cache.view(-1, W)[untouched], before[:, 1].reshape(-1, W)[untouched])
    assert torch.equal(pool_rows(pool, blocks, W, 0), before[:, 0])
    assert pool.check_errors() == 0


@pytest.mark.parametrize("il", [True, False])
def test_write_turns_queries_in_place(il):
    g = gen(5)
    n, H = 9, 20
    pool = pkv.Pool(1, 1, 512, "latent", max_slabs=2)
    pool.reserve_rows(2)
    full = normal(g, n, H, DH + P)
    q0 = full.clone()
    kv, pos, tab = normal(g, n, 576), torch.arange(100, 100 + n, device="cuda").int(), tables(256)
    place = torch.arange(n, device="cuda").int()
    out = pool.write_latent(0, place // 32, place % 32, kv, pos, tab, interleaved=il, q_rope=full[..., DH:],
                            q_out=full[..., DH:])
    _, ref = write_ref(kv, 512, pos, tab, None, 0, il, q0[..., DH:])
    assert out.data_ptr() == full[..., DH:].data_ptr()
    assert ((full[..., DH:].double() - ref).abs() <= write_tol(ref)).all()
    assert torch.equal(full[..., :DH], q0[..., :DH])


def test_write_extreme_values():
    """Zero rows (the norm's epsilon alone), rows of 2^60 (no: their squares pass fp32) and
    infinities: what the formula gives in fp32, and no other token is touched."""
    g = gen(6)
    pool = pkv.Pool(1, 1, 256, "latent", max_slabs=2)
    pool.reserve_rows(1)
    kv = normal(g, 5, 320)
    kv[0] = 0
    kv[1] *= 2.0 ** -60
    kv[2] *= 2.0 ** 50
    kv[3, 7] = math.inf
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    s = torch.arange(5, device="cuda").int()
    pool.write_latent(0, s * 0, s, kv, s, tables(8), norm_weight=w, eps=1e-6)
    got = pool_rows(pool, 1, 320)[0]
    assert not got[0, :256].any()
    ref, _ = write_ref(kv, 256, s, tables(8), w, 1e-6, True, None)
    for i in (1, 2, 4):
        assert ((got[i].double() - ref[i]).abs() <= write_tol(ref)[i]).all()
    assert torch.isnan(got[3, 7]) and torch.isfinite(got[3, 256:]).all()


def test_write_flags_bad_rows_slots_and_positions():
    g = gen(7)
    pool = pkv.Pool(1, 1, 512, "latent", max_slabs=1)
    pool.reserve_rows(32)
    tab = tables(16)
    kv, q = normal(g, 3, 576), normal(g, 3, 2, P)
    for rows, slots, pos, bit, skipped_q in [([0, 32, 1], [0, 0, 0], [1, 1, 1], pkv.ERR_ROW, False),
                                             ([0, -1, 1], [0, 0, 0], [1, 1, 1], pkv.ERR_ROW, False),
                                             ([0, 2, 1], [0, 32, 0], [1, 1, 1], pkv.ERR_SLOT, False),
                                             ([0, 2, 1], [0, -1, 0], [1, 1, 1], pkv.ERR_SLOT, False),
                                             ([0, 2, 1], [0, 0, 0], [1, 16, 1], pkv.ERR_POS, True),
                                             ([0, 2, 1], [0, 0, 0], [1, -1, 1], pkv.ERR_POS, True)]:
        clear = torch.zeros((32, 32 * 576 * 2), dtype=torch.uint8, device="cuda")
        pool.import_blocks(pool.config(), torch.arange(32, dtype=torch.int32, device="cuda"), clear)
        qo = torch.full((3, 2, P), 9.0, dtype=torch.bfloat16, device="cuda")
        pool.write_latent(0, i32(rows), i32(slots), kv, i32(pos), tab, q_rope=q, q_out=qo)
        assert pool.check_errors() == bit
        ref, qref = write_ref(kv, 512, i32([1, 1, 1]), tab, None, 0, True, q)
        got = pool_rows(pool, 32, 576)
        for r, i in ((0, 0), (1, 2)):
            assert ((got[r, 0].double() - ref[i]).abs() <= write_tol(ref)[i]).all()
        got[0, 0], got[1, 0] = 0, 0
        assert not got.any(), "a bad token was written somewhere"
        for i in (0, 2):
            assert ((qo[i].double() - qref[i]).abs() <= write_tol(qref)[i]).all()
        if skipped_q:
            assert (qo[1] == 9).all()
        else:
            assert ((qo[1].double() - qref[1]).abs() <= write_tol(qref)[1]).all()


# ---------------------------------------------------------------------------
# absorbed
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("R", [256, 512])
@pytest.mark.parametrize("H", [1, 3, 8, 16, 20, 64, 65, 128])
def test_absorbed_heads(R, H):
    case = Case([1, 31, 0, 64, 65, 700], R, seed=H)
    q = normal(gen(H), 6, 1, H, R + P)
    out = absorbed(case, q, SCALE)
    assert out.shape == (6, 1, H, R)
    check_absorbed(case, out, q, SCALE)
    three = case.pool.paged_latent_attention(0, q[:, 0, :, :R], q[:, 0, :, R:], case.table, case.ctx, SCALE)
    assert torch.equal(three, out[:, 0])
    assert case.pool.check_errors() == 0


@pytest.mark.parametrize("R", [256, 512])
@pytest.mark.parametrize("n_q,H", [(2, 16), (3, 5), (4, 16), (5, 128), (8, 1), (33, 3), (70, 2)])
def test_absorbed_several_queries(R, n_q, H):
    case = Case([n_q, n_q + 1, 200, 0, 64 * 5 + n_q, 95], R, seed=n_q)
    q = normal(gen(H), 6, n_q, H, R + P)
    check_absorbed(case, absorbed(case, q, SCALE), q, SCALE)
    assert case.pool.check_errors() == 0


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 191, 192, 193, 257])
def test_absorbed_lengths(L):
    case = Case([L], 512, seed=L, extra=2)
    q = normal(gen(L), 1, 1, 24, 576)
    check_absorbed(case, absorbed(case, q, SCALE), q, SCALE)
    assert case.pool.check_errors() == 0


@pytest.mark.parametrize("stale", [0x7FC0, 0x7F80, 0xFF80, 0x7F7F])
@pytest.mark.parametrize("n_q", [1, 3])
def test_stale_slots_never_reach_an_output(stale, n_q):
    """NaN, both infinities and the largest value in the slots past each length."""
    case = Case([5, 40, 70, 97, 128], 512, seed=3, stale=stale)
    q = normal(gen(1), 5, n_q, 16, 576)
    check_absorbed(case, absorbed(case, q, SCALE), q, SCALE)
    wk, wv = normal(gen(2), 16, DH, 512) / 22, normal(gen(3), 16, DH, 512) / 22
    qe = normal(gen(4), 5, n_q, 16, DH + P)
    out = case.pool.latent_prefill_attention(0, qe, wk, wv, case.table, case.ctx, SCALE)
    for b in range(5):
        check(out[b], *expanded_ref(case, qe[b], wk, wv, b, SCALE), f"sequence {b}")


def test_absorbed_split_counts_and_repeats():
    """Results agree with the formula for every number of CTAs, and repeats are bit-identical."""
    rng = np.random.default_rng(1)
    lens = [int(x) if rng.random() > 0.2 else 0 for x in rng.integers(1, 400, size=40)] + [3001]
    case = Case(lens, 512, seed=11)
    for n_q, H in ((1, 16), (1, 128)):
        q = normal(gen(12), 41, n_q, H, 576)
        for ctas in (1, 2, 5, 37, 0, 400):
            case.pool.decode_set_ctas(ctas)
            a = absorbed(case, q, SCALE)
            assert torch.equal(a, absorbed(case, q, SCALE))
            check_absorbed(case, a, q, SCALE, seqs=None if ctas in (0, 5) else [0, 7, 39, 40])
    assert case.pool.check_errors() == 0


def test_absorbed_one_long_sequence():
    case = Case([70001], 512, seed=13, slab_blocks=512)
    q = normal(gen(14), 1, 1, 16, 576)
    check_absorbed(case, absorbed(case, q, SCALE), q, SCALE)
    assert case.pool.check_errors() == 0


@pytest.mark.parametrize("order", ["rising", "falling", "spike"])
def test_absorbed_running_maximum(order):
    """Logits that rise by hundreds along the sequence (every tile raises the maximum), fall,
    or have one token far above the rest."""
    L = 1000
    case = Case([L], 512, seed=15)
    q = normal(gen(16), 1, 1, 16, 576)
    # every head's query shares a direction; row t carries t (or L - t) steps along it
    d = torch.zeros(576, device="cuda")
    d[:8] = 1.0
    ramp = torch.arange(L, device="cuda").float() * 0.6
    if order == "falling":
        ramp = ramp.flip(0)
    if order == "spike":
        ramp = torch.zeros(L, device="cuda")
        ramp[611] = 500.0
    rows = (case.seq[0].float() + ramp[:, None] * d).bfloat16()
    case.seq[0] = rows
    q[..., :8] = 1.0
    tok = torch.arange(L, device="cuda")
    case.pool.write_latent(0, case.table[0][(tok // 32).long()], (tok % 32).int(), rows, tok.int() * 0,
                           torch.cat((torch.ones(1, 32), torch.zeros(1, 32)), 1).cuda())
    for ctas in (1, 0):
        case.pool.decode_set_ctas(ctas)
        check_absorbed(case, absorbed(case, q, SCALE), q, SCALE)


@pytest.mark.parametrize("e", [-30, -8, 8])
def test_absorbed_magnitudes(e):
    """Latents scaled by 2^e with the logits kept (the scale divided by 2^e)."""
    case = Case([33, 300], 512, seed=17, scale_kv=2.0 ** e)
    q = normal(gen(18), 2, 1, 16, 576)
    s = SCALE * 2.0 ** -e
    check_absorbed(case, absorbed(case, q, s), q, s)


def test_absorbed_zero_and_negative_scale():
    case = Case([33, 300], 256, seed=19)
    q = normal(gen(20), 2, 2, 16, 320)
    for s in (0.0, -0.05):
        out = absorbed(case, q, s)
        for b in range(2):
            ref, tol = absorbed_ref(case, q[b], b, s)
            check(out[b], ref, tol + 2 * absorbed_ref(case, q[b], b, -s)[1], f"scale {s}")


def test_absorbed_separate_and_strided_queries():
    case = Case([100, 37], 512, seed=21)
    base = normal(gen(22), 2, 3, 16, 576)
    ref = absorbed(case, base, SCALE)
    ql = torch.zeros(2, 3, 16, 520, dtype=torch.bfloat16, device="cuda")
    ql[..., :512] = base[..., :512]
    qr = torch.zeros(2, 3, 16, DH + P, dtype=torch.bfloat16, device="cuda")
    qr[..., DH:] = base[..., 512:]
    out = case.pool.paged_latent_attention(0, ql[..., :512], qr[..., DH:], case.table, case.ctx, SCALE)
    assert torch.equal(out, ref)
    with pytest.raises(ValueError):  # rows not evenly spaced
        case.pool.paged_latent_attention(0, base.transpose(0, 1)[:2, :2, :, :512], base[:, :2, :, 512:], case.table,
                                         case.ctx, SCALE)


@pytest.mark.parametrize("call", ["absorbed", "expanded"])
def test_bad_lengths_and_rows(call):
    lens = [40, 50, 60, 10, 70]
    case = Case(lens, 512, seed=23)
    n_q, H = 4, 8
    q = normal(gen(24), 5, n_q, H, 576)
    qe = normal(gen(25), 5, n_q, H, DH + P)
    wk, wv = normal(gen(26), H, DH, 512) / 22, normal(gen(27), H, DH, 512) / 22

    def run(table, ctx):
        if call == "absorbed":
            return case.pool.paged_latent_attention(0, q[..., :512], q[..., 512:], table, ctx, SCALE)
        return case.pool.latent_prefill_attention(0, qe, wk, wv, table, ctx, SCALE)

    good = run(case.table, case.ctx)
    assert case.pool.check_errors() == 0
    for bad in (-1, 3, case.width * 32 + 1, -2 ** 31, 2 ** 31 - 1):
        ctx = case.ctx.clone()
        ctx[1] = bad
        out = run(case.table, ctx)
        assert case.pool.check_errors() == pkv.ERR_CTX
        assert not out[1].any()
        for b in (0, 2, 3, 4):
            assert torch.allclose(out[b].float(), good[b].float(), rtol=2 ** -6, atol=2 ** -6)
    for bad in (-1, 10 ** 6, 2 ** 31 - 1):
        table = case.table.clone()
        table[2, 1] = bad
        out = run(table, case.ctx)
        assert case.pool.check_errors() == pkv.ERR_ROW
        for b in (0, 1, 3, 4):
            assert torch.allclose(out[b].float(), good[b].float(), rtol=2 ** -6, atol=2 ** -6)
    # table entries past a sequence's blocks are never read as rows
    table = case.table.clone()
    table[3, 1:] = -7
    run(table, case.ctx)
    assert case.pool.check_errors() == 0


@pytest.mark.parametrize("call", ["absorbed", "expanded"])
def test_streams_and_graphs(call):
    """Another stream; two captured graphs replayed in turn and at once; new lengths and
    rows in the captured buffers."""
    case = Case([300, 45, 128], 512, seed=29, extra=1)
    H, n_q = 16, 2
    q = normal(gen(30), 3, n_q, H, 576)
    qe = normal(gen(31), 3, n_q, H, DH + P)
    wk, wv = normal(gen(32), H, DH, 512) / 22, normal(gen(33), H, DH, 512) / 22

    def run(**kw):
        if call == "absorbed":
            return absorbed(case, q, SCALE, **kw)
        return case.pool.latent_prefill_attention(0, qe, wk, wv, case.table, case.ctx, SCALE, **kw)

    ref = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = run()
    b = run(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a, ref) and torch.equal(b, ref)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    for g, out in graphs:
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert torch.equal(out, ref)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        for (g, _), st in zip(graphs, (s1, s2)):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert torch.equal(out, ref)
    case.ctx.copy_(i32([77, 45, 0]))
    want = run()
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], want) and not want[2].any()
    assert case.pool.check_errors() == 0


def test_rows_past_32_bits():
    """More than 2^31 query and output values in one call."""
    B, n_q, H, R = 64, 66, 1000, 512
    case = Case([70] * B, R, seed=35)
    q = torch.zeros(B, n_q, H, R + P, dtype=torch.bfloat16, device="cuda")
    assert q.numel() > 2 ** 31 and B * n_q * H * R > 2 ** 31
    some = [(0, 0), (63, 0), (63, n_q - 1)]
    for b, i in some:
        q[b, i] = normal(gen(b + i), H, R + P)
    out = absorbed(case, q, SCALE)
    for b, i in some:
        ref, tol = _one_query(case, q[b, i], b, 70 - n_q + i + 1)
        check(out[b, i], ref, tol, f"({b}, {i})")


def _one_query(case, q, b, vis):
    kv = case.seq[b][:vis].double()
    p = torch.softmax(q.double() @ kv.t() * SCALE, -1)
    out, mag = p @ kv[:, :case.R], p @ kv[:, :case.R].abs()
    d = case.W * 2.0 ** -23 * SCALE * (q.double().abs() @ kv.abs().t()).amax(-1, keepdim=True)
    return out, U * out.abs() + (U + 2 * d) * mag + 1e-30


def test_second_layer_and_large_slabs():
    case = Case([500, 33], 512, seed=37, n_layers=3, layer=2, slab_blocks=4)
    q = normal(gen(38), 2, 1, 16, 576)
    check_absorbed(case, absorbed(case, q, SCALE), q, SCALE)


# ---------------------------------------------------------------------------
# expanded
# ---------------------------------------------------------------------------
def expanded_check(case, n_q, H, seed=0, scale=SCALE, max_ctx=0, factor=1.0):
    B, R = len(case.lens), case.R
    g = gen(seed + 100)
    q = normal(g, B, n_q, H, DH + P)
    wk = (normal(g, H, DH, R).float() * R ** -0.5 * factor).bfloat16()
    wv = (normal(g, H, DH, R).float() * R ** -0.5 * factor).bfloat16()
    out = case.pool.latent_prefill_attention(case.layer, q, wk, wv, case.table, case.ctx, scale, max_ctx=max_ctx)
    assert out.shape == (B, n_q, H, DH)
    for b in range(B):
        if case.lens[b] == 0:
            assert not out[b].any()
        else:
            check(out[b], *expanded_ref(case, q[b], wk, wv, b, scale), f"sequence {b} of {case.lens[b]}")
    assert case.pool.check_errors() == 0
    return out


@pytest.mark.parametrize("R", [256, 512])
@pytest.mark.parametrize("n_q,H,lens", [
    (1, 1, [1]), (1, 3, [1, 0, 33, 500]), (5, 2, [5, 6, 130]), (31, 4, [31, 64, 0]), (64, 1, [64, 65]),
    (100, 4, [100]), (127, 2, [127, 300]), (128, 2, [128, 129]), (129, 3, [129, 700]), (200, 16, [200, 1000, 333]),
    (256, 2, [256, 257]), (257, 1, [257, 511, 512, 513]), (700, 5, [700, 1500]), (1025, 2, [1025, 2050])])
def test_expanded(R, n_q, H, lens):
    expanded_check(Case(lens, R, seed=n_q), n_q, H, seed=H)


@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 63, 65, 96, 127, 128, 129, 160, 191, 193, 255, 256, 257, 384, 385])
def test_expanded_lengths(L):
    expanded_check(Case([L], 512, seed=L, extra=3), L, 2, seed=L)
    expanded_check(Case([L], 512, seed=L, extra=3), 1, 2, seed=L, max_ctx=L)


@pytest.mark.parametrize("ctas", [1, 7, 40, 152, 400])
@pytest.mark.parametrize("n_q,H,lens", [(1, 1, [5000]), (3, 2, [4100, 4, 2000]), (300, 1, [3000, 301, 0]),
                                        (129, 3, [1025])])
def test_expanded_split_over_the_context(ctas, n_q, H, lens):
    """Every number of parts the launch may choose, some of them past a sequence's last tile;
    repeats are bit-identical."""
    case = Case(lens, 512, seed=n_q + H)
    case.pool.decode_set_ctas(ctas)
    a = expanded_check(case, n_q, H, seed=ctas)
    assert torch.equal(a, expanded_check(case, n_q, H, seed=ctas))


def test_expanded_many_heads_and_a_long_context():
    expanded_check(Case([5000], 512, seed=41), 140, 40, max_ctx=5000)


@pytest.mark.parametrize("order", ["rising", "falling"])
def test_expanded_running_maximum(order):
    """Position keys that raise (lower) the logits by hundreds along the sequence."""
    L, n_q, H = 900, 300, 2
    case = Case([L], 512, seed=43)
    ramp = torch.arange(L, device="cuda").float() * 0.5
    rows = case.seq[0].clone()
    rows[:, 512:520] = (ramp if order == "rising" else ramp.flip(0))[:, None].bfloat16()
    case.seq[0] = rows
    tok = torch.arange(L, device="cuda")
    case.pool.write_latent(0, case.table[0][(tok // 32).long()], (tok % 32).int(), rows, tok.int() * 0,
                           torch.cat((torch.ones(1, 32), torch.zeros(1, 32)), 1).cuda())
    g = gen(44)
    q = normal(g, 1, n_q, H, DH + P)
    q[..., DH:DH + 8] = 1.0
    wk, wv = normal(g, H, DH, 512) / 22, normal(g, H, DH, 512) / 22
    out = case.pool.latent_prefill_attention(0, q, wk, wv, case.table, case.ctx, SCALE)
    ref, tol = expanded_ref(case, q[0], wk, wv, 0, SCALE)
    assert ((out[0].double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("factor", [2.0 ** -20, 2.0 ** 6])
def test_expanded_magnitudes(factor):
    """Projections scaled by a power of two, the logits' scale divided by it."""
    case = Case([50, 200], 512, seed=45)
    rows = [s.clone() for s in case.seq]
    for s in rows:
        s[:, 512:] = 0  # the position part does not scale with the projections
    tok = [torch.arange(len(s), device="cuda") for s in rows]
    one = torch.cat((torch.ones(1, 32), torch.zeros(1, 32)), 1).cuda()
    for b, s in enumerate(rows):
        case.pool.write_latent(0, case.table[b][(tok[b] // 32).long()], (tok[b] % 32).int(), s, tok[b].int() * 0, one)
        case.seq[b] = s
    expanded_check(case, 50, 4, scale=SCALE / factor, factor=factor)


@pytest.mark.parametrize("scale", [0.0, -0.05])
def test_expanded_zero_and_negative_scale(scale):
    case, n_q, H = Case([40, 300], 512, seed=49), 40, 3
    g = gen(51)
    q = normal(g, 2, n_q, H, DH + P)
    wk, wv = normal(g, H, DH, 512) / 22, normal(g, H, DH, 512) / 22
    out = case.pool.latent_prefill_attention(0, q, wk, wv, case.table, case.ctx, scale)
    for b in range(2):
        ref, tol = expanded_ref(case, q[b], wk, wv, b, scale)
        _, room = expanded_ref(case, q[b], wk, wv, b, abs(scale))  # the bounds count |scale|
        err = (out[b].double() - ref).abs()
        assert (err <= torch.maximum(tol, tol.clamp_min(0) + 2 * room)).all()


@pytest.mark.parametrize("x", [1e29, -1e31, 2e37])
def test_logits_near_the_end_of_fp32(x):
    """Every logit the same huge value (an equal softmax), through the position part alone."""
    case = Case([100], 512, seed=52)
    rows = case.seq[0].clone()
    rows[:, 512:] = 0
    rows[:, 512] = 2.0 ** 60
    tok = torch.arange(100, device="cuda")
    one = torch.cat((torch.ones(1, 32), torch.zeros(1, 32)), 1).cuda()
    case.pool.write_latent(0, case.table[0][(tok // 32).long()], (tok % 32).int(), rows, tok.int() * 0, one)
    q = torch.zeros(1, 1, 4, 576, dtype=torch.bfloat16, device="cuda")
    q[..., 512] = x / 2.0 ** 60
    want = rows[:, :512].double().mean(0)
    for ctas in (0, 1):
        case.pool.decode_set_ctas(ctas)
        out = case.pool.paged_latent_attention(0, q[..., :512], q[..., 512:], case.table, case.ctx, 1.0)
        assert ((out[0, 0].double() - want).abs() <= U * want.abs() + U * rows[:, :512].double().abs().mean(0)).all()
    wv = torch.zeros(4, 128, 512, dtype=torch.bfloat16, device="cuda")
    wv[:, torch.arange(128), torch.arange(128)] = 1
    qe = torch.zeros(1, 1, 4, 192, dtype=torch.bfloat16, device="cuda")
    qe[..., 128] = x / 2.0 ** 60
    out = case.pool.latent_prefill_attention(0, qe, wv, wv, case.table, case.ctx, 1.0)
    assert ((out[0, 0].double() - want[:128]).abs() <=
            U * want[:128].abs() + 2 * U * rows[:, :128].double().abs().mean(0)).all()


@pytest.mark.parametrize("e", [-12, 12])
def test_expanded_values_of_mixed_magnitudes(e):
    """The first 200 tokens' latents 2^e times the others', and queries that look at either
    part alone (through the position keys)."""
    L, n_q, H = 700, 6, 2
    case = Case([L], 512, seed=53)
    rows = case.seq[0].clone()
    rows[:200, :512] = (rows[:200, :512].float() * 2.0 ** e).bfloat16()
    rows[:, 512:] = 0
    rows[:200, 512] = 1
    rows[200:, 513] = 1
    tok = torch.arange(L, device="cuda")
    one = torch.cat((torch.ones(1, 32), torch.zeros(1, 32)), 1).cuda()
    case.pool.write_latent(0, case.table[0][(tok // 32).long()], (tok % 32).int(), rows, tok.int() * 0, one)
    g = gen(54)
    wv = normal(g, H, DH, 512) / 22
    wk = torch.zeros_like(wv)
    q = torch.zeros(1, n_q, H, DH + P, dtype=torch.bfloat16, device="cuda")
    q[:, ::2, :, DH] = 400
    q[:, 1::2, :, DH + 1] = 400
    for ctas in (0, 1):
        case.pool.decode_set_ctas(ctas)
        out = case.pool.latent_prefill_attention(0, q, wk, wv, case.table, case.ctx, 1.0)
        kv = rows.double()
        for i in range(n_q):
            part = kv[:200] if i % 2 == 0 else kv[200:L - n_q + i + 1]
            for h in range(H):
                v = part[:, :512] @ wv[h].double().t()
                want = v.mean(0)
                tol = U * want.abs() + 2 * H16 * v.abs().mean(0) + 2.0 ** -24 * v.abs().max()
                assert ((out[0, i, h].double() - want).abs() <= tol).all(), (i, h, ctas)


def test_expanded_context_beyond_its_bound():
    case = Case([64, 90], 512, seed=47)
    g = gen(48)
    q, w = normal(g, 2, 2, 4, DH + P), normal(g, 4, DH, 512) / 22
    full = case.pool.latent_prefill_attention(0, q, w, w, case.table, case.ctx, SCALE)
    out = case.pool.latent_prefill_attention(0, q, w, w, case.table, case.ctx, SCALE, max_ctx=89)
    assert case.pool.check_errors() == pkv.ERR_CTX
    assert not out[1].any()
    check(out[0], *expanded_ref(case, q[0], w, w, 0, SCALE), "the other sequence")
    assert torch.isfinite(full).all()


# ---------------------------------------------------------------------------
# together, and the pool's other operations on latent rows
# ---------------------------------------------------------------------------
def test_prompt_then_decode_steps():
    """A layer of a model: prompts are written and attended in expanded form; then tokens are
    decoded one by one, each written first, in absorbed form, with a shared prefix made
    private by copy-on-write.  Every output is compared with attention in 64 bits over
    the rows as the formulas give them (rounded once to bf16, as they are stored)."""
    R, H = 512, 8
    g = gen(50)
    pool = pkv.Pool(1, 1, R, "latent", max_slabs=4)
    w = (1 + 0.1 * normal(g, R))
    wk, wv = normal(g, H, DH, R) / 22, normal(g, H, DH, R) / 22
    tab = tables(512)
    L0, steps = 77, 5
    rows = pool.alloc_rows(3)
    table = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    table[0, :3] = torch.from_numpy(rows).cuda()
    t = torch.arange(L0, device="cuda")
    kv = normal(g, L0, R + P)
    q = normal(g, 1, L0, H, DH + P)
    qin = q[0].clone()
    pool.write_latent(0, table[0][(t // 32).long()], (t % 32).int(), kv, t.int(), tab, norm_weight=w,
                      q_rope=q[0, :, :, DH:], q_out=q[0, :, :, DH:])
    stored, qref = write_ref(kv, R, t, tab, w, 1e-6, True, qin[..., DH:])
    stored = stored.bfloat16()

    class Seq:
        pass

    def view(lens, seqs):
        c = Seq()
        c.lens, c.seq, c.R, c.W = lens, seqs, R, R + P
        return c

    out = pool.latent_prefill_attention(0, q, wk, wv, table[:1], i32([L0]), SCALE)
    qr = torch.cat((qin[..., :DH], qref.bfloat16()), -1)
    check(out[0], *_loose(expanded_ref(view([L0], [stored]), qr, wk, wv, 0, SCALE)), "prompt")
    # the same prompt's last queries in absorbed form agree with the expanded form
    ql = torch.einsum("ihd,hdr->ihr", q[0, -3:, :, :DH].double(), wk.double()).bfloat16().contiguous()
    a = pool.paged_latent_attention(0, ql[None], q[:, -3:, :, DH:], table[:1], i32([L0]), SCALE)
    av = torch.einsum("ihr,hdr->ihd", a[0].double(), wv.double())
    assert (av - out[0, -3:].double()).norm() / av.norm() < 3e-2
    # a second sequence shares the prefix: its last, partial block becomes its own
    for r in rows:
        pool.retain_row(int(r))
    fresh = pool.alloc_rows(1)
    pool.copy_on_write_block(i32([int(rows[2])]), i32([int(fresh[0])]))
    pool.release_row(int(rows[2]))
    table[1, :2], table[1, 2] = table[0, :2], int(fresh[0])
    seqs = [stored.clone(), stored.clone()]
    for step in range(steps):
        n = L0 + step
        kv, ql = normal(g, 2, R + P), normal(g, 2, H, R + P)
        pos = i32([n, n])
        rws = table[torch.arange(2, device="cuda"), n // 32].contiguous()
        qi = ql.clone()
        pool.write_latent(0, rws, i32([n % 32] * 2), kv, pos, tab, norm_weight=w, q_rope=ql[..., R:],
                          q_out=ql[..., R:])
        new, qref = write_ref(kv, R, pos, tab, w, 1e-6, True, qi[..., R:])
        seqs = [torch.cat((s, new[b:b + 1].bfloat16())) for b, s in enumerate(seqs)]
        out = pool.paged_latent_attention(0, ql[..., :R], ql[..., R:], table, i32([n + 1] * 2), SCALE)
        c = view([n + 1] * 2, seqs)
        full = torch.cat((qi[..., :R], qref.bfloat16()), -1)
        for b in range(2):
            check(out[b:b + 1], *_loose(absorbed_ref(c, full[b][None], b, SCALE)), f"step {step} sequence {b}")
    got = pool.gather_visible(0, table[1], L0 + steps)
    assert len(got) == 1
    assert ((got[0].view(torch.bfloat16)[0].double() - seqs[1].double()).abs() <=
            2 * write_tol(seqs[1].double())).all()
    assert pool.check_errors() == 0


def _loose(rt):
    """A stored value computed in fp32 may round to the neighbour of the 64-bit value's
    rounding: one more u of the rows and of the queries, in the output and in the logits
    (of size about sqrt(W) scale in these seeds, below 2)."""
    ref, tol = rt
    return ref, 3 * tol + 6 * U * ref.abs().amax()


def test_records_identity_and_stats():
    a = Case([100, 40], 256, seed=60)
    assert a.pool.stats()["n_kinds"] == 1 and a.pool.row_bytes == [640]
    assert a.pool.block_record_bytes() == 32 * 640
    rec = a.pool.export_blocks(a.table[0, :4].contiguous())
    b = pkv.Pool(1, 1, 256, "latent", max_slabs=2, hadamard_seed=9)
    rows = b.alloc_rows(4)
    b.import_blocks(a.pool.config(), i32([int(r) for r in rows]), rec)
    bt = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    bt[0] = torch.from_numpy(rows).cuda()
    q = normal(gen(61), 1, 1, 16, 320)
    assert torch.equal(b.paged_latent_attention(0, q[..., :256], q[..., 256:], bt, i32([100]), SCALE),
                       a.pool.paged_latent_attention(0, q[..., :256], q[..., 256:], a.table[:1], i32([100]), SCALE))
    assert not a.pool.check_identity(pkv.make_config(1, 1, 512, "latent", group_size=64))
    assert not a.pool.check_identity(pkv.make_config(1, 1, 256, "bf16"))
    price = a.pool.price_request(40, 4, 16, n_q=2, max_blocks=10)
    assert price["workspace_bytes"] == a.pool.latent_workspace_bytes(4, 2, 16)
    assert price["fixed_bytes"] == 44 + 2 * 16 * (320 + 256) * 2
    assert price["page_bytes"] == 40 * 32 * 640


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def test_configurations_refused():
    for kw in (dict(n_kv_heads=2, head_dim=512), dict(n_kv_heads=1, head_dim=128), dict(n_kv_heads=1, head_dim=576)):
        with pytest.raises(pkv.PkvError) as e:
            pkv.Pool(1, format="latent", **kw)
        assert e.value.status == pkv.PKV_ERR_INVALID
    with pytest.raises(pkv.PkvError):
        pkv.Pool(1, 1, 512, "latent", rope_dim=32)
    with pytest.raises(ValueError):
        pkv.Pool(1, 1, 128, "bf16", rope_dim=64)


def test_calls_of_the_other_formats_refused():
    p = pkv.Pool(1, 1, 512, "latent", max_slabs=2)
    p.reserve_rows(2)
    z = i32([0])
    kv = torch.zeros(1, 1, 512, dtype=torch.bfloat16, device="cuda")
    bt = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    for call in (lambda: p.write_block(0, z, z, kv, kv), lambda: p.paged_decode_attention(0, kv, bt, z, 0.1),
                 lambda: p.paged_decode_attention_noalloc(0, kv, bt, z, 0.1),
                 lambda: p.paged_prefill_attention(0, kv[None], bt, z, 0.1), lambda: p.decode_workspace_bytes(1, 1)):
        with pytest.raises(pkv.PkvError) as e:
            call()
        assert e.value.status == pkv.PKV_ERR_FORMAT
    b = pkv.Pool(1, 1, 128, "bf16", max_slabs=2)
    b.reserve_rows(2)
    q = torch.zeros(1, 4, 576, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: b.write_latent(0, z, z, q[:, 0], z, tables(2)),
                 lambda: b.paged_latent_attention(0, q[..., :512], q[..., 512:], bt, z, 0.1),
                 lambda: b.latent_prefill_attention(0, q[None], q, q, bt, z, 0.1),
                 lambda: b.latent_workspace_bytes(1, 1, 1), lambda: b.latent_prefill_workspace_bytes(1, 1, 1, 1)):
        with pytest.raises(pkv.PkvError) as e:
            call()
        assert e.value.status == pkv.PKV_ERR_FORMAT
    torch.cuda.synchronize()
    assert p.check_errors() == 0 and b.check_errors() == 0


def test_arguments_refused():
    case = Case([40], 512, seed=70)
    p, z, tab = case.pool, i32([0]), tables(4)
    kv = torch.zeros(1, 576, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, 1, 4, 576, dtype=torch.bfloat16, device="cuda")
    ok = dict(layer=0, rows=z, slots=z, kv=kv, positions=z, cos_sin=tab)

    def write(**kw):
        return lambda: p.write_latent(**{**ok, **kw})

    def attn(layer=0, ql=q[..., :512], qr=q[..., 512:], bt=case.table, ctx=case.ctx, scale=0.1, **kw):
        return lambda: p.paged_latent_attention(layer, ql, qr, bt, ctx, scale, **kw)

    qe = torch.zeros(1, 2, 4, 192, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(4, 128, 512, dtype=torch.bfloat16, device="cuda")

    def pre(layer=0, q=qe, wk=w, wv=w, bt=case.table, ctx=case.ctx, scale=0.1, **kw):
        return lambda: p.latent_prefill_attention(layer, q, wk, wv, bt, ctx, scale, **kw)

    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    big = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    odd = torch.zeros(577 * 4 + 8, dtype=torch.bfloat16, device="cuda")
    for call in (write(layer=1), write(layer=-1), write(kv=kv.float()), write(kv=kv[:, :512]), write(kv=kv.cpu()),
                 write(kv=odd[1:577][None]), write(norm_weight=kv[0, :64]), write(rows=i32([0, 0])),
                 write(norm_weight=kv[0, :512], eps=-1.0), write(norm_weight=kv[0, :512], eps=float("nan")),
                 write(cos_sin=tab[:, :32].contiguous()), write(cos_sin=tab.double()), write(positions=z.long()),
                 write(q_rope=q[0, :, :, 512:], q_out=q[0, :, :2, 512:]), write(q_out=q[0, :, :, 512:]),
                 write(q_rope=q[0, :, :, 512:], q_out=q[0, :, :1, 512:].expand(1, 4, 64)),
                 attn(layer=1), attn(scale=float("inf")), attn(scale=float("nan")), attn(ql=q[..., :256]),
                 attn(qr=q[..., :32]), attn(ql=q[..., :512].float()), attn(bt=case.table[0]), attn(bt=case.table.long()),
                 attn(ctx=i32([1, 2])), attn(workspace=small[:16]), attn(workspace=big[8:]),
                 attn(out=q[..., :512]), attn(ql=odd[:577 * 4].view(1, 1, 4, 577)[..., :512]),
                 attn(ql=odd[1:1 + 576 * 4].view(1, 1, 4, 576)[..., :512]),
                 pre(layer=2), pre(q=qe[..., :128]), pre(wk=w[:3]), pre(wv=w[..., :256]), pre(scale=float("nan")),
                 pre(workspace=small[:16]), pre(workspace=big[8:]), pre(max_ctx=-1), pre(q=qe[:, :0]), pre(q=qe[0]),
                 pre(bt=case.table[:0])):
        with pytest.raises((pkv.PkvError, TypeError, ValueError)):
            call()
    assert pkv.lib().pkv_paged_latent_attention(
        p.handle, 0, 4097, 1, 1, q.data_ptr(), 576, q.data_ptr(), 576, case.table.data_ptr(), 1, case.ctx.data_ptr(), 0,
        ctypes.c_float(0.1), q.data_ptr(), big.data_ptr(), big.numel(), None) == pkv.PKV_ERR_INVALID
    torch.cuda.synchronize()
    assert p.check_errors() == 0


def test_empty_calls():
    case = Case([40, 0], 512, seed=71)
    p = case.pool
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    p.write_latent(0, e, e, torch.zeros(0, 576, dtype=torch.bfloat16, device="cuda"), e, tables(2))
    bt = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    q = torch.zeros(0, 2, 4, 576, dtype=torch.bfloat16, device="cuda")
    assert p.paged_latent_attention(0, q[..., :512], q[..., 512:], bt, e, 0.1).shape == (0, 2, 4, 512)
    w = torch.zeros(4, 128, 512, dtype=torch.bfloat16, device="cuda")
    assert p.latent_prefill_attention(0, q[..., :192].contiguous(), w, w, bt, e, 0.1).shape == (0, 2, 4, 128)
    # nothing but empty sequences, and a block table without columns
    q = normal(gen(1), 2, 1, 4, 576)
    bt0 = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    out = torch.full((2, 1, 4, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    p.paged_latent_attention(0, q[..., :512], q[..., 512:], bt0, i32([0, 0]), 0.1, out=out)
    assert not out.any()
    out = torch.full((2, 1, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    p.latent_prefill_attention(0, q[..., :192].contiguous(), w, w, bt0, i32([0, 0]), 0.1, out=out)
    assert not out.any()
    assert p.check_errors() == 0


def test_limits_of_pricing_and_of_the_block_table():
    a = Case([40], R=256)
    for B, Hq, n_q, mb in ((1, 2048, 1, 2), (4097, 1, 1, 2), (1, 1 << 30, 4, 2), (1, 16, 1, (1 << 20) + 1)):
        with pytest.raises(pkv.PkvError):
            a.pool.price_request(1, B, Hq, n_q=n_q, max_blocks=mb)
    q = torch.zeros(1, 1, 256 + P, dtype=torch.bfloat16, device="cuda")
    wide = torch.zeros(1, (1 << 20) + 1, dtype=torch.int32, device="cuda")
    with pytest.raises(pkv.PkvError):
        a.pool.paged_latent_attention(0, q[..., :256], q[..., 256:], wide, i32([40]), 1.0)


@pytest.mark.parametrize("tok,head,ok", [(64, 64, False), (128, 64, False), (192, 64, True), (64, 192, True),
                                         (64, 256, True), (200, 72, False), (208, 72, True), (1 << 62, 64, True)])
def test_write_output_rows_do_not_overlap(tok, head, ok):
    a = Case([40], R=256)
    n, H = (1, 3) if tok > 1 << 40 else (3, 3)
    span = ((n - 1) * tok if n > 1 else 0) + (H - 1) * head + P
    out = torch.zeros(span, dtype=torch.bfloat16, device="cuda")
    g = gen(5)
    q, kv, tab = normal(g, n, H, P), normal(g, n, 256 + P), tables(8)
    row, slot, pos = i32([int(a.table[0, 0])] * n), i32(list(range(n))), i32([3, 1, 2][:n])
    st = a.pool._lib.pkv_write_latent(
        a.pool._h, 0, n, row.data_ptr(), slot.data_ptr(), kv.data_ptr(), 256 + P, pos.data_ptr(), tab.data_ptr(), 8, None,
        ctypes.c_float(0), 0, H, q.data_ptr(), H * P, P, out.data_ptr(), tok, head, pkv._stream(None))
    assert st == (pkv.PKV_OK if ok else pkv.PKV_ERR_INVALID)
    assert a.pool.check_errors() == 0
    if ok:
        got = torch.as_strided(out, (n, H, P), (tok if n > 1 else span, head, 1))
        want = a.pool.write_latent(0, row, slot, kv, pos, tab, interleaved=False, q_rope=q)
        assert torch.equal(got, want)
    # in place with other strides than the input's
    st = a.pool._lib.pkv_write_latent(
        a.pool._h, 0, n, row.data_ptr(), slot.data_ptr(), kv.data_ptr(), 256 + P, pos.data_ptr(), tab.data_ptr(), 8, None,
        ctypes.c_float(0), 0, H, q.data_ptr(), H * P, P, q.data_ptr(), H * 2 * P, 2 * P, pkv._stream(None))
    assert st == pkv.PKV_ERR_INVALID


def test_uneven_values_keep_the_documented_errors():
    """128 tokens 2^-18 below the next 128's largest, whose others are as small: queries that see
    only small values and queries that see the large ones too."""
    L, H, R = 300, 2, 256
    g = gen(11)
    a = Case([L], R=R)
    x = a.rows[:L].float()
    x[:256, :R] *= 2.0 ** -18
    x[200, :R] *= 2.0 ** 18
    kv = x.bfloat16()
    t = torch.arange(L, dtype=torch.int32, device="cuda")
    still = torch.cat((torch.ones(1, P // 2, device="cuda"), torch.zeros(1, P // 2, device="cuda")), 1)
    a.pool.write_latent(0, a.table[0][(t // 32).long()].contiguous(), t % 32, kv, torch.zeros_like(t), still)
    q = normal(g, 1, L, H, DH + P)
    q[..., :DH] = 0  # the logits hang on the position keys alone
    wk, wv = ((normal(g, H, DH, R).float() / R ** 0.5).bfloat16() for _ in range(2))
    out = a.pool.latent_prefill_attention(0, q, wk, wv, a.table, i32([L]), 0.1, max_ctx=L)
    assert a.pool.check_errors() == 0
    c, r, qr = kv[:, :R].double(), kv[:, R:].double(), q[0, :, :, DH:].double()
    v = torch.einsum("tr,hdr->htd", c, wv.double())
    v_mag = torch.einsum("tr,hdr->htd", c.abs(), wv.double().abs())
    hidden = hidden_for(L, L)
    s = (0.1 * torch.einsum("ihp,tp->hit", qr, r)).masked_fill(hidden, -math.inf)
    p = s.softmax(-1)
    want, mag = p @ v, p @ v.abs()
    # besides the roundings of the other tests: P is off by 2^(k - 31) of the row's largest in
    # tokens whose 128 have values 2^-k of the largest (k at most 19 for the first 128, as two
    # maxima of scaled normal values are within a factor of two; 1 for the others), values by
    # 2^-38 of the largest of their 128
    part = torch.full((L,), 2.0 ** -30, dtype=torch.float64, device="cuda")
    part[:128] = 2.0 ** (19 - 31)
    p_abs = p.amax(-1, keepdim=True) * (((~hidden) * part).double()[None] @ v.abs())
    v_abs = 2.0 ** -38 * v.abs().amax((1, 2), keepdim=True)
    d = (P * 2.0 ** -23 * 0.1 * torch.einsum("ihp,tp->hit", qr.abs(), r.abs())).amax(-1, keepdim=True)
    tol = U * want.abs() + (2 * H16 + 2 * d) * mag + p_abs + v_abs + R * 2.0 ** -23 * (p @ v_mag)
    err = (out[0].permute(1, 0, 2).double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
