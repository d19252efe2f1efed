"""Latent-pool calls at the edges: running maxima that move in a segment's last tile, huge
and lowest logits, tiles of zero, uneven or non-finite values, memory that belongs to no
sequence, two tokens at one place, pricing at the calls' limits.

References are the formulas in 64 bits, with the bounds derived in test_gpu_latent.py."""
import math

import numpy as np
import pytest

import paged_kv_cache_split_gb300 as pkv
from test_gpu_latent import (DH, H16, P, SCALE, U, Case, _needs_gpu, absorbed, check, check_absorbed,
                             expanded_ref, gen, i32, normal, pool_rows)  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def still():
    """A rotary table that turns nothing."""
    return torch.cat((torch.ones(1, P // 2), torch.zeros(1, P // 2)), 1).cuda()


def rewrite(case, b, rows):
    """Sequence b's rows become `rows`, stored as they are."""
    t = torch.arange(len(rows), device="cuda")
    case.pool.write_latent(0, case.table[b][(t // 32).long()].contiguous(), (t % 32).int(), rows, t.int() * 0, still())
    case.seq[b] = rows


@pytest.mark.parametrize("R,n_q,H", [(512, 1, 64), (512, 1, 128), (512, 3, 40), (256, 1, 64), (512, 1, 16), (512, 1, 32)])
def test_absorbed_maximum_raised_in_every_last_tile(R, n_q, H):
    """Logits that rise by far more than the reference's slack from tile to tile, so that each
    CTA's last tile raises it, over many splits; repeats are bit-identical."""
    lens = [1000, 65, 129, 640]
    case = Case(lens, R, seed=91)
    for b, L in enumerate(lens):
        rows = case.seq[b].float()
        rows[:, :8] += 0.6 * torch.arange(L, device="cuda").float()[:, None]
        rewrite(case, b, rows.bfloat16())
    q = normal(gen(92), len(lens), n_q, H, R + P)
    q[..., :8] = 1.0
    for ctas in (1, 3, 16, 40, 0):
        case.pool.decode_set_ctas(ctas)
        out = absorbed(case, q, SCALE)
        check_absorbed(case, out, q, SCALE)
        for _ in range(10):
            assert torch.equal(out, absorbed(case, q, SCALE))
    assert case.pool.check_errors() == 0


def picked_values(H, R=512):
    """A value projection that takes the latent's first 128 values."""
    w = torch.zeros(H, DH, R, dtype=torch.bfloat16, device="cuda")
    w[:, torch.arange(DH), torch.arange(DH)] = 1
    return w


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("k", [20, 23, 24, 25, 26, 27, 30, 100])
def test_expanded_huge_logits_over_uneven_tiles(k, sign):
    """Logits of 2^k or 2^k + step in log2 units, exact in fp32 (two products a logit, a scale
    that becomes 1.0), over tiles whose values differ by powers of two.  The bound has no
    term for the logits."""
    L, n_q, H = 1280, 4, 2
    step = max(8.0, 2.0 ** (k - 23))
    case = Case([L], 512, seed=101)
    rows = case.seq[0].clone()
    tile = torch.arange(L, device="cuda") // 128
    e = torch.tensor([0, -3, 2, -6, 1, 1, -1, 4, -2, 0], device="cuda")[tile]
    up = torch.tensor([0, 1, 1, 0, 1, 0, 1, 1, 0, 1], device="cuda")[tile].double()
    rows[:, :512] = (rows[:, :512].float() * 2.0 ** e[:, None]).bfloat16()
    rows[:, 512:] = 0
    half = min(60, k // 2)
    rows[:, 512] = 2.0 ** half
    rows[:, 513] = (up * step).bfloat16()
    rewrite(case, 0, rows)
    scale = float(np.float32(math.log(2)))
    assert np.float32(scale * math.log2(math.e)) == 1.0
    q = torch.zeros(1, n_q, H, DH + P, dtype=torch.bfloat16, device="cuda")
    q[..., DH] = sign * 2.0 ** (k - half)
    q[..., DH + 1] = 1
    wv = picked_values(H)
    v = rows[:, :DH].double()
    for ctas in (1, 0):
        case.pool.decode_set_ctas(ctas)
        out = case.pool.latent_prefill_attention(0, q, torch.zeros_like(wv), wv, case.table, case.ctx, scale)
        for i in range(n_q):
            n = L - n_q + i + 1
            p = torch.exp2((up[:n] - 1) * step)
            p /= p.sum()
            want, mag = p @ v[:n], p @ v[:n].abs()
            tol = U * want.abs() + 2 * H16 * mag + 2.0 ** -24 * v.abs().max()
            for h in range(H):
                assert ((out[0, i, h].double() - want).abs() <= tol).all(), (i, h, ctas)
    assert case.pool.check_errors() == 0


def test_pools_that_follow_one_another_at_one_address():
    """Slabs of two pools with other row widths at the same memory, their tensor maps at the
    same addresses (20 blocks of 1152-byte rows, 36 of 640)."""
    memory = torch.zeros(20 * 32 * 1152 + 4096, dtype=torch.uint8, device="cuda")
    alloc = pkv.Allocator(pkv.ALLOC_FN(lambda ctx, n, stream: memory.data_ptr()),
                          pkv.RELEASE_FN(lambda ctx, ptr, stream: None), None)
    g = gen(123)
    for turn in range(6):
        R, blocks = ((512, 20), (256, 36))[turn % 2]
        pool = pkv.Pool(1, 1, R, "latent", slab_blocks=blocks, max_slabs=1, allocator=alloc)
        pool.reserve_rows(blocks)
        L, H = 500, 4
        case = Case.__new__(Case)
        case.pool, case.R, case.W, case.layer, case.lens = pool, R, R + P, 0, [L]
        case.table = torch.randperm(blocks, generator=g, device="cuda")[None, :16].int().contiguous()
        case.ctx, case.seq = i32([L]), [None]
        rewrite(case, 0, normal(g, L, R + P))
        q = normal(g, 1, 1, H, R + P)
        check_absorbed(case, absorbed(case, q, SCALE), q, SCALE)
        qe, w = normal(g, 1, 3, H, DH + P), normal(g, H, DH, R) / 22
        out = pool.latent_prefill_attention(0, qe, w, w, case.table, case.ctx, SCALE)
        check(out[0], *expanded_ref(case, qe[0], w, w, 0, SCALE), f"turn {turn}")
        assert pool.check_errors() == 0
        pool.close()


def test_latent_requests_are_priced_under_the_calls_limits():
    p = Case([40], 512, seed=117).pool
    for B, n_q, H in ((1, 8192, 16), (64, 66, 1000), (4096, 1, 16), (4096, 2, 16)):
        pr = p.price_request(3, B, H, n_q=n_q, max_blocks=256)
        assert pr["workspace_bytes"] == p.latent_workspace_bytes(B, n_q, H)
        assert pr["fixed_bytes"] == 256 * 4 + 4 + n_q * H * (576 + 512) * 2


def test_pricing_of_the_expanded_form():
    p = Case([40], 512, seed=125).pool
    W = 512 + P
    for B, n_q, H, mb, ctx in ((1, 8192, 16, 256, 0), (1, 8192, 16, 300, 8192), (4, 1000, 16, 128, 4096), (3, 1, 2, 40, 0)):
        pr = p.price_latent_prefill(70, B, H, n_q, mb, max_ctx=ctx)
        assert pr["workspace_bytes"] == p.latent_prefill_workspace_bytes(B, n_q, H, mb, ctx)
        assert pr["workspace_bytes"] >= 2 * B * H * (ctx or 32 * mb) * DH * 2
        assert pr["fixed_bytes"] == 4 * mb + 4 + n_q * H * (DH + P + DH) * 2
        same = p.price_request(70, B, H, n_q=n_q, max_blocks=mb)
        for k in ("slabs_to_append", "free_rows", "storage_bytes", "page_bytes"):
            assert pr[k] == same[k]
        assert pr["page_bytes"] == 70 * 32 * W * 2 and pr["slabs_to_append"] > 0
    # the price covers the call
    case = Case([300], 512, seed=127)
    pr = case.pool.price_latent_prefill(0, 1, 2, 5, case.width)
    g = gen(1)
    ws = torch.empty(pr["workspace_bytes"], dtype=torch.uint8, device="cuda")
    w = normal(g, 2, DH, 512) / 22
    case.pool.latent_prefill_attention(0, normal(g, 1, 5, 2, DH + P), w, w, case.table, case.ctx, SCALE, workspace=ws)
    assert case.pool.check_errors() == 0
    for bad in ((-1, 1, 1, 1, 1, 0), (1, 0, 1, 1, 1, 0), (1, 1, 0, 1, 1, 0), (1, 1, 1, 0, 1, 0), (1, 1, 1, 1, -1, 0),
                (1, 1, 1, 1, 1, -1), (1, 4097, 1, 1, 1, 0), (1, 1, 1025, 1, 1, 0), (1, 1, 1, 1, (1 << 20) + 1, 0),
                (1, 64, 1024, 1, 1 << 20, 0), (10 ** 8, 1, 1, 1, 1, 0)):
        with pytest.raises(pkv.PkvError):
            p.price_latent_prefill(*bad)
    other = pkv.Pool(1, 1, 128, "bf16")
    with pytest.raises(pkv.PkvError) as e:
        other.price_latent_prefill(1, 1, 1, 1, 1)
    assert e.value.status == pkv.PKV_ERR_FORMAT


@pytest.mark.parametrize("e", [0, -12, -40, -90])
@pytest.mark.parametrize("ctas", [1, 0])
def test_expanded_tile_of_zero_values(e, ctas):
    """128 tokens without any value, beside values of 2^e."""
    L, n_q, H = 900, 5, 2
    case = Case([L], 512, seed=103)
    case.pool.decode_set_ctas(ctas)
    rows = case.seq[0].clone()
    rows[128:256, :512] = 0
    rewrite(case, 0, rows)
    g = gen(104)
    q = normal(g, 1, n_q, H, DH + P)
    wk = normal(g, H, DH, 512) / 22
    wv = (normal(g, H, DH, 512).float() / 22 * 2.0 ** e).bfloat16()
    out = case.pool.latent_prefill_attention(0, q, wk, wv, case.table, case.ctx, SCALE)
    check(out[0], *expanded_ref(case, q[0], wk, wv, 0, SCALE), f"values of 2^{e}")
    assert case.pool.check_errors() == 0


def test_expanded_many_zero_values_weigh_in_the_sum():
    """One token with values and 400000 without, each with 2^-24.5 of its probability: together
    they take 1.6% from the output, four times its rounding."""
    L, H = 400001, 1
    case = Case([L], 256, seed=129)
    rows = torch.zeros(L, 256 + P, dtype=torch.bfloat16, device="cuda")
    rows[0, :DH] = normal(gen(130), DH)
    rows[1:, 256] = 1
    rewrite(case, 0, rows)
    q = torch.zeros(1, 1, H, DH + P, dtype=torch.bfloat16, device="cuda")
    q[..., DH] = -24.5
    wv = picked_values(H, 256)
    want = rows[0, :DH].double() / (1 + (L - 1) * 2.0 ** -24.5)
    for ctas in (1, 0):
        case.pool.decode_set_ctas(ctas)
        out = case.pool.latent_prefill_attention(0, q, torch.zeros_like(wv), wv, case.table, case.ctx, math.log(2))
        assert ((out[0, 0, 0].double() - want).abs() <= (U + 2 * H16) * want.abs()).all()
    assert case.pool.check_errors() == 0


@pytest.mark.parametrize("bits", [0x7F80, 0xFF80, 0x7FC0])
def test_expanded_nonfinite_row_stays_in_its_tile(bits):
    """A latent with an infinity or a NaN among tokens 128 to 255: the queries that see only the
    first 128 tokens keep the formula's bounds."""
    L = n_q = 256
    H = 2
    case = Case([L], 512, seed=105)
    rows = case.seq[0].clone()
    rows.view(torch.int16)[200, 77] = bits if bits < 0x8000 else bits - 0x10000
    rewrite(case, 0, rows)
    g = gen(106)
    q = normal(g, 1, n_q, H, DH + P)
    wk, wv = normal(g, H, DH, 512) / 22, normal(g, H, DH, 512) / 22
    out = case.pool.latent_prefill_attention(0, q, wk, wv, case.table, case.ctx, SCALE)
    assert not torch.isfinite(out[0, 200:]).all()

    class Head:
        seq, lens, R = [rows[:128]], [128], 512
    check(out[0, :128], *expanded_ref(Head, q[0, :128], wk, wv, 0, SCALE), "queries of the first tile")
    assert case.pool.check_errors() == 0


def test_expanded_results_do_not_hang_on_bytes_outside_the_sequence():
    """Bit-identical whatever the slots past the lengths and the queries of unused slots hold."""
    n_q, H = 3, 16
    lens = [417, 0] * 16
    g = gen(107)
    q = normal(g, 32, n_q, H, DH + P)
    wk, wv = normal(g, H, DH, 512) / 22, normal(g, H, DH, 512) / 22
    ref = None
    for ctas in (1, 0):
        ref = None
        for stale in (0x0000, 0x7F7F, 0x7FC0, 0x7F80):
            for junk in (0.0, 1000.0, float("inf"), float("nan")):
                case = Case(lens, 512, seed=109, stale=stale)
                case.pool.decode_set_ctas(ctas)
                qj = q.clone()
                qj[1::2] = junk
                out = case.pool.latent_prefill_attention(0, qj, wk, wv, case.table, case.ctx, SCALE)
                if ref is None:
                    ref = out
                assert torch.equal(out, ref), (ctas, hex(stale), junk, int((out != ref).sum()))


@pytest.mark.parametrize("n_q,H", [(1, 5), (1, 20), (3, 7), (1, 65)])
def test_absorbed_results_do_not_hang_on_unused_queries(n_q, H):
    """Bit-identical whatever the queries of unused batch slots hold, head counts that leave
    a row tile partly empty."""
    case = Case([417, 0] * 16, 512, seed=111)
    q = normal(gen(112), 32, n_q, H, 576)
    for ctas in (1, 0):
        case.pool.decode_set_ctas(ctas)
        ref = None
        for junk in (0.0, 1000.0, float("inf"), float("nan")):
            qj = q.clone()
            qj[1::2] = junk
            out = absorbed(case, qj, SCALE)
            if ref is None:
                ref = out
            assert torch.equal(out, ref), (ctas, junk, int((out != ref).sum()))


@pytest.mark.parametrize("ctas", [1, 0])
def test_logits_at_the_lowest_of_fp32(ctas):
    """Every logit the same, within 5% of the lowest finite value in log2 units."""
    L, H, x = 700, 4, -2.25e38
    case = Case([L], 512, seed=113)
    rows = case.seq[0].clone()
    rows[:, 512:] = 0
    rows[:, 512] = 2.0 ** 60
    rewrite(case, 0, rows)
    case.pool.decode_set_ctas(ctas)
    q = torch.zeros(1, 1, H, 576, dtype=torch.bfloat16, device="cuda")
    q[..., 512] = x / 2.0 ** 60
    assert -3.4e38 < float(q[0, 0, 0, 512]) * 2.0 ** 60 * math.log2(math.e) < -3e38
    want, mag = rows[:, :512].double().mean(0), rows[:, :512].double().abs().mean(0)
    out = absorbed(case, q, 1.0)
    assert ((out[0, 0].double() - want).abs() <= U * want.abs() + U * mag).all()
    qe = torch.zeros(1, 1, H, DH + P, dtype=torch.bfloat16, device="cuda")
    qe[..., DH] = x / 2.0 ** 60
    wv = picked_values(H)
    out = case.pool.latent_prefill_attention(0, qe, torch.zeros_like(wv), wv, case.table, case.ctx, 1.0)
    assert ((out[0, 0].double() - want[:DH]).abs() <= U * want[:DH].abs() + 2 * H16 * mag[:DH] + 2.0 ** -24 * 8).all()


def test_scales_beyond_fp32_in_powers_of_two_are_refused():
    case = Case([40], 512, seed=115)
    q, w = normal(gen(1), 1, 1, 4, 576), torch.zeros(4, DH, 512, dtype=torch.bfloat16, device="cuda")
    for scale in (3e38, -3e38, 2.4e38):
        with pytest.raises(pkv.PkvError):
            absorbed(case, q, scale)
        with pytest.raises(pkv.PkvError):
            case.pool.latent_prefill_attention(0, q[..., :192].contiguous(), w, w, case.table, case.ctx, scale)


@pytest.mark.parametrize("R", [256, 512])
def test_write_of_one_place_twice(R):
    """64 tokens at one place: each 16-byte piece of the row is one token's, and nothing else
    of the pool changes."""
    case = Case([64], R, seed=121)
    before = pool_rows(case.pool, 4, R + P).clone()
    n = 64
    kv = normal(gen(122), n, R + P)
    row = int(case.table[0, 1])
    case.pool.write_latent(0, i32([row] * n), i32([7] * n), kv, i32([0] * n), still())
    after = pool_rows(case.pool, 4, R + P)
    got = after[row, 7].view(torch.int16).view(-1, 8)
    want = kv.view(torch.int16).view(n, -1, 8)
    assert ((want == got).all(-1)).any(0).all()
    after[row, 7] = before[row, 7]
    assert torch.equal(after.view(torch.int16), before.view(torch.int16))


def test_workspace_sizes_kept_are_bounded():
    case = Case([40], 256, seed=119)
    q, w = normal(gen(1), 1, 1, 1, DH + P), torch.zeros(1, DH, 256, dtype=torch.bfloat16, device="cuda")
    wide = torch.zeros(1, 64, dtype=torch.int32, device="cuda")
    wide[0, :2] = case.table[0, :2]
    for m in range(40, 2048):
        case.pool.latent_prefill_attention(0, q, w, w, wide, case.ctx, SCALE, max_ctx=m)
    assert len(case.pool._ws_bytes) <= 1024
    assert case.pool.check_errors() == 0


def test_tensors_of_another_device_are_refused():
    """(The pool's device is moved instead of the tensors: one device is enough.)"""
    case = Case([40], 256, seed=131)
    q, w = normal(gen(1), 1, 1, 2, 256 + P), torch.zeros(2, DH, 256, dtype=torch.bfloat16, device="cuda")
    case.pool._device += 1
    with pytest.raises(ValueError, match="the pool is on"):
        absorbed(case, q, SCALE)
    with pytest.raises(ValueError, match="the pool is on"):
        case.pool.latent_prefill_attention(0, q[..., :DH + P].contiguous(), w, w, case.table, case.ctx, SCALE)
    with pytest.raises(ValueError, match="the pool is on"):
        case.pool.write_latent(0, i32([0]), i32([0]), q[0, 0, :1], i32([0]), still())
