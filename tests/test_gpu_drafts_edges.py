"""Trees of drafted tokens where the softmax's references and the packed pools' powers of two
move: against the formulas in 64 bits, with the bounds and helpers of test_gpu_drafts.py."""
import math

import pytest

from tests.test_gpu_drafts import Case, basis, run_tree

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def steep(D, n_q, by):
    """Keys whose logits with a query of ones rise by `by` (log2) every 32 tokens, at scale D^-0.5."""
    def f(k, v):
        t = torch.arange(k.shape[0] * 32, device="cuda").view(-1, 32, 1, 1)
        return k * 0.02 + t * (by / 32 * math.log(2) * D ** -0.5), v
    return f


@pytest.mark.parametrize("fmt,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("k4v4", 64), ("k4v4", 128), ("k8v4", 256),
                                   ("k8v8", 128)])
@pytest.mark.parametrize("n_q,Hq", [(9, 2), (64, 2), (70, 2), (140, 2)])
@pytest.mark.parametrize("ctas", [1, 3])
def test_both_halves_of_a_tile_move_the_reference(fmt, D, n_q, Hq, ctas):
    """Logits that rise by 12 (log2, slack: 8) with every 32 tokens: each half of each tile rescales
    what is there.  Beside them rows that fall, half as steep ones and flat ones, in the same warps."""
    case = Case(fmt, D, 1, [n_q + 250], seed=n_q, shape_kv=steep(D, n_q, 12.0))
    case.pool.decode_set_ctas(ctas)
    way = torch.tensor([1.0, -1.0, 0.5, 0.0, 1.0, 1.0, -0.5], device="cuda")
    q = way[torch.arange(n_q * Hq, device="cuda") % 7].view(1, n_q, Hq, 1).expand(1, n_q, Hq, D).bfloat16().contiguous()
    run_tree(case, n_q, Hq, seed=n_q, q=q, l2=False)
    assert case.pool.check_errors() == 0


def by_tile(powers, zero=()):
    """Values of each tile of 64 tokens times 2 to the powers, in turns; tiles of `zero` hold none."""
    def f(k, v):
        tile = torch.arange(k.shape[0], device="cuda") // 2
        p = torch.tensor(powers, dtype=torch.float64, device="cuda")[tile % len(powers)]
        m = torch.where(torch.isin(tile % len(powers), torch.tensor(list(zero), device="cuda")), 0.0, 2.0 ** p)
        return k, (v.double() * m[:, None, None, None]).float()
    return f


PACKED = [("k4v4", 64), ("k4v4", 128), ("k8v4", 128), ("k8v8", 256), ("k8v8", 64)]


@pytest.mark.parametrize("fmt,D", PACKED + [("bf16", 128)])
@pytest.mark.parametrize("powers,zero", [((0, 40), (0,)), ((60, -60), ()), ((100, 0, -100, 30), ()), ((118, 0), (1,)),
                                         ((0, 0, 100), (0, 1))])
@pytest.mark.parametrize("n_q,ctas", [(8, 1), (8, 3), (8, 40), (70, 2)])
def test_tiles_of_very_different_values(fmt, D, powers, zero, n_q, ctas):
    """The values' sizes say nothing about a token's weight: tiles of nothing, or of tiny values, keep
    their share of the softmax beside tiles of huge ones, within a CTA and over several."""
    if fmt == "bf16" and max(powers) > 110:
        pytest.skip("O in fp32 does not hold sums of such values")
    case = Case(fmt, D, 1, [n_q + 700, max(64, n_q), n_q + 129], seed=n_q, shape_kv=by_tile(powers, zero))
    case.pool.decode_set_ctas(ctas)
    run_tree(case, n_q, 2, seed=n_q, l2=False)
    assert case.pool.check_errors() == 0


@pytest.mark.parametrize("fmt,D", PACKED)
@pytest.mark.parametrize("scale", [1.0, 2.0 ** 20, -2.0 ** 20, 2.0 ** 40, 2.0 ** 110])
@pytest.mark.parametrize("ctas", [1, 5])
def test_equal_logits_of_any_size_weigh_the_same(fmt, D, scale, ctas):
    """One key for all tokens: whatever the logits' size, each token weighs the same, so the output is
    the values' mean, in tiles of any values.  Bounds: the output's rounding, a value's 4 h of its group's
    largest M, P's h, and what fp16 drops of small operands and probabilities (2^-38 and 2^-24 of the
    largest of a tile, each)."""
    U, h = 2.0 ** -8, 2.0 ** -11

    def f(k, v):
        return k[:1, :1].expand_as(k).contiguous(), by_tile((0, 12, -9, 30, 3))(k, v)[1]
    n_q = 5
    case = Case(fmt, D, 2, [n_q + 630], seed=3, shape_kv=f)
    case.pool.decode_set_ctas(ctas)
    q = torch.randn(1, n_q, 4, D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    out = case.pool.paged_tree_attention(0, q, torch.full((n_q, 1), 31, dtype=torch.int32, device="cuda"), case.table, case.ctx,
                                         scale)[0].double()
    _, v, _, vm = case.kv(0)
    L = v.shape[0]
    for hq in range(4):
        x, m = v[:, hq // 2], vm[:, hq // 2]
        top = m.max()
        tol = U * x.mean(0).abs() + 4 * h * m.mean(0) + h * x.abs().mean(0) + 2 * 2.0 ** -38 * top + 2.0 ** -24 * top
        err = (out[:, hq] - x.mean(0)).abs()
        assert (err <= tol).all(), (err / tol).max().item()


@pytest.mark.parametrize("fmt,D,group", [("k4v4", 64, 32), ("k4v4", 128, 32), ("k4v4", 128, 64), ("k8v4", 128, 32),
                                         ("k8v8", 64, 32), ("k8v8", 128, 32), ("k8v8", 256, 32)])
@pytest.mark.parametrize("apart", [18, 22, 24, 26])
@pytest.mark.parametrize("L", [2, 9])
def test_small_tokens_beside_a_huge_one(fmt, D, group, apart, L):
    """A drafted token 2^apart larger lies in the tile of the others, seen by one query alone: the other
    queries keep the accuracy of what they see.  A value s c + o, all three rounded to fp16, is off by
    4 h of its group's largest M, h = 2^-11, and where they fall below fp16's normal range by 2^-25 each, which is
    2^-38 of the tile's largest T, of 2^13 at least; the queries by h, the logits' fp32 sums by D 2^-23,
    P by h and the output by u = 2^-8.  Errors d of the logits count 2 d, as p moves with its sum; a token
    that is alone has p = 1 whatever its logit."""
    U, h = 2.0 ** -8, 2.0 ** -11
    n_q, Hq = 2, 4

    def f(k, v):
        huge = (torch.arange(k.shape[0] * 32, device="cuda").view(-1, 32, 1, 1) == L - n_q) * (2.0 ** apart - 1) + 1
        return k * huge, v * huge
    case = Case(fmt, D, 2, [L], seed=apart, group=group, shape_kv=f)
    q = torch.randn(1, n_q, Hq, D, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    mask = torch.tensor([[1], [2]], dtype=torch.int32, device="cuda")
    scale = D ** -0.5
    out = case.pool.paged_tree_attention(0, q, mask, case.table, case.ctx, scale)[0, 1].double()
    k, v, km, vm = case.kv(0)
    see = [t for t in range(L) if t != L - n_q]
    for hq in range(Hq):
        kv = hq // 2
        Tk, Tv = km[:, kv].max(), vm[:, kv].max()
        K, V, KM, VM = (y[see, kv] for y in (k, v, km, vm))
        qd = q[0, 1, hq].double() @ basis(D)
        p = torch.softmax(K @ qd * scale, 0)
        size = K.abs() @ qd.abs()
        d = (D * 2.0 ** -23 + h) * size + 4 * h * (KM @ qd.abs()) + 3 * 2.0 ** -38 * Tk * qd.abs().sum()
        d = d.max() * scale if L > n_q else 0.0
        ref = p @ V
        tol = U * ref.abs() + (h + 2 * d) * (p @ V.abs()) + 4 * h * (p @ VM) + 3 * 2.0 ** -38 * Tv
        err = (out[hq] - ref).abs()
        assert (err <= tol).all(), (err / tol).max().item()


@pytest.mark.parametrize("fmt,D", [("bf16", 128), ("k4v4", 64), ("k8v8", 256)])
@pytest.mark.parametrize("Hk,Hq,n_q", [(1, 128, 5), (1, 1024, 1), (2, 1024, 3)])
def test_many_query_heads_a_kv_head(fmt, D, Hk, Hq, n_q):
    case = Case(fmt, D, Hk, [n_q + 100, 0, n_q + 65], seed=Hq)
    run_tree(case, n_q, Hq, seed=Hq)
    assert case.pool.check_errors() == 0


@pytest.mark.parametrize("fmt,D", PACKED)
@pytest.mark.parametrize("mk,mq,scale", [(114, -100, 2.0 ** 30), (-80, 120, 2.0 ** 40), (-80, 100, -2.0 ** -60), (100, -60, 2.0 ** -100)])
def test_logits_of_extreme_factors(fmt, D, mk, mq, scale):
    """Keys, queries and scales whose products two by two leave fp32's range, all three not.  One key for
    all tokens: the output is the values' mean (bounds as above)."""
    U, h = 2.0 ** -8, 2.0 ** -11
    case = Case(fmt, D, 2, [205], seed=3, shape_kv=lambda k, v: ((k[:1, :1] * 2.0 ** mk).expand_as(k).contiguous(), v))
    q = torch.randn(1, 5, 4, D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") * 2.0 ** mq
    out = case.pool.paged_tree_attention(0, q.bfloat16(), torch.full((5, 1), 31, dtype=torch.int32, device="cuda"), case.table,
                                         case.ctx, scale)[0].double()
    _, v, _, vm = case.kv(0)
    for hq in range(4):
        x, m = v[:, hq // 2], vm[:, hq // 2]
        tol = U * x.mean(0).abs() + 4 * h * m.mean(0) + h * x.abs().mean(0) + 3 * 2.0 ** -38 * m.max() + 2.0 ** -24 * m.max()
        err = (out[:, hq] - x.mean(0)).abs()
        assert (err <= tol).all(), (err / tol).max().item()
