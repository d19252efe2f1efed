"""Latent-pool calls at the edges: running maxima that move in a segment's last tile, huge
and lowest logits, tiles of zero, uneven or non-finite values, memory that belongs to no
sequence, two tokens at one place, pricing at the calls' limits.

References are the formulas in 64 bits, with the bounds derived in test_gpu_latent.py."""
import pytest

from test_gpu_latent import P, SCALE, Case, _needs_gpu, absorbed, check_absorbed, gen, normal  # noqa: F401

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
