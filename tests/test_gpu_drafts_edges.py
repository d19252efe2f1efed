"""Trees of drafted tokens where the softmax's references and the packed pools' powers of two
move: against the formulas in 64 bits, with the bounds and helpers of test_gpu_drafts.py."""
import math

import pytest

from tests.test_gpu_drafts import Case, run_tree

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
