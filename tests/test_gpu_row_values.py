"""Values of the operators over vocabulary rows where rounding, masks or close scores decide them: what one operator
leaves is given to the next, and results are compared with 64-bit forms of their own (H: half a float32 step)."""
import numpy as np
import pytest
import torch

import causal_draft_correction_amd as dca
import rows_plain as plain

pytestmark = pytest.mark.gpu

H = 2.0 ** -24
DTYPES = [torch.float32, torch.bfloat16]
# rows by one block, by one block with the gradient only, and split
LENGTHS = (300, 9001, 70001)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dca.load_library()


def host(t):
    return t.float().cpu().numpy()


def logits(B, R, V, dtype, seed, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((B, R, V), generator=g).mul_(scale).to(dtype).cuda()


def three_ways(z, ids, values, lse, g, **kw):
    """Loss and gradient by one call, and by a forward and a backward call; the forward call's statistics."""
    both = dca.distill(z, ids, values, lse, grad_loss=g, **kw)
    first = dca.distill(z, ids, values, lse, **kw)
    second = dca.distill_backward(z, ids, first["stats"], g, **kw)
    torch.cuda.synchronize()
    return (both["loss"], both["grad"]), (first["loss"], second), first["stats"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", LENGTHS)
def test_teacher_rows_whose_mask_leaves_nothing_are_left_out(V, dtype):
    k = 20
    z = logits(1, 4, V, dtype, V)
    target = logits(1, 4, V, torch.float32, V + 1)
    target[0, 1] = -np.inf
    top = dca.top_logits(target, k)
    assert float(top["lse"][0, 1]) == -np.inf and bool((top["ids"][0, 1] >= 0).all())
    g = torch.ones((1, 4), device="cuda")
    for lse in (top["lse"], None):
        one, two, stats = three_ways(z, top["ids"], top["values"], lse, g)
        for loss, grad in (one, two):
            assert float(loss[0, 1]) == 0.0 and not bool(grad[0, 1].float().abs().max() > 0)
            assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(grad.float()).all())
            assert bool((loss[0, [0, 2, 3]] > 0).all())
        assert not bool(stats[0, 1].abs().max() > 0)
        z2 = z.clone()
        z2[0, 1] = np.nan  # whatever the student's row holds
        again = three_ways(z2, top["ids"], top["values"], lse, g)
        assert torch.equal(again[0][0], one[0]) and torch.equal(again[1][1], two[1])
    # a NaN among the values is no mask
    values = top["values"].clone()
    values[0, 1, 3] = np.nan
    one, two, _ = three_ways(z, top["ids"], values, top["lse"], g)
    assert np.isnan(float(one[0][0, 1])) and np.isnan(float(two[0][0, 1]))
