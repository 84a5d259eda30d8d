"""The query/key preparation and its gradient where values are not finite and where positions are far, on the GPU."""
import pytest
import torch

import test_layer_amd as tla

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# heads by 4 pairs apart, by neighbours, handed over through LDS and value by value, of each number of lanes
SHAPES = [(64, (16, 16), False), (64, (), False), (64, (32,), True), (64, (12, 10, 10), False), (63, (10, 7), False), (128, (32, 16), False),
          (104, (20, 6), False), (200, (40, 20), True), (512, (100,), False), (7, (2,), True)]


def _randn(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _pos(n, sections, far=1000):
    if not sections:
        return None
    return torch.randint(-far, far, (n, len(sections)), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,sections,interleaved", SHAPES, ids=str)
def test_length_of_a_head_with_nan(d, sections, interleaved, dtype):
    # |x| is NaN, and so are x / max(|x|, eps) and its gradient, all over the head and nowhere else
    n, heads = 9, 3
    x, dy = (_randn(n, heads * d, seed=s, dtype=DT[dtype]) for s in (1, 2))
    rest = dict(norm="l2", eps=1e-6, pos=_pos(n, sections), sections=sections, interleaved=interleaved)
    y, _ = tla.qk_norm_rope(x, None, heads, **rest)
    g = tla.qk_norm_rope_grad(x, None, dy, None, heads, **rest).dq
    for row, head, at in ((0, 0, 0), (4, 2, d - 1), (8, 1, d // 2)):
        bad = x.clone()
        bad[row, head * d + at] = float("nan")
        spoilt = torch.zeros_like(x, dtype=torch.bool)
        spoilt[row, head * d:head * d + d] = True
        for got, want in ((tla.qk_norm_rope(bad, None, heads, **rest)[0], y),
                          (tla.qk_norm_rope_grad(bad, None, dy, None, heads, **rest).dq, g)):
            assert torch.isnan(got[spoilt]).all() and torch.equal(got[~spoilt], want[~spoilt])
