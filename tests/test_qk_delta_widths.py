"""Counts past 32 bits are refused by the binding, before they would wrap in the C call's 32-bit arguments."""
import pytest
import torch

import test_layer_amd as tla

FAR = 2 ** 32 + 64  # a head of 64 in its low 32 bits


def _t(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


def test_sections_and_norms():
    q, pos = torch.zeros(4, 64), torch.zeros(4, 1, dtype=torch.int32)
    for sections in ((2 ** 32 + 16,), (-2 ** 32 + 16,), (2 ** 40,)):
        with pytest.raises(ValueError, match="sections.*32 bits"):
            tla.qk_norm_rope(q, None, 1, pos=pos, sections=sections)
        with pytest.raises(ValueError, match="sections.*32 bits"):
            tla.qk_norm_rope_grad(q, None, q, None, 1, pos=pos, sections=sections)
    with pytest.raises(ValueError, match="norm.*32 bits"):
        tla.qk_norm_rope(q, None, 1, norm=2 ** 32 + tla.NORM_L2)
    with pytest.raises(ValueError, match="norm.*32 bits"):
        tla.qk_norm_rope_grad(q, None, q, None, 1, norm=2 ** 32 + tla.NORM_L2)


def test_widths():
    wide, q = _t(1, FAR), _t(1, 64)
    f = _t(1, 1, dtype=torch.float32)
    state = _t(1, 1, 64, 64, dtype=torch.float32)
    calls = [lambda: tla.qk_norm_rope(wide, None, 1), lambda: tla.qk_norm_rope(q, wide, 1, 1),
             lambda: tla.qk_norm_rope_grad(wide, None, wide, None, 1), lambda: tla.qk_norm_rope(wide, None, FAR // 64)]
    for a in ((wide, wide, q), (q, q, wide)):
        calls += [lambda a=a: tla.gated_delta(*a, f, f, 1), lambda a=a: tla.gated_delta_grad(*a, f, f, a[2], 1),
                  lambda a=a: tla.gated_delta_step(*a, f, f, 1, state)]
    for call in calls:
        with pytest.raises(ValueError, match="32 bits"):
            call()
