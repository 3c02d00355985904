"""RMSNorm over more rows than 31 bits count: T goes up to 2^31 - 1, and a CTA's next row lies up to a grid further."""
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16


def test_rows_are_counted_unsigned():
    src = open(os.path.join(ROOT, "mixture_experts_layer_aux_b200", "csrc", "rmsnorm.cu")).read()
    src = re.sub(r"//[^\n]*", "", src)
    assert "(int)gridDim.x" not in src and not re.search(r"\bint row\b", src)
    assert len(re.findall(r"for \(uint32_t row = blockIdx\.x; row < \(uint32_t\)p\.T; row \+= gridDim\.x\)", src)) == 2


@pytest.mark.gpu
def test_the_most_rows(moe):
    """2^31 - 1 rows of 8 (34 GB), in place. Rows of 2 are normed to rows of 1. Then, with dY = h = rstd = weight = 1,
    dX = 1 - mean(1) = 0 and dweight counts the rows: a CTA's share is below 2^24, so exact, and 296 of them are added
    in 15 steps, each off by half a step of 2^-23 at most."""
    T, H = 2 ** 31 - 1, 8
    if torch.cuda.mem_get_info()[0] < 56 << 30:
        pytest.skip("needs 44 GB of device memory")
    x = torch.full((T + 1, H), 2.0, dtype=BF, device="cuda")
    w = torch.ones(H, dtype=BF, device="cuda")
    rstd = torch.zeros(T, device="cuda")
    moe.moe_rmsnorm_fwd(x[:T], None, w, 0.0, None, x[:T], None, None, rstd)
    flat = x.view(-1)

    def all_are(t, v):
        return all(bool((c == v).all()) for c in t.split(1 << 28))

    assert all_are(flat[:T * H], 1.0) and all_are(flat[T * H:], 2.0) and all_are(rstd, 0.5)
    rstd.fill_(1.0)
    dw = torch.empty(H, device="cuda")
    moe.moe_rmsnorm_bwd(x[:T], x[:T], w, rstd, None, x[:T], dw, moe.workspace(moe.moe_rmsnorm_bwd_workspace_size(T, H)))
    assert all_are(flat[:T * H], 0.0) and all_are(flat[T * H:], 2.0)
    assert bool(((dw.double() / T - 1).abs() <= 15 * 2.0 ** -24).all())
