"""RMSNorm with the residual's addition, forward (bf16 and MXFP8 outputs) and backward, against 64 bits."""
import pytest
import torch

from block_ref import F32, U, check_mx, norm_bwd, norm_fwd

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# fp32 error of y before its rounding, relative: the sum of squares adds at most 32 terms in one thread and 10 levels
# of a tree (42 half steps, halved by the square root), the mean, eps, the root, the addition of the residual (twice
# in the square), two products: below 32 + 21 half steps of 2^-24
REL = 64 * F32

SHAPES = [(1, 8), (1, 4096), (2, 32), (3, 40), (7, 2056), (5, 7168), (64, 96), (147, 1000), (148, 1024), (149, 1032),
          (300, 2880), (1300, 512), (2, 16384), (400, 16384), (333, 8200)]


def draw(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(BF).cuda()


def run_fwd(moe, x, r, w, eps, mx=True, y=True, h=True):
    T, H = x.shape
    o = {"h": torch.full((T + 1, H), 7.0, dtype=BF, device="cuda") if h else None,
         "y": torch.full((T + 1, H), 7.0, dtype=BF, device="cuda") if y else None,
         "rstd": torch.full((T + 1,), 7.0, device="cuda"), "q": None, "sf": None}
    if mx:
        o["q"] = torch.full((T + 1, H), 9, dtype=torch.uint8, device="cuda")
        o["sf"] = torch.full((T + 1, H // 32), 9, dtype=torch.uint8, device="cuda")
    moe.moe_rmsnorm_fwd(x, r, w, eps, o["h"], o["y"], o["q"], o["sf"], o["rstd"])
    torch.cuda.synchronize()
    for n, t in o.items():  # the row behind the last is left as it was
        if t is not None:
            assert bool((t[T].float() == (9.0 if n in ("q", "sf") else 7.0)).all()), n
    return {n: (t[:T] if t is not None else None) for n, t in o.items()}


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_forward(moe, T, H, residual):
    x, w = draw((T, H), 1), draw((H,), 2, 0.5)
    r = draw((T, H), 3, 3.0) if residual else None
    o = run_fwd(moe, x, r, w, 1e-5, mx=H % 32 == 0)
    h, rstd, y = norm_fwd(x.cpu(), None if r is None else r.cpu(), w.cpu(), 1e-5)
    s = x.float() + (r.float() if residual else 0.0)
    assert torch.equal(o["h"], s.to(BF))
    assert bool(((o["rstd"].double().cpu() - rstd).abs() <= REL * rstd).all())
    d = (o["y"].double().cpu() - y).abs()
    assert bool((d <= (U + 2 * REL) * y.abs()).all()), float((d / y.abs().clamp_min(1e-30)).max())
    if H % 32 == 0:
        check_mx(o["q"], o["sf"], y, REL)


def test_mxfp8_alone_and_rows_of_zeros(moe):
    x = draw((9, 256), 5)
    x[3] = 0
    x[4, 32:64] = 0
    w = torch.ones(256, dtype=BF, device="cuda")
    o = run_fwd(moe, x, None, w, 1e-6, y=False, h=False)
    h, rstd, y = norm_fwd(x.cpu(), None, w.cpu(), 1e-6)
    check_mx(o["q"], o["sf"], y, REL)
    assert int(o["q"][3].max()) & 0x7F == 0 and int(o["sf"][3].max()) == 0 and int(o["sf"][4, 1]) == 0


def test_codes_are_those_of_the_quantiser(moe):
    """On values that are bf16 already (a weight of powers of two, rows of mean square one), the codes and scales are
    those that moe_quantize_mxfp8 gives for y."""
    T, H = 40, 512
    x = torch.where(torch.rand((T, H), generator=torch.Generator().manual_seed(1)) < 0.5, -1.0, 1.0).to(BF).cuda()
    w = torch.pow(2.0, torch.randint(-9, 9, (H,), generator=torch.Generator().manual_seed(2)).float()).to(BF).cuda()
    o = run_fwd(moe, x, None, w, 0.0)
    q, sf = torch.empty_like(o["q"]), torch.empty_like(o["sf"])
    moe.moe_quantize_mxfp8(o["y"].contiguous(), q, sf)
    assert torch.equal(q, o["q"]) and torch.equal(sf, o["sf"])


def test_extremes(moe):
    """Large, tiny, infinite and NaN values: as the formula in fp32 gives them."""
    H = 64
    x = draw((6, H), 3)
    x[0] *= 2.0 ** 60      # squares of 2^120: in range
    x[1] = x[1] * 2.0 ** -100  # squares vanish, eps rules
    x[2, 5] = float("inf")
    x[3, 6] = float("nan")
    x[4] = 3e38
    w = torch.ones(H, dtype=BF, device="cuda")
    o = run_fwd(moe, x, None, w, 1e-5, mx=True)
    h32 = x.float()
    rstd = torch.rsqrt(h32.pow(2).mean(-1) + 1e-5)
    y = h32 * rstd[:, None]
    fin = torch.isfinite(y)
    assert torch.equal(torch.isfinite(o["y"]), fin)
    assert torch.equal(torch.isnan(o["y"]), torch.isnan(y))
    d = (o["y"].float() - y).abs()[fin]
    assert bool((d <= (U + 2 * REL) * y.abs()[fin] + 1e-38).all())
    assert bool((o["q"][3] & 0x7F == 0x7F).all())  # NaN is NaN in e4m3


def test_in_place(moe):
    x, r, w = draw((211, 1024), 1), draw((211, 1024), 2), draw((1024,), 3)
    ref = run_fwd(moe, x, r, w, 1e-5, mx=False)
    x2, r2 = x.clone(), r.clone()
    moe.moe_rmsnorm_fwd(x2, r2, w, 1e-5, r2, x2, None, None, None)  # h over the residual, y over x
    assert torch.equal(r2, ref["h"]) and torch.equal(x2, ref["y"])


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dh", [True, False])
def test_backward(moe, T, H, dh):
    h, w, dy = draw((T, H), 1, 2.0), draw((H,), 2, 0.7), draw((T, H), 3)
    up = draw((T, H), 4) if dh else None
    rstd = torch.rsqrt(h.float().pow(2).mean(-1) + 1e-5)
    dx = torch.full((T + 1, H), 7.0, dtype=BF, device="cuda")
    dw = torch.empty(H, device="cuda")
    ws = moe.workspace(moe.moe_rmsnorm_bwd_workspace_size(T, H))
    moe.moe_rmsnorm_bwd(dy, h, w, rstd, up, dx[:T], dw, ws)
    torch.cuda.synchronize()
    assert bool((dx[T] == 7.0).all())
    c = [t.cpu() if t is not None else None for t in (dy, h, w, rstd, up)]
    rx, rw = norm_bwd(*c)
    xhat = (c[1].double() * c[3].double()[:, None]).abs()
    g = (c[0].double() * c[2].double()).abs()
    # terms of dx before its rounding: each carries the few half steps of its products; the mean adds 42
    terms = c[3].double()[:, None] * (g + xhat * (g * xhat).mean(-1, keepdim=True))
    if dh:
        terms = terms + c[4].double().abs()
    d = (dx[:T].double().cpu() - rx).abs()
    assert bool((d <= U * rx.abs() + REL * terms).all()), float((d / (U * rx.abs() + REL * terms)).max())
    # dweight: at most T / 296 + 1 rows, ten partials and five levels of sums in a row
    depth = T / 296 + 1 + 10 + 5 + 3
    tw = (c[0].double().abs() * xhat).sum(0)
    assert bool(((dw.double().cpu() - rw).abs() <= depth * F32 * tw).all())


def test_backward_parts_and_repeat(moe):
    T, H = 700, 1032
    h, w, dy, up = draw((T, H), 1), draw((H,), 2), draw((T, H), 3), draw((T, H), 4)
    rstd = torch.rsqrt(h.float().pow(2).mean(-1) + 1e-5)
    ws = moe.workspace(moe.moe_rmsnorm_bwd_workspace_size(T, H))
    dx, dw = torch.empty_like(h), torch.empty(H, device="cuda")
    moe.moe_rmsnorm_bwd(dy, h, w, rstd, up, dx, dw, ws)
    dx2, dw2 = torch.empty_like(h), torch.empty(H, device="cuda")
    moe.moe_rmsnorm_bwd(dy, h, w, rstd, up, dx2, None, None)
    ws.fill_(255)
    moe.moe_rmsnorm_bwd(dy, h, w, rstd, up, None, dw2, ws)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)  # bitwise, whatever the workspace holds
    acc = up.clone()
    moe.moe_rmsnorm_bwd(dy, h, w, rstd, acc, acc, None, None)  # dX over dh
    assert torch.equal(acc, dx)


def test_graph_replay_and_side_stream(moe):
    T, H = 257, 2048
    x, r, w = draw((T, H), 1), draw((T, H), 2), draw((H,), 3)
    ref = run_fwd(moe, x, r, w, 1e-5)
    o = {n: torch.zeros_like(t) for n, t in ref.items()}
    xs, rs = torch.zeros_like(x), torch.zeros_like(r)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(g, stream=st):
            moe.moe_rmsnorm_fwd(xs, rs, w, 1e-5, o["h"], o["y"], o["q"], o["sf"], o["rstd"])
        xs.copy_(x)
        rs.copy_(r)
        g.replay()
    st.synchronize()
    for n in o:
        assert torch.equal(o[n], ref[n]), n
