"""RMSNorm and feed-forward entry points: refusals on the host before anything is launched (no GPU needed), sizes of
workspaces, and the 64-bit definitions' gradients against central differences."""
import ctypes

import pytest
import torch

from block_ref import ffn_bwd, ffn_fwd, norm_bwd, norm_fwd

OK, INVALID, UNSUPPORTED, ALIGN, WS = 0, 1, 2, 3, 4
P = 0x10000  # aligned, never dereferenced (every call fails validation first)


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_aux_b200 import binding
    binding.load()
    return binding


def test_rmsnorm_refusals(B):
    f = B.load().moe_rmsnorm_fwd

    def call(T=4, H=256, x=P, r=P, w=P, eps=1e-5, h=P, y=P, q=P, sf=P, rstd=P):
        return f(T, H, x, r, w, eps, h, y, q, sf, rstd, None)

    assert call(T=0) == INVALID and call(H=0) == INVALID and call(T=-1) == INVALID
    assert call(H=252) == UNSUPPORTED and call(H=16392) == UNSUPPORTED and call(H=264) == UNSUPPORTED  # y_q: % 32
    assert call(x=None) == INVALID and call(w=None) == INVALID
    assert call(eps=-1.0) == INVALID and call(eps=float("nan")) == INVALID
    assert call(sf=None) == INVALID and call(q=None) == INVALID
    assert call(h=None, y=None, q=None, sf=None) == INVALID
    for n in ("x", "r", "w", "h", "y", "q"):
        assert call(**{n: P + 8}) == ALIGN, n
    assert call(rstd=P + 2) == ALIGN


def test_rmsnorm_bwd_refusals(B):
    lib = B.load()
    f, size = lib.moe_rmsnorm_bwd, lib.moe_rmsnorm_bwd_workspace_size
    need = size(4, 256)
    assert need == 4 * 256 * 4 and size(5000, 256) == 296 * 256 * 4
    assert size(0, 256) == 0 and size(4, 100) == 0 and size(4, 20000) == 0

    def call(T=4, H=256, dy=P, h=P, w=P, rstd=P, dh=P, dx=P, dw=P, ws=P, n=need):
        return f(T, H, dy, h, w, rstd, dh, dx, dw, ws, n, None)

    assert call(T=0) == INVALID and call(H=100) == UNSUPPORTED
    for n in ("dy", "h", "w", "rstd"):
        assert call(**{n: None}) == INVALID, n
    assert call(dx=None, dw=None) == INVALID
    for n in ("dy", "h", "w", "dh", "dx", "ws"):
        assert call(**{n: P + 8}) == ALIGN, n
    assert call(dw=P + 2) == ALIGN and call(rstd=P + 1) == ALIGN
    assert call(ws=None) == WS and call(n=need - 1) == WS


def test_ffn_sizes(B):
    lib = B.load()
    by = ctypes.byref
    for bad in (dict(T=0), dict(H=0), dict(F=-8), dict(H=260), dict(F=100), dict(dtype=7), dict(dtype="nvfp4"),
                dict(T=(1 << 24) + 1), dict(F=(1 << 20) + 8), dict(dtype="mxfp8", H=384), dict(dtype="mxfp8", F=192),
                dict(dtype="mxfp8", save_for_bwd=1)):
        c = B.make_ffn_config(**{**dict(T=4, H=256, F=512), **bad})
        assert lib.moe_ffn_workspace_size(by(c)) == 0 and lib.moe_ffn_saved_size(by(c)) == 0, bad
        assert lib.moe_ffn_bwd_workspace_size(by(c)) == 0, bad
        code = INVALID if bad.get("T") == 0 or bad.get("H") == 0 or bad.get("F") == -8 or bad.get("dtype") == 7 \
            else UNSUPPORTED
        assert lib.moe_ffn_fwd(by(c), P, None, P, P, P, None, None, None, P, None, P, 1 << 40, None) == code, bad
        assert lib.moe_ffn_bwd(by(c), P, P, P, P, P, P, P, P, P, P, P, 1 << 40, None) == code, bad
    c = B.make_ffn_config(T=100, H=264, F=520, save_for_bwd=1)
    assert lib.moe_ffn_saved_size(by(c)) >= 100 * 3 * 520 * 2
    assert lib.moe_ffn_bwd_workspace_size(by(c)) >= 100 * 2 * 520 * 2
    # few tokens need no room for partial sums
    assert lib.moe_ffn_workspace_size(by(B.make_ffn_config(T=1, H=4096, F=14336))) == 14336 * 2
    assert lib.moe_ffn_workspace_size(None) == 0


def test_ffn_refusals(B):
    lib = B.load()
    by = ctypes.byref
    big = 1 << 40

    def fwd(c, x=P, x_sf=None, g=P, u=P, d=P, gs=None, us=None, ds=None, y=P, saved=None, ws=P, n=big):
        return lib.moe_ffn_fwd(by(c), x, x_sf, g, u, d, gs, us, ds, y, saved, ws, n, None)

    c = B.make_ffn_config(T=64, H=256, F=512)
    for n in ("x", "g", "u", "d", "y"):
        assert fwd(c, **{n: None}) == INVALID, n
        assert fwd(c, **{n: P + 8}) == ALIGN, n
    for n in ("x_sf", "gs", "us", "ds"):
        assert fwd(c, **{n: P}) == INVALID, n            # bf16 has no scales
    assert fwd(c, saved=P) == INVALID                    # not asked for
    need = lib.moe_ffn_workspace_size(by(c))
    assert fwd(c, n=need - 1) == WS and fwd(c, ws=None) == WS and fwd(c, ws=P + 8) == ALIGN
    cs = B.make_ffn_config(T=64, H=256, F=512, save_for_bwd=1)
    assert fwd(cs) == INVALID and fwd(cs, saved=P + 4) == ALIGN
    m = B.make_ffn_config(T=64, H=256, F=512, dtype="mxfp8")
    s = dict(gs=P, us=P, ds=P)
    for n in s:
        assert fwd(m, **{**s, n: None}) == INVALID, n
        assert fwd(m, **{**s, n: P + 2}) == ALIGN, n
    assert fwd(m, **s, x_sf=P + 1) == ALIGN
    assert fwd(m, **s, n=lib.moe_ffn_workspace_size(by(m)) - 1) == WS

    bneed = lib.moe_ffn_bwd_workspace_size(by(cs))

    def bwd(c=cs, dy=P, x=P, g=P, u=P, d=P, saved=P, dx=P, dg=P, du=P, dd=P, ws=P, n=bneed):
        return lib.moe_ffn_bwd(by(c), dy, x, g, u, d, saved, dx, dg, du, dd, ws, n, None)

    assert bwd(c=c) == INVALID                           # nothing was saved
    assert bwd(c=m) == UNSUPPORTED
    for n in ("dy", "x", "g", "u", "d", "saved", "dg", "du"):
        assert bwd(**{n: None}) == INVALID, n            # dW_g and dW_u come together
    assert bwd(dx=None, dg=None, du=None, dd=None) == INVALID
    for n in ("dy", "x", "g", "u", "d", "saved", "dx", "dg", "du", "dd", "ws"):
        assert bwd(**{n: P + 8}) == ALIGN, n
    assert bwd(n=bneed - 1) == WS and bwd(ws=None) == WS


def _differences(f, t, step=1e-6):
    d = torch.empty_like(t)
    for i in range(t.numel()):
        v = t.reshape(-1)[i].item()
        t.reshape(-1)[i] = v + step
        a = f()
        t.reshape(-1)[i] = v - step
        b = f()
        t.reshape(-1)[i] = v
        d.reshape(-1)[i] = (a - b) / (2 * step)
    return d


def test_norm_gradient_is_the_differences():
    torch.manual_seed(0)
    x, r, w = (torch.randn(s, dtype=torch.float64) for s in ((3, 8), (3, 8), (8,)))
    dy, dh = torch.randn(3, 8, dtype=torch.float64), torch.randn(3, 8, dtype=torch.float64)

    def loss():
        h, _, y = norm_fwd(x, r, w, 1e-3)
        return float((y * dy).sum() + (h * dh).sum())

    h, rstd, _ = norm_fwd(x, r, w, 1e-3)
    dx, dw = norm_bwd(dy, h, w, rstd, dh)
    assert torch.allclose(dx, _differences(loss, x), rtol=1e-6, atol=1e-7)
    assert torch.allclose(dx, _differences(loss, r), rtol=1e-6, atol=1e-7)
    assert torch.allclose(dw, _differences(loss, w), rtol=1e-6, atol=1e-7)


def test_ffn_gradient_is_the_differences():
    torch.manual_seed(1)
    x, W_g, W_u, W_d = (torch.randn(s, dtype=torch.float64) for s in ((3, 5), (4, 5), (4, 5), (5, 4)))
    dy = torch.randn(3, 5, dtype=torch.float64)
    loss = lambda: float((ffn_fwd(x, W_g, W_u, W_d)[3] * dy).sum())  # noqa: E731
    r = ffn_bwd(dy, x, W_g, W_u, W_d)
    for n, t in (("dX", x), ("dW_g", W_g), ("dW_u", W_u), ("dW_d", W_d)):
        assert torch.allclose(r[n], _differences(loss, t), rtol=1e-6, atol=1e-7), n
