"""The gated feed-forward block: forward in bf16 and MXFP8, backward in bf16, against 64 bits."""
import pytest
import torch

from block_ref import F32, RMS_U, check_sum, ffn_bwd, ffn_fwd, mx_quant, mx_values

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# (T, H, F): both sides of every choice by the number of tokens, odd sizes, tails of a tile and of a k-block, many
# tiles with a rest, one tile
SHAPES = [(1, 8, 8), (1, 256, 512), (1, 2056, 1544), (3, 1000, 264), (8, 520, 1040), (9, 256, 384), (16, 136, 4104),
          (17, 264, 200), (31, 2048, 768), (33, 1032, 136), (48, 2056, 1544), (64, 1032, 1160), (60, 1032, 2312), (50, 520, 4096), (65, 1032, 1160),
          (65, 256, 512), (2, 136, 9480), (40, 264, 19208), (64, 19016, 136), (1, 4096, 9600), (3, 320, 19208),
          (2, 64, 19208), (5, 19016, 320), (2, 19016, 64), (127, 72, 200), (128, 384, 640), (129, 136, 1032), (200, 8, 8), (257, 520, 2568), (300, 2048, 4104),
          (1001, 1288, 1160), (1100, 136, 520), (1030, 512, 328), (520, 328, 640),
          (1500, 2568, 3592)]


def draw(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


def inputs(T, H, F, seed=0):
    return (draw((T, H), seed + 1), draw((F, H), seed + 2, H ** -0.5), draw((F, H), seed + 3, H ** -0.5),
            draw((H, F), seed + 4, F ** -0.5))


def guarded(T, n):
    return torch.full((T + 1, n), 7.0, dtype=BF, device="cuda")


def forward(moe, x, W_g, W_u, W_d, save=0):
    T, H = x.shape
    F = W_g.shape[0]
    cfg = moe.make_ffn_config(T, H, F, save_for_bwd=save)
    y = guarded(T, H)
    saved = moe.workspace(moe.moe_ffn_saved_size(cfg)) if save else None
    ws = moe.workspace(moe.moe_ffn_workspace_size(cfg)).fill_(255)  # NaN, should any of it be read before written
    moe.moe_ffn_fwd(cfg, x, None, W_g, W_u, W_d, None, None, None, y[:T], saved, ws)
    torch.cuda.synchronize()
    assert moe.moe_get_device_status() == 0
    assert bool((y[T] == 7.0).all())
    return cfg, y[:T], saved


def check_forward(y, x, W_g, W_u, W_d):
    g, u, a, ref = ffn_fwd(x, W_g, W_u, W_d)
    sigma = (a.pow(2) @ W_d.double().pow(2).T).sqrt()
    # each term of y carries the rounding of a
    return check_sum(y, ref, sigma, RMS_U, W_d.shape[1])


@pytest.mark.parametrize("T,H,F", SHAPES)
def test_forward_bf16(moe, T, H, F):
    t = inputs(T, H, F)
    _, y, _ = forward(moe, *t)
    check_forward(y, *t)


@pytest.mark.parametrize("T,H,F", SHAPES)
def test_backward_bf16(moe, T, H, F):
    x, W_g, W_u, W_d = inputs(T, H, F)
    dy = draw((T, H), 9)
    cfg, y, saved = forward(moe, x, W_g, W_u, W_d, save=1)
    assert torch.equal(y, forward(moe, x, W_g, W_u, W_d)[1])  # saving changes nothing
    o = {"dX": guarded(T, H), "dW_g": guarded(F, H), "dW_u": guarded(F, H), "dW_d": guarded(H, F)}
    ws = moe.workspace(moe.moe_ffn_bwd_workspace_size(cfg)).fill_(255)
    moe.moe_ffn_bwd(cfg, dy, x, W_g, W_u, W_d, saved, o["dX"][:T], o["dW_g"][:F], o["dW_u"][:F], o["dW_d"][:H], ws)
    torch.cuda.synchronize()
    assert moe.moe_get_device_status() == 0
    for n, v in o.items():
        assert bool((v[-1] == 7.0).all()), n
    r = ffn_bwd(dy, x, W_g, W_u, W_d)
    sq = lambda v: v.double().pow(2)  # noqa: E731
    # dgate and dup are rounded to bf16 (relative, RMS_U), and come from gate and up kept to 24 bits, each off by up to
    # 2^-16 = P RMS_U of itself. dgate = v u f(g), f = silu', |f'| <= 1/2; dup = v silu(g).
    P = 2.0 ** -16 / RMS_U
    # To that come the fp32 sums g, u and v: off by up to 2 K 2^-24 of the size of their sums (check_sum), which is
    # no small part of a sum that cancels (a g of 1.28e-5 whose terms add up to a size of 1 was 3.2e-7 off: 2.5 % of
    # it, and of dup = v silu(g)).
    g, u, a, _ = ffn_fwd(x, W_g, W_u, W_d)
    v = (dy.double() @ W_d.double()).abs()
    s = torch.sigmoid(g)
    f = s * (1 + g * (1 - s))
    off = lambda p, q, K: 2 * F32 * K * (sq(p) @ sq(q)).sqrt() / RMS_U  # noqa: E731
    og, ou, ov = off(x, W_g.T, H), off(x, W_u.T, H), off(dy, W_d, H)
    og, ou = og + P * g.abs(), ou + P * u.abs()
    eg = (sq(r["dg"]) + sq(v * u / 2 * og) + sq(v * f * ou) + sq(u * f * ov)).sqrt()
    eu = (sq(r["du"]) + sq(v * f * og) + sq(g * s * ov)).sqrt()
    check_sum(o["dX"][:T], r["dX"], (sq(eg) @ sq(W_g) + sq(eu) @ sq(W_u)).sqrt(), RMS_U, 2 * F)
    check_sum(o["dW_g"][:F], r["dW_g"], (sq(eg).T @ sq(x)).sqrt(), RMS_U, T)
    check_sum(o["dW_u"][:F], r["dW_u"], (sq(eu).T @ sq(x)).sqrt(), RMS_U, T)
    ea = (sq(a) + sq(u * f * og) + sq(g * s * ou)).sqrt()
    check_sum(o["dW_d"][:H], r["dW_d"], (sq(dy).T @ sq(ea)).sqrt(), RMS_U, T)


def test_backward_parts(moe):
    """Data and weight gradients run apart give the same bits as together, whatever the workspace holds."""
    T, H, F = 300, 520, 1160
    x, W_g, W_u, W_d = inputs(T, H, F)
    dy = draw((T, H), 9)
    cfg, _, saved = forward(moe, x, W_g, W_u, W_d, save=1)
    ws = moe.workspace(moe.moe_ffn_bwd_workspace_size(cfg))
    new = lambda *s: torch.empty(s, dtype=BF, device="cuda")  # noqa: E731
    a = [new(T, H), new(F, H), new(F, H), new(H, F)]
    b = [new(T, H), new(F, H), new(F, H), new(H, F)]
    moe.moe_ffn_bwd(cfg, dy, x, W_g, W_u, W_d, saved, *a, ws)
    moe.moe_ffn_bwd(cfg, dy, None, W_g, W_u, W_d, saved, b[0], None, None, None, ws.fill_(255))
    moe.moe_ffn_bwd(cfg, dy, None, None, None, W_d, saved, None, None, None, b[3], ws.fill_(255))
    moe.moe_ffn_bwd(cfg, dy, x, None, None, W_d, saved, None, b[1], b[2], None, ws.fill_(255))
    for p, q in zip(a, b):
        assert torch.equal(p, q)


# ------------------------------------------------------------------ MXFP8

MX_SHAPES = [(1, 256, 128), (5, 4096, 512), (48, 4096, 640), (64, 2048, 1280), (1, 7168, 2048), (5, 512, 384), (8, 256, 640), (12, 768, 256), (20, 1024, 512),
             (33, 768, 4096), (64, 512, 256), (65, 512, 256), (7, 256, 19072), (50, 256, 9600), (3, 19200, 128),
             (130, 768, 640), (700, 1024, 384), (2100, 512, 4224), (1300, 4352, 640)]


def mx_of(moe, w):
    q = torch.empty(w.shape, dtype=torch.uint8, device="cuda")
    sf = torch.empty(w.shape[:-1] + (w.shape[-1] // 32,), dtype=torch.uint8, device="cuda")
    moe.moe_quantize_mxfp8(w, q, sf)
    return q, sf


@pytest.mark.parametrize("T,H,F", MX_SHAPES)
def test_forward_mxfp8(moe, T, H, F):
    x, W_g, W_u, W_d = inputs(T, H, F)
    (gq, gs), (uq, us), (dq, ds) = (mx_of(moe, w) for w in (W_g, W_u, W_d))
    xq, xs = mx_of(moe, x)
    cfg = moe.make_ffn_config(T, H, F, dtype="mxfp8")
    out = []
    for xin, sfin in ((x, None), (xq, xs)):
        y = guarded(T, H)
        ws = moe.workspace(moe.moe_ffn_workspace_size(cfg)).fill_(255)
        moe.moe_ffn_fwd(cfg, xin, sfin, gq, uq, dq, gs, us, ds, y[:T], None, ws)
        torch.cuda.synchronize()
        assert moe.moe_get_device_status() == 0
        assert bool((y[T] == 7.0).all())
        out.append(y[:T])
    assert torch.equal(out[0], out[1])  # x quantised on the way or before
    val = lambda q, s: mx_values(q.cpu(), s.cpu()).cuda()  # noqa: E731
    xv, gv, uv, dv = val(xq, xs), val(gq, gs), val(uq, us), val(dq, ds)
    g, u = xv @ gv.T, xv @ uv.T
    a = g * torch.sigmoid(g) * u
    av = mx_quant(a.cpu())[0].cuda()
    # An element of a whose fp32 value falls on the other side of a rounding border moves by one e4m3 step, at most
    # 2^-3 of it; a block whose maximum crosses a power of two changes all of it. fp32 dot products are off by about
    # sqrt(H) 2^-24 of their terms' size, so that a share of some sqrt(H) 2^-24 / 2^-4 of the elements (below 1 in
    # 1000 for H <= 8192, and 1 in 10^4 for H < 10^4) does: terms' errors of root mean square sqrt(1e-3) / 8.
    # Such an error is not small beside its term, as check_sum's are: it is 1/8 of it, or nothing. Eight deviations,
    # sqrt(1e-3) sqrt(F) = 1.7 mean terms at F = 2944, are passed by the step of one term of 14 mean terms (of 28, if
    # the step is the binade's finest, 1/16). Terms a d are products of three normal factors, of which one in 10^6 is
    # that large; a row has F 1e-4 = 0.3 such steps, so of 5 10^7 outputs some tens are expected to pass, each by no
    # more than the step of its largest term, and a second such step in one row in 10^6 of those.
    sigma = (av.pow(2) @ dv.pow(2).T).sqrt()
    step = lambda i, j: (av[i.cuda()] * dv[j.cuda()]).abs().amax(1) / 8  # noqa: E731
    check_sum(out[0], av @ dv.T, sigma, (1e-3 ** 0.5) / 8, F, step)


def test_mxfp8_few_and_many_tokens_agree(moe):
    """The same tokens through the streaming kernels and the tensor-core kernels: the same values, up to sums in
    another order (bf16 steps) and the rare step of the activation's quantisation."""
    H, F = 1024, 512
    x, W_g, W_u, W_d = inputs(80, H, F)
    w = [mx_of(moe, v) for v in (W_g, W_u, W_d)]
    ys = []
    for T in (80, 8):
        cfg = moe.make_ffn_config(T, H, F, dtype="mxfp8")
        y = torch.empty((T, H), dtype=BF, device="cuda")
        moe.moe_ffn_fwd(cfg, x[:T], None, w[0][0], w[1][0], w[2][0], w[0][1], w[1][1], w[2][1], y, None,
                        moe.workspace(moe.moe_ffn_workspace_size(cfg)))
        ys.append(y[:8].double())
    d = (ys[0] - ys[1]).norm() / ys[1].norm()
    assert float(d) < 2.0 ** -8


def run_mxfp8(moe, T, H, F, x, x_sf, w):
    cfg = moe.make_ffn_config(T, H, F, dtype="mxfp8")
    y = torch.empty((T, H), dtype=BF, device="cuda")
    moe.moe_ffn_fwd(cfg, x, x_sf, w[0][0], w[1][0], w[2][0], w[0][1], w[1][1], w[2][1], y, None,
                    moe.workspace(moe.moe_ffn_workspace_size(cfg)).fill_(255))
    torch.cuda.synchronize()
    assert moe.moe_get_device_status() == 0
    return y


@pytest.mark.parametrize("T", [3, 16, 17, 130])
@pytest.mark.parametrize("H,F", [(1024, 512), (768, 640)])
def test_mxfp8_scales_at_any_word(moe, T, H, F):
    """Scales that start 4 bytes past a 16-byte boundary (four k-blocks are read at a time where they may be)."""
    x, W_g, W_u, W_d = inputs(T, H, F)
    w = [mx_of(moe, v) for v in (W_g, W_u, W_d)]
    xq, xs = mx_of(moe, x)

    def moved(s):
        m = torch.full((s.numel() + 16,), 255, dtype=torch.uint8, device="cuda")[4:4 + s.numel()].view(s.shape)
        return m.copy_(s)

    ref = run_mxfp8(moe, T, H, F, xq, xs, w)
    assert torch.equal(run_mxfp8(moe, T, H, F, xq, moved(xs), [(q, moved(s)) for q, s in w]), ref)


@pytest.mark.parametrize("T", [4, 80])
def test_mxfp8_nan_stays_in_its_row(moe, T):
    H, F = 512, 256
    x, W_g, W_u, W_d = inputs(T, H, F)
    w = [mx_of(moe, v) for v in (W_g, W_u, W_d)]
    ref = run_mxfp8(moe, T, H, F, x, None, w)
    bad = x.clone()
    bad[1, 7] = float("nan")
    y = run_mxfp8(moe, T, H, F, bad, None, w)
    keep = [t for t in range(T) if t != 1]
    assert torch.equal(y[keep], ref[keep])
    assert bool(torch.isnan(y[1]).all())


@pytest.mark.parametrize("T,H,F", [(128, 512, 4096), (200, 4096, 1024)])
def test_cut_tiles_repeat(moe, T, H, F):
    """Tiles that are cut along K are added in a fixed order, whatever the pieces' timing."""
    x, W_g, W_u, W_d = inputs(T, H, F)
    w = [mx_of(moe, v) for v in (W_g, W_u, W_d)]
    one = forward(moe, x, W_g, W_u, W_d)[1], run_mxfp8(moe, T, H, F, x, None, w)
    for _ in range(5):
        assert torch.equal(forward(moe, x, W_g, W_u, W_d)[1], one[0])
        assert torch.equal(run_mxfp8(moe, T, H, F, x, None, w), one[1])


def test_refuses_tensors_elsewhere(moe):
    x, W_g, W_u, W_d = inputs(4, 64, 64)
    cfg = moe.make_ffn_config(4, 64, 64)
    ws = moe.workspace(moe.moe_ffn_workspace_size(cfg))
    y = torch.empty_like(x)
    with pytest.raises(ValueError):
        moe.moe_ffn_fwd(cfg, x.cpu(), None, W_g, W_u, W_d, None, None, None, y, None, ws)
    with pytest.raises(ValueError):
        moe.moe_rmsnorm_fwd(x, None, W_g[0].contiguous(), 1e-6, None, y.cpu(), None, None, None)


# ------------------------------------------------------------------ every form of the dense kernel
# One CTA or a pair, 128 or 256 columns, whole tiles or a last round cut along K (a piece per CTA, or one line), and
# both orders of the tiles, alone and in groups of panels: on 148 SMs these sizes, with those of test_gpu_ffn_forms.py,
# take each that plan() gives a product (test_ffn_plans.py).

FORMS = [
    (69, 64, 64), (278, 4904, 64), (327, 64, 9560), (4487, 64, 1568), (65, 1104, 6304),
    (4848, 1584, 64), (1543, 5496, 64), (72, 6192, 1312), (1822, 64, 2336), (70, 5640, 5592),
    (73, 6392, 3856), (3913, 144, 9488), (73, 1856, 8320), (5108, 72, 3080), (139, 6920, 1672),
    (150, 6688, 5016), (135, 2384, 8576), (68, 6752, 6440), (3311, 680, 6592), (3265, 272, 5632),
    (268, 6568, 4544), (172, 6488, 9512), (5422, 4720, 5608), (5296, 5400, 2544), (2359, 2088, 6032),
    (2151, 2360, 5984), (5343, 6480, 4744)]
FORMS_MX = [
    (17, 256, 128), (260, 256, 6528), (388, 9728, 128), (17, 256, 10112), (3620, 2560, 128),
    (18, 8960, 9984), (20, 7936, 3200), (2314, 256, 1024), (141, 6656, 1792), (139, 3328, 7040),
    (129, 9728, 9600), (5224, 9728, 2944), (5860, 9472, 2816), (4661, 4608, 11392),
    (4655, 5888, 10880),
    (17, 9984, 1792), (17, 256, 4992), (21, 9984, 3584), (21, 6400, 11392), (132, 3584, 11264)]


@pytest.mark.parametrize("T,H,F", FORMS)
def test_forms_bf16(moe, T, H, F):
    test_backward_bf16(moe, T, H, F)


@pytest.mark.parametrize("T,H,F", FORMS_MX)
def test_forms_mxfp8(moe, T, H, F):
    test_forward_mxfp8(moe, T, H, F)


# ------------------------------------------------------------------ special values, graphs, streams, the chain

@pytest.mark.parametrize("T", [4, 80])
def test_nonfinite_tokens_stay_in_their_rows(moe, T):
    H, F = 256, 520
    x, W_g, W_u, W_d = inputs(T, H, F)
    ref = forward(moe, x, W_g, W_u, W_d)[1]
    bad = x.clone()
    bad[1, 7] = float("nan")
    bad[2, 9] = float("inf")
    y = forward(moe, bad, W_g, W_u, W_d)[1]
    keep = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(y[keep], ref[keep])
    assert bool(torch.isnan(y[1]).all()) and not bool(torch.isfinite(y[2]).any())


@pytest.mark.parametrize("T", [1, 80])
def test_zero_weights_and_saturated_gates(moe, T):
    H, F = 256, 256
    x, W_g, W_u, W_d = inputs(T, H, F)
    z = torch.zeros_like(W_g)
    assert float(forward(moe, x, z, W_u, W_d)[1].abs().max()) == 0.0
    x = x.abs() + 1
    big = torch.full_like(W_g, 1.0)       # gates of several hundred: silu(g) = g
    big[::2] = -1.0                       # and of minus several hundred: silu(g) = 0, no NaN from exp
    t = (x, big, W_u, W_d)
    check_forward(forward(moe, *t)[1], *t)


@pytest.mark.parametrize("T", [3, 80, 300])
def test_graph_replay_and_two_streams(moe, T):
    """A captured step (forward and backward) replayed on new inputs, beside the same work on another stream with
    buffers of its own, gives the eager results."""
    H, F = 520, 1160
    sets = [(*inputs(T, H, F, 10 * i), draw((T, H), 10 * i + 9)) for i in range(2)]
    cfg = moe.make_ffn_config(T, H, F, save_for_bwd=1)
    new = lambda *s: torch.zeros(s, dtype=BF, device="cuda")  # noqa: E731

    def buffers():
        return {"y": new(T, H), "dX": new(T, H), "dW_g": new(F, H), "dW_u": new(F, H), "dW_d": new(H, F),
                "saved": moe.workspace(moe.moe_ffn_saved_size(cfg)),
                "ws": moe.workspace(moe.moe_ffn_workspace_size(cfg)),
                "bws": moe.workspace(moe.moe_ffn_bwd_workspace_size(cfg))}

    def step(b, x, W_g, W_u, W_d, dy):
        moe.moe_ffn_fwd(cfg, x, None, W_g, W_u, W_d, None, None, None, b["y"], b["saved"], b["ws"])
        moe.moe_ffn_bwd(cfg, dy, x, W_g, W_u, W_d, b["saved"], b["dX"], b["dW_g"], b["dW_u"], b["dW_d"], b["bws"])

    names = ("y", "dX", "dW_g", "dW_u", "dW_d")
    refs = []
    for s in sets:
        b = buffers()
        step(b, *s)
        refs.append([b[n].clone() for n in names])
    torch.cuda.synchronize()
    static = [t.clone() for t in sets[0]]
    b0, b1 = buffers(), buffers()
    s0, s1 = torch.cuda.Stream(), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s0):
        step(b0, *static)
    for i in (0, 1, 0):
        with torch.cuda.stream(s0):
            for d, v in zip(static, sets[i]):
                d.copy_(v)
            g.replay()
        with torch.cuda.stream(s1):
            step(b1, *sets[1 - i])
        s0.synchronize()
        s1.synchronize()
        for k, n in enumerate(names):
            assert torch.equal(b0[n], refs[i][k]) and torch.equal(b1[n], refs[1 - i][k]), (i, n)
    assert moe.moe_get_device_status() == 0


def test_norm_ffn_norm_chain(moe):
    """A dense layer as it stands in a stack: norm, block, the next norm with the block's output added to the
    residual stream, and the backward through all of them, against 64 bits."""
    from block_ref import U, norm_bwd, norm_fwd
    T, H, F = 150, 512, 776
    x, W_g, W_u, W_d = inputs(T, H, F)
    w1, w2 = draw((H,), 21, 0.3) + 1, draw((H,), 22, 0.3) + 1
    dy2, dh2 = draw((T, H), 23), draw((T, H), 24)
    new = lambda *s: torch.empty(s, dtype=BF, device="cuda")  # noqa: E731
    n1, r1 = new(T, H), torch.empty(T, device="cuda")
    moe.moe_rmsnorm_fwd(x, None, w1, 1e-5, None, n1, None, None, r1)
    cfg = moe.make_ffn_config(T, H, F, save_for_bwd=1)
    f, saved = new(T, H), moe.workspace(moe.moe_ffn_saved_size(cfg))
    moe.moe_ffn_fwd(cfg, n1, None, W_g, W_u, W_d, None, None, None, f, saved,
                    moe.workspace(moe.moe_ffn_workspace_size(cfg)))
    h2, n2, r2 = new(T, H), new(T, H), torch.empty(T, device="cuda")
    moe.moe_rmsnorm_fwd(f, x, w2, 1e-5, h2, n2, None, None, r2)
    ws = moe.workspace(moe.moe_rmsnorm_bwd_workspace_size(T, H))
    dh, dw2 = new(T, H), torch.empty(H, device="cuda")
    moe.moe_rmsnorm_bwd(dy2, h2, w2, r2, dh2, dh, dw2, ws)
    dn, gW = new(T, H), [new(F, H), new(F, H), new(H, F)]
    moe.moe_ffn_bwd(cfg, dh, n1, W_g, W_u, W_d, saved, dn, *gW, moe.workspace(moe.moe_ffn_bwd_workspace_size(cfg)))
    dx, dw1 = new(T, H), torch.empty(H, device="cuda")
    moe.moe_rmsnorm_bwd(dn, x, w1, r1, dh, dx, dw1, ws)
    torch.cuda.synchronize()
    # 64 bits, end to end
    _, q1, m1 = norm_fwd(x, None, w1, 1e-5)
    _, _, _, f64 = ffn_fwd(m1, W_g, W_u, W_d)
    h64, q2, m2 = norm_fwd(x.double() + f64, None, w2, 1e-5)
    dh64, dw2_64 = norm_bwd(dy2, h64, w2, q2, dh2)
    r = ffn_bwd(dh64, m1, W_g, W_u, W_d)
    dx64, dw1_64 = norm_bwd(r["dX"], x, w1, q1, dh64)
    # Norm-wise: every stage adds roundings of root mean square RMS_U to what it passes on (norm 1, a, f, h2 and n2
    # forward; dh, dgate/dup, dn and dx backward), nine in all: 3 RMS_U < 2 U
    for got, ref in ((n2, m2), (h2, h64), (dh, dh64), (dx, dx64), (dw1, dw1_64), (dw2, dw2_64), (gW[0], r["dW_g"]),
                     (gW[1], r["dW_u"]), (gW[2], r["dW_d"])):
        assert float((got.double() - ref).norm() / ref.norm()) < 2 * U


def test_norm_codes_into_ffn(moe):
    """The norm's MXFP8 output is the block's MXFP8 input as it is."""
    T, H, F = 6, 512, 256
    x, W_g, W_u, W_d = inputs(T, H, F)
    w = draw((H,), 5, 0.2) + 1
    q = torch.empty((T, H), dtype=torch.uint8, device="cuda")
    sf = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
    moe.moe_rmsnorm_fwd(x, None, w, 1e-5, None, None, q, sf, None)
    (gq, gs), (uq, us), (dq, ds) = (mx_of(moe, v) for v in (W_g, W_u, W_d))
    cfg = moe.make_ffn_config(T, H, F, dtype="mxfp8")
    y = torch.empty((T, H), dtype=BF, device="cuda")
    moe.moe_ffn_fwd(cfg, q, sf, gq, uq, dq, gs, us, ds, y, None, moe.workspace(moe.moe_ffn_workspace_size(cfg)))
    val = lambda c, s: mx_values(c.cpu(), s.cpu()).cuda()  # noqa: E731
    xv, gv, uv, dv = val(q, sf), val(gq, gs), val(uq, us), val(dq, ds)
    g, u = xv @ gv.T, xv @ uv.T
    av = mx_quant((g * torch.sigmoid(g) * u).cpu())[0].cuda()
    check_sum(y, av @ dv.T, (av.pow(2) @ dv.pow(2).T).sqrt(), (1e-3 ** 0.5) / 8, F)
