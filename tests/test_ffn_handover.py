"""MXFP8 feed-forward block on CTA pairs: the hand-over of the scales.

Either CTA of a pair writes scales to its own shared memory with ordinary stores, and the first CTA's tensor core reads
both CTAs'. Between the stores and the read stand, in this order: the writer's proxy fence, its release at the cluster's
scope, its arrival, and the issuer's wait with an acquire at that scope. No run shows a missing one for certain, so the
order is checked in the source; and on the GPU outputs must follow every change of the scales exactly."""
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_layer_aux_b200", "csrc")
BF = torch.bfloat16


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_scales_are_released_before_the_arrival():
    src = source("dense.cuh")
    loader = src[src.index("warp == 10"):]
    loader = loader[:loader.index("tfull[acc]")]  # the epilogue's first wait
    stores, proxy = loader.rindex("make_uint4(cur["), loader.index("fence_proxy_async_smem()")
    release, arrive = loader.find("release_smem_cluster()"), loader.index("arrive_first<CG>(&full[")
    assert stores < proxy < release < arrive
    assert "fence.release.sync_restrict::shared::cta.cluster" in source("elect.cuh")


def test_the_issuer_acquires_what_the_other_cta_released():
    src = source("dense.cuh")
    issuer = src[src.index("else if (warp == 1)"):src.index("warp == 10")]
    assert re.search(r"if constexpr \(C::MX && CG == 2\)\s*ready = mbar_wait_warp_cluster\(&full\[stage\]", issuer)
    wait = source("elect.cuh")
    wait = wait[wait.index("bool mbar_wait_warp_cluster"):]
    fence = "fence.acquire.sync_restrict::shared::cluster.cluster"
    assert wait.index("try_wait.parity.relaxed.cluster") < wait.index(fence)


def quantised(moe, w):
    q = torch.empty(w.shape, dtype=torch.uint8, device="cuda")
    sf = torch.empty(w.shape[:-1] + (w.shape[-1] // 32,), dtype=torch.uint8, device="cuda")
    moe.moe_quantize_mxfp8(w, q, sf)
    return q, sf


# Pairs of 128 columns cut along K, of 128 whole, and of 256, in either product or both (148 SMs)
@pytest.mark.gpu
@pytest.mark.parametrize("T,H,F", [(96, 6912, 1792), (150, 6912, 2560), (200, 4096, 8064), (2500, 2560, 2048),
                                   (3000, 1024, 4096)])
def test_outputs_follow_the_scales(moe, T, H, F):
    """W_u's scales times 2^j and W_d's times 2^k: the activation's scales move by j, its codes stay, and y is 2^(j + k)
    times what it was, to the bit (all in range). A word of an earlier pass, or of the ring's last turn, would show."""
    def draw(shape, seed, std):
        g = torch.Generator(device="cuda").manual_seed(seed)
        return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)

    cfg = moe.make_ffn_config(T, H, F, dtype="mxfp8")
    ws = moe.workspace(moe.moe_ffn_workspace_size(cfg))
    y = torch.empty((T, H), dtype=BF, device="cuda")
    sets = []
    for i in range(2):
        x, *w = (draw(s, 10 * i + n, std) for n, (s, std) in enumerate(
            [((T, H), 1.0), ((F, H), H ** -0.5), ((F, H), H ** -0.5), ((H, F), F ** -0.5)]))
        sets.append((quantised(moe, x), [quantised(moe, v) for v in w]))

    def run(i, j, k):
        (xq, xs), ((gq, gs), (uq, us), (dq, ds)) = sets[i]
        moe.moe_ffn_fwd(cfg, xq, xs, gq, uq, dq, gs, us + j, ds + k, y, None, ws)
        return y.clone()

    refs = [run(i, 0, 0) for i in range(2)]
    for n in range(24):
        i, j, k = n % 2, n % 3, n % 4
        assert torch.equal(run(i, j, k), refs[i] * 2.0 ** (j + k)), n
    torch.cuda.synchronize()
    assert moe.moe_get_device_status() == 0
