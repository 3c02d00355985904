"""The forms of the feed-forward block's kernels, dense and streaming, that the sizes of test_gpu_ffn.py leave out,
against 64 bits. What all these sizes take together is checked on the host by test_ffn_plans.py."""
import pytest

import test_gpu_ffn as ffn

pytestmark = pytest.mark.gpu

FORMS = [(1, 5768, 64), (1, 7584, 4744), (57, 5240, 9800), (58, 1864, 64), (60, 2200, 13344), (60, 5376, 11400),
         (65, 64, 12488), (115, 2432, 12440), (137, 3976, 64), (268, 7896, 6456), (269, 6528, 7784), (3281, 264, 9984),
         (5299, 64, 6456), (5327, 3384, 64), (6391, 4848, 144), (6729, 136, 9992), (7245, 528, 3816),
         (8096, 3328, 336)]
FORMS_MX = [(17, 256, 14720), (17, 5120, 14976), (18, 256, 11648), (18, 9472, 9856), (36, 4864, 128), (113, 3584, 8832),
            (138, 9984, 12160), (156, 9984, 10624), (259, 6400, 11008)]
STREAM = [(1, 8, 64), (1, 8, 9760), (1, 64, 8), (1, 72, 8), (1, 128, 5384), (1, 448, 3000), (1, 600, 1600), (1, 19232, 8),
          (11, 8, 2128), (12, 8, 2176), (47, 5024, 2048)]
STREAM_MX = [(1, 256, 9600), (1, 3840, 128), (1, 8192, 128), (11, 256, 4096), (11, 256, 4224)]


@pytest.mark.parametrize("T,H,F", FORMS + STREAM)
def test_bf16(moe, T, H, F):
    ffn.test_forward_bf16(moe, T, H, F)
    ffn.test_backward_bf16(moe, T, H, F)


@pytest.mark.parametrize("T,H,F", FORMS_MX + STREAM_MX)
def test_mxfp8(moe, T, H, F):
    ffn.test_forward_mxfp8(moe, T, H, F)
