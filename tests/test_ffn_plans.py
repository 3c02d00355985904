"""Launch plans of the feed-forward block's kernels, evaluated on the host (nvcc, no GPU): 148 SMs."""
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    """Compiles tests/<name>.cu; returns a function that runs it on arguments and gives its lines."""
    if shutil.which("nvcc") is None:
        pytest.skip("no nvcc")
    out = tmp_path_factory.mktemp("plans")

    def run(name, args):
        exe = out / name
        if not exe.exists():
            subprocess.run(["nvcc", "-O1", "-std=c++17", "--expt-relaxed-constexpr", "-gencode",
                            "arch=compute_100a,code=sm_100a", "-o", str(exe), os.path.join(HERE, name + ".cu")],
                           check=True, capture_output=True)
        return subprocess.run([str(exe), *map(str, args)], check=True, capture_output=True,
                              text=True).stdout.splitlines()

    return run


@pytest.mark.parametrize("mx", [False, True])
def test_down_weights_are_asked_for_evenly(host, mx):
    """The stages of the down weights that the gate/up kernel asks into L2 follow, for each CTA of a tile, those that
    its ring takes, as many for each, within the budget: a tile is done when the last of its CTAs is."""
    rng = random.Random(1)
    args = [] if mx else [48, 4096, 14336, 48, 2048, 5504, 56, 4096, 14336, 1, 4096, 14336]
    for _ in range(400):
        step = (256, 128) if mx else (8, 64)
        args += [rng.randint(1, 16 if mx else 56), step[0] * rng.randint(1, 8192 // step[0]),
                 step[1] * rng.randint(1, 16384 // step[1])]
    split = 0
    for line in host("stream_plan", ["mx" if mx else "bf16", *args]):
        shape, plan, asked = (part.split() for part in line.split(":", 2))
        cs, KS, stages, s, r, tiles, stage_bytes, budget = map(int, plan)
        split += cs > 1
        per = budget // (tiles * cs * stage_bytes)
        for k, a in enumerate(asked):
            rank, span = a.split(":")
            a0, a1 = map(int, span.rsplit("-", 1)) if not span.startswith("-") else (-1, -1)
            k0, k1 = k * KS // cs, (k + 1) * KS // cs  # this CTA's part of K
            first, last = k0 + stages, min(k0 + stages + per, k1)
            want = (first, last) if first < last else (-1, -1)
            assert int(rank) == k and (a0, a1) == want, line
    assert mx or split > 20


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("pairs", [74, 72])  # CTA pairs that fit the device at once
def test_the_gpu_tests_take_every_form(host, mx, pairs):
    """Every form of the dense GEMM that plan() gives some size of T <= 8192, H <= 10240 and F <= 16384 is taken by a
    size of the GPU tests: for each product the CTAs per tile, the columns, and how a last round's tiles are cut; and
    the order of the tiles."""
    import test_gpu_ffn as a
    import test_gpu_ffn_forms as b
    tested = a.FORMS_MX + a.MX_SHAPES + b.FORMS_MX if mx else a.FORMS + a.SHAPES + b.FORMS
    kind = "mx" if mx else "bf16"
    have = {line.split()[0] for line in host("dense_plan", [kind, pairs, "list", *(v for t in tested for v in t)])}
    found = host("dense_plan", [kind, pairs, "search", 200000, 2])
    assert len(found) > (25 if mx else 80)
    missing = [line for line in found if line.split()[0] not in have]
    assert not missing, missing


@pytest.mark.parametrize("mx", [False, True])
def test_the_gpu_tests_take_every_streaming_form(host, mx):
    """The same for the streaming kernels, of sizes up to H, F <= 25600."""
    import test_gpu_ffn as a
    import test_gpu_ffn_forms as b
    tested = a.MX_SHAPES + b.STREAM_MX if mx else a.SHAPES + b.STREAM
    kind = "mx" if mx else "bf16"
    have = {line.split()[0] for line in host("stream_plan", [kind, "list", *(v for t in tested for v in t)])}
    found = host("stream_plan", [kind, "search", 200000, 3])
    assert len(found) > (12 if mx else 25)
    missing = [line for line in found if line.split()[0] not in have]
    assert not missing, missing
