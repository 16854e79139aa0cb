"""How the 8-bit layers and the orthogonalised update run, on the CPU (a host build of
their C entry points and plans, ``cpp/more_plans.cpp``): runs cover every stage
once, and the sizes that the GPU tests use reach every kernel."""
import os
import random
import subprocess

import pytest

import linear_plan
import test_i8_gpu as i8
import test_orthogonalize_gpu as ortho

ROOT = linear_plan.ROOT
pytestmark = pytest.mark.skipif(linear_plan.hipcc() is None, reason="needs hipcc")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plans") / "plans")
    subprocess.run([linear_plan.hipcc(), "--offload-arch=gfx950", "--offload-host-only", "-O1", "-std=c++17",
                    f"-I{ROOT}/include", f"-I{ROOT}/dense_gemm_optimisation_row_amd/csrc", "-x", "hip",
                    os.path.join(ROOT, "tests", "cpp", "more_plans.cpp"), "-o", exe], check=True, capture_output=True)

    def ask(lines):
        out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True).stdout
        found = out.splitlines()
        assert len(found) == len(lines)
        return [f.split(":", 1)[1] for f in found]
    return ask


def test_every_stage_of_drawn_sizes_is_in_one_run(plans):
    rng = random.Random(7)
    lines = []
    for _ in range(1500):
        m, n = (int(round(2 ** rng.uniform(0, 13))) for _ in range(2))
        lines.append(f"orthogonalize {rng.choice([1, 1, 1, 2, 3, 8, 30])} {m} {n}")
    lines += ["orthogonalize 1 1 2097120", "orthogonalize 300 64 64", "orthogonalize 1000 30 30"]
    for line, plan in zip(lines, plans(lines)):
        assert "BAD" not in plan and "status" not in plan, (line, plan)


def test_parts_of_drawn_8_bit_products_cover_them(plans):
    rng = random.Random(8)
    lines = [f"{rng.choice(['linear', 'gated'])} {int(2 ** rng.uniform(0, 13))} {int(2 ** rng.uniform(0, 13))} "
             f"{int(2 ** rng.uniform(0, 17))} {rng.randint(0, 1)} {rng.randint(0, 1)}" for _ in range(1500)]
    for line, plan in zip(lines, plans(lines)):
        assert "BAD" not in plan and plan.endswith("status 0"), (line, plan)


def test_the_gpu_tests_reach_every_8_bit_kernel(plans):
    lines = [f"{what} {M} {N} {K} {op} {off}" for M, N, K in i8.SHAPES + i8.LARGE for what in ("linear", "gated")
             for op in (0, 1) for off in (0, 1)]
    text = "\n".join(plans(lines))
    for tile in ("256x256", "128x128", "128x64", "64x64"):
        for gated in ("", " gated"):
            assert f"ring {tile}{gated} splits" in text, tile + gated
    for blocks in (1, 2, 3, 4):
        assert f"rows blocks={blocks} " in text and f"rows blocks={blocks} gated" in text
    assert " copy " in text and " copy-turned" in text and " join" in text


def test_the_gpu_tests_reach_every_way_of_the_update(plans):
    lines = [f"orthogonalize {batch} {M} {N}" for M, N, _ in ortho.EXACT for batch in (1, 3)]
    text = "\n".join(plans(lines))
    assert " small" in text and " strips" in text
    many = plans([f"orthogonalize {batch} {M} {N}" for batch, M, N in ortho.MANY])
    assert [p.split()[0] for p in many] == ["small", "strips", "strips", "gram", "strips"]
    for side in (64, 128, 256):
        for product in ("gram", "polynomial", "update"):
            assert f"{product} tile={side} " in text, (product, side)
    for way in ("gram tile=64 whole+runs", "gram tile=64 +runs", "gram tile=128 whole+runs", "gram tile=256 +runs",
                "polynomial tile=256 +runs", "update tile=128 whole+runs", "update tile=256 whole"):
        assert way in text, way
