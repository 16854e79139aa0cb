"""That the orthogonalised update's GPU tests reach each way in which it runs, by its
plans on the CPU."""
import test_orthogonalize_padding_gpu as padding
from test_more_plans_cpu import plans, pytestmark  # noqa: F401


def test_padded_rows_on_every_tile(plans):  # noqa: F811
    found = plans([f"orthogonalize {batch} {M} {N}" for batch, M, N, _ in padding.SIZES])
    ways = {(way.split(" update")[0], min(size[1], size[2]) <= 128)
            for plan, size in zip(found, padding.SIZES) for way in plan.split("polynomial ")[1:]}
    assert all(min(M, N) % 8 for _, M, N, _ in padding.SIZES)
    assert ("tile=64 whole", True) in ways      # with sums apart
    for way in ("tile=64 whole", "tile=128 whole", "tile=256 whole", "tile=128 whole+runs", "tile=256 +runs"):
        assert (way, False) in ways, way
    assert any(" strips" in plan for plan in found) and any(" small" in plan for plan in found)
