"""That the orthogonalised update's GPU tests reach each way in which it runs, by its
plans on the CPU."""
import test_orthogonalize_padding_gpu as padding
import test_orthogonalize_terms_gpu as terms
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


def ways(plans, sizes):
    """(product, tile, whole and runs, up to 128 rows) of all, and the sizes not in products."""
    products, other = set(), {}
    for plan, (batch, M, N) in zip(plans([f"orthogonalize {b} {m} {n}" for b, m, n in sizes]), sizes):
        words = plan.split()
        if words[0] in ("small", "strips"):
            other.setdefault(words[0], []).append((batch, M, N))
        for i, w in enumerate(words):
            if w in ("gram", "polynomial", "update"):
                products.add((w, int(words[i + 1][5:]), words[i + 2], min(M, N) <= 128))
    return products, other


def test_both_terms_in_every_way(plans):  # noqa: F811
    products, other = ways(plans, terms.SIZES)
    for product in ("gram", "polynomial", "update"):
        for tile in (64, 128, 256):
            assert {w for p, t, w, few in products if (p, t, few) == (product, tile, False)}, (product, tile)
        assert any(p == product and few and tile == 64 for p, tile, _, few in products) or product == "update"
    for tile in (64, 128, 256):
        found = {w for _, t, w, _ in products if t == tile}
        assert any("runs" in w for w in found) and "whole" in found, (tile, found)
    assert {(min(M, N) + 31) // 32 for _, M, N in other["strips"]} == {1, 2, 3, 4} and len(other["small"]) >= 4


def test_full_matrices_in_every_way(plans):  # noqa: F811
    products, other = ways(plans, terms.FULL)
    assert {tile for _, tile, _, _ in products} == {64, 128, 256}
    assert {(min(M, N) + 31) // 32 for _, M, N in other["strips"]} == {1, 2, 3, 4} and other["small"]
