"""Which tile a call takes (host only): the GPU tests' sizes reach every instance."""
import pytest

from group_tiles import ADAPTER_SIZES, ADAPTERS, DW, DWS, DX, DXS, FORWARD, FORWARDS, choice


@pytest.mark.parametrize("op,sizes,instances", [
    (FORWARD, FORWARDS, ["16x32", "32x64", "64x64", "64x128", "128x64", "128x128", "128x128 deep", "256x128", "256x256"]),
    (DX, DXS, ["32x128", "64x128", "128x128 transposed", "256x128", "256x256"]),
    (DW, DWS, ["128x128 transposed", "256x128"])])
def test_products(op, sizes, instances):
    for name, *size in sizes:
        assert choice(op, *size) == name, size
    assert {name for name, *_ in sizes} == set(instances)


def test_adapters():
    for name, T, groups, N, K, R in ADAPTER_SIZES:
        assert choice(ADAPTERS, T, 1, groups, N, K, R) == name, (T, groups, N, K, R)
    names = {name for name, *_ in ADAPTER_SIZES}
    assert {n for n in names if not n.startswith("whole")} == \
        {f"token {r}" for r in (1, 2, 3, 4)} | {f"slices {r}" for r in (32, 64, 128)}
    whole = [n[len("whole "):].split(", inner ") for n in names if n.startswith("whole")]
    assert {t for t, _ in whole} == {"16x32", "32x64", "64x64", "64x128", "128x64", "128x128", "128x128 deep", "256x128",
                                     "256x256"}
    assert {i for _, i in whole} == {"row", "16x16", "32x16", "32x32", "64x16", "32x64", "64x32", "64x64"}
    # both ways to add the ranks in the small tiles
    for tile in ("16x32", "32x64", "64x64", "64x128"):
        ranks = [R for name, *_, R in ADAPTER_SIZES if name.startswith(f"whole {tile},")]
        assert min(ranks) <= 32 < max(ranks)
