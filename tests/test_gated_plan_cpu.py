"""The planner of the gated products, without a GPU: ranges, tile shapes,
forced shapes, workspace and refusals."""

import pytest

from fp4_weight_only_gb300 import binding

SMS, PAIRS = 152, 76


@pytest.fixture(autouse=True)
def free():
    binding.load()
    yield
    binding.set_tile_config()
    binding.set_pair_mode()


def check(p, off, n, k):
    s = p["range_starts"]
    assert s[0] == 0 and s[-1] == p["units"] and len(s) == p["num_ranges"] + 1
    assert all(a < b for a, b in zip(s, s[1:]))                      # every range has work
    assert p["num_ctas"] == p["num_ranges"] * (2 if p["cta_pairs"] else 1) and p["num_ctas"] <= SMS
    rows = 256 if p["cta_pairs"] else 128
    tiles = sum(-(-(b - a) // p["bn"]) for a, b in zip(off, off[1:])) * (2 * n // rows)
    assert p["num_tiles"] == tiles and p["units_per_tile"] == k // 128 // p["ku"] and p["units"] == tiles * p["units_per_tile"]
    assert p["workspace_bytes"] == 4352 + 1024 * p["num_ctas"] * p["bn"]
    assert p["bn"] <= 128 or p["ku"] == 1
    assert not p["cta_pairs"] or p["bn"] >= 128


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "nvfp4_f16"])
@pytest.mark.parametrize("m", [1, 16, 17, 100, 256, 300, 1200, 4096])
@pytest.mark.parametrize("n,k", [(64, 128), (64, 8192), (192, 640), (512, 1024), (2752, 2048), (14336, 4096), (28672, 8192)])
def test_dense(m, n, k, fmt):
    p = binding.gated_plan([0, m], n, k, fmt, SMS, PAIRS)
    check(p, [0, m], n, k)
    assert not p["cta_pairs"] or n % 128 == 0
    assert not binding.gated_plan([0, m], n, k, fmt, SMS, 0)["cta_pairs"]


def test_choices():
    """Few rows of large matrices take small tiles, prompts pairs of 256 rows; small matrices whole tiles."""
    one = binding.gated_plan([0, 1], 28672, 8192, "nvfp4", SMS, PAIRS)
    assert one["bn"] == 16 and one["num_ctas"] == SMS
    prompt = binding.gated_plan([0, 4096], 28672, 8192, "nvfp4", SMS, PAIRS)
    assert prompt["bn"] == 256 and prompt["cta_pairs"]
    small = binding.gated_plan([0, 300], 2048, 512, "nvfp4", SMS, PAIRS)
    per = small["units_per_tile"]
    assert all(x % per == 0 for x in small["range_starts"])


@pytest.mark.parametrize("off", [[0, 1], [0, 0, 5], [0, 39, 66, 160, 190, 215, 403, 442, 512], [0] * 30 + [700], list(range(65))])
def test_grouped(off):
    p = binding.gated_plan(off, 1408, 2048, "mxfp4", SMS, PAIRS)
    check(p, off, 1408, 2048)


def test_ranges_follow_the_groups_heights():
    """Groups of few rows have lower tiles, whose units take less time: ranges over them hold more."""
    off = [0] + [200 + 8 * i for i in range(9)]        # one group of 200 rows, eight of 8
    p = binding.gated_plan(off, 14336, 4096, "mxfp4", SMS, PAIRS)
    check(p, off, 14336, 4096)
    sizes = [b - a for a, b in zip(p["range_starts"], p["range_starts"][1:])]
    if p["bn"] >= 128:
        assert sizes[0] < sizes[-1]


def test_forced_shapes():
    for bn in (16, 32, 64, 128, 256):
        for ku in (1, 2) if bn <= 64 else (1,):
            binding.set_tile_config(bn, ku)
            for mode in (0, 1, 2):
                binding.set_pair_mode(mode)
                p = binding.gated_plan([0, 200], 1024, 1024, "nvfp4", SMS, PAIRS)
                check(p, [0, 200], 1024, 1024)
                assert (p["bn"], p["ku"]) == (bn, ku)
                if mode:
                    assert p["cta_pairs"] == (mode == 2 and bn >= 128)


def test_refusals():
    assert binding.gated_plan([0, 0], 64, 128, "nvfp4", SMS, PAIRS)["num_ranges"] == 0
    for bad, status in ((([0, 1], 96, 128), 2), (([0, 1], 64, 100), 2), (([1, 2], 64, 128), 1), (([0] * 66, 64, 128), 2),
                        (([0, 1], 1 << 24, 128), 2), (([0, 1], 0, 128), 2)):
        with pytest.raises(binding.PetitError) as e:
            binding.gated_plan(*bad, "nvfp4", SMS, PAIRS)
        assert e.value.status == status, bad
    for sms, pairs in ((0, 0), (1025, 0), (152, 161), (152, -1)):
        with pytest.raises(binding.PetitError):
            binding.gated_plan([0, 1], 64, 128, "nvfp4", sms, pairs)
