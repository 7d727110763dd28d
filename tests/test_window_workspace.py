"""The workspace bounds that the header states for attention through a window."""
import pytest


@pytest.fixture(scope="module")
def size():
    from paged_kv_cache_varlen_gb300 import binding, build

    build.build()
    return binding.load_library().pkv_window_attention_workspace_size


@pytest.mark.parametrize("eight", [0, 1])
@pytest.mark.parametrize("d", [64, 128])
def test_bounds(size, eight, d):
    short = long = 0
    for hkv in [*range(1, 60), 100, 152, 153, 304, 456, 457, 1000]:
        for g in [*range(1, 35), 48, 64, 100, 128, 256]:
            if g * hkv > 32767:
                continue
            most = max(1, 32 // g)
            for q in (1, most):
                short = max(short, size(q, g * hkv, hkv, d, 131072, 0, 0, eight))
            if g <= 128:
                long = max(long, size(8192, g * hkv, hkv, d, 131072, 0, 0, eight))
    # pieces of 3 x 152 CTAs, two of 16 rows each, their maxima and sums (and the cuts);
    # those of 2 x 8 warps of 152 CTAs
    pieces = 3 * 152 * 2 * 16 * (d + 2) * 4
    assert pieces // 2 < short <= pieces + 152 * 3 * 20 + 256
    assert short <= 8 * 10 ** 6 and long <= 46 * 10 ** 6
    assert long <= short + 152 * 2 * 8 * 32 * (d + 2) * 4 + 8192
