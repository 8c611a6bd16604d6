"""The rule that chooses a tile's rows (csrc/tile_rows.cuh), built for the host: what it takes is one of the choices whose
measured times (one GB300, us of 256, 128 and 64 rows) are within 5 % of the best."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from conftest import ROOT

SOURCE = """
#include "tile_rows.cuh"
using namespace moe;
extern "C" int choose(const unsigned* parts, unsigned rows16, unsigned longest, int tiles, int steps, int pairs, int slope) {
    RowSums s{{parts[0], parts[1], parts[2]}, rows16, longest};
    const float share = (float)tiles / (float)pairs;
    return slope ? choose_rows<true>(s, (float)steps, share) : choose_rows<false>(s, (float)steps, share);
}
extern "C" int turns(unsigned several_parts, unsigned several_groups, unsigned single_parts) {
    return by_turns(several_parts, several_groups, single_parts);
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    gxx = shutil.which("g++") or shutil.which("c++")
    if not gxx:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("rule")
    (d / "rule.cpp").write_text(SOURCE)
    subprocess.run([gxx, "-std=c++17", "-O2", "-shared", "-fPIC", "-I", os.path.join(ROOT, "moe_expert_layer_count_gb300", "csrc"),
                    str(d / "rule.cpp"), "-o", str(d / "rule.so")], check=True)
    lib = ctypes.CDLL(str(d / "rule.so"))
    lib.turns.argtypes = [ctypes.c_uint] * 3
    f = lib.choose
    f.argtypes = [ctypes.POINTER(ctypes.c_uint), ctypes.c_uint, ctypes.c_uint, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int]

    def choose(counts, outputs, tile_outputs, depth, slope=False, pairs=76):
        parts = (ctypes.c_uint * 3)(*(sum(-(-r // (256 >> c)) for r in counts) for c in range(3)))
        return f(parts, sum((r + 15) // 16 for r in counts), max(counts, default=0), -(-outputs // tile_outputs), -(-depth // 64), pairs, slope)
    choose.lib = lib
    return choose


def zipf(experts, topk, tokens, s, seed=1):
    """Rows of each expert: every token's distinct experts, drawn by popularity rank ** -s."""
    r = random.Random(seed)
    popular = [(i + 1.0) ** -s for i in range(experts)]
    r.shuffle(popular)
    counts = [0] * experts
    for _ in range(tokens):
        for e in sorted(range(experts), key=lambda e: r.random() ** (1 / popular[e]), reverse=True)[:topk]:
            counts[e] += 1
    return counts


# groups, outputs, depth, {operator: times of 256, 128, 64 rows}. fwd: 2 N outputs of K; gated: N (128 a tile); dgrad and the
# gated backward pass: N
MEASURED = [
    ([2048], 512, 512, dict(fwd=(8.63, 7.35, 8.72), dgrad=(8.29, 6.84, 6.46), gated=(10.25, 8.46, 9.78), bwd=(15.33, 11.15, 9.19))),
    ([512] * 3, 384, 1024, dict(fwd=(10.81, 9.14, 8.63), dgrad=(10.72, 8.80, 8.25), gated=(12.52, 10.30, 9.53), bwd=(17.76, 12.86, 10.64))),
    ([1000] * 2, 768, 2048, dict(fwd=(15.84, 19.81, 25.76), dgrad=(15.12, 12.60, 18.53), gated=(17.34, 21.22, 27.02), bwd=(22.39, 16.95, 21.48))),
    ([7521], 216, 184, dict(fwd=(7.78, 7.91, 9.10), dgrad=(7.35, 6.63, 7.57), gated=(9.23, 9.49, 10.59), bwd=(15.67, 11.49, 12.05))),
    ([100] * 16, 512, 512, dict(fwd=(8.58, 8.58, 9.51), dgrad=(7.57, 7.53, 7.20), gated=(9.58, 9.58, 10.40), bwd=(11.00, 11.00, 9.69))),
    ([1024] * 8, 1024, 1024, dict(fwd=(27.51, 33.78, 57.27), dgrad=(17.51, 21.65, 30.82), gated=(29.94, 36.34, 60.69), bwd=(32.76, 32.21, 38.58))),
    ([512] * 16, 768, 2048, dict(fwd=(38.19, 51.21, 84.85), dgrad=(26.86, 28.77, 46.67), gated=(40.95, 53.26, 85.34), bwd=(41.55, 38.03, 52.68))),
    ([300] * 16, 768, 2048, dict(fwd=(32.85, 36.69, 54.63), dgrad=(20.58, 19.81, 32.63), gated=(35.13, 38.90, 56.85), bwd=(29.99, 27.51, 37.92))),
    ([8192], 64, 2048, dict(fwd=(15.66, 13.57, 19.06), dgrad=(15.45, 13.33, 18.73), gated=(17.26, 14.68, 20.12), bwd=(20.21, 16.44, 21.07))),
    ([65536], 64, 256, dict(fwd=(16.74, 16.57, 23.46), dgrad=(15.76, 18.53, 28.83))),
    ([200] * 128, 768, 2048, dict(fwd=(159.94, 185.97, 304.83), dgrad=(90.67, 102.52, 155.84), bwd=(120.36, 126.22, 170.47))),
    ([512] * 128, 768, 2048, dict(fwd=(251.86, 337.24, 624.85), dgrad=(142.93, 179.54, 313.94), gated=(264.53, 346.45, 633.56), bwd=(211.79, 226.38, 350.03))),
    (zipf(128, 8, 256, 1.2), 768, 2048, dict(fwd=(124.22, 131.73, 128.14), dgrad=(62.78, 69.07, 66.34), gated=(125.84, 133.18, 129.85), bwd=(67.70, 72.18, 70.01))),
    (zipf(128, 8, 512, 1.2), 768, 2048, dict(fwd=(134.24, 137.14, 135.14), dgrad=(71.54, 68.94, 70.86))),
    (zipf(128, 8, 2048, 0.6), 768, 2048, dict(fwd=(151.36, 153.05, 204.34), dgrad=(80.52, 83.02, 104.56), gated=(156.17, 158.12, 211.02), bwd=(103.32, 100.56, 117.83))),
    (zipf(128, 8, 2048, 1.2), 768, 2048, dict(fwd=(151.09, 160.35, 203.00), dgrad=(82.93, 86.80, 104.03), gated=(156.34, 165.87, 209.41), bwd=(105.99, 102.78, 117.12))),
    (zipf(60, 4, 333, 1.2), 712, 1000, dict(fwd=(33.31, 32.67, 34.85), gated=(35.32, 34.00, 35.96), bwd=(26.77, 25.29, 22.18))),
    (zipf(60, 4, 2000, 1.2), 712, 1000, dict(fwd=(43.45, 46.56, 60.13), dgrad=(27.47, 26.21, 34.79), gated=(49.00, 52.37, 64.48), bwd=(48.82, 38.86, 43.96))),
    (zipf(16, 2, 1000, 1.2), 512, 1024, dict(fwd=(12.22, 14.35, 13.33), gated=(13.84, 15.59, 14.26), bwd=(17.08, 13.96, 11.92))),
]


@pytest.mark.parametrize("case", range(len(MEASURED)))
def test_takes_what_measured_fast(rule, case):
    counts, N, K, times = MEASURED[case]
    for op, t in times.items():
        outputs, tile = {"fwd": (2 * N, 256), "gated": (N, 128)}.get(op, (N, 256))
        c = rule(counts, outputs, tile, K, op == "bwd")
        assert t[c] <= 1.05 * min(t), (op, c, t)


def test_choice_is_always_one(rule):
    """No groups, no rows, one row, sums past 2^31: a choice comes back, and the largest tiles where all are alike."""
    for counts in ([], [0], [1], [2 ** 31 - 1], [2 ** 31 - 1] * 2, [0] * 1024):
        for slope in (False, True):
            assert rule(counts, 8, 256, 8, slope) in (0, 1, 2)
    assert rule([64] * 128, 1536, 256, 2048) == 0 and rule([1] * 128, 1536, 256, 2048) == 0


# 128 experts, top-8, 768 x 2048, forward products: us in the groups' own order and by turns
@pytest.mark.parametrize("tokens,s,seed,own,turns", [
    (1024, 1.2, 2, 141.8, 141.7), (1024, 1.2, 3, 135.5, 138.8), (1024, 0.6, 3, 138.2, 139.3), (2048, 0.6, 2, 151.2, 152.8),
    (2048, 0.6, 4, 149.8, 154.2), (2048, 1.2, 4, 150.7, 151.2), (4096, 1.2, 2, 189.7, 179.5), (4096, 1.2, 3, 185.3, 181.1),
    (8192, 1.2, 3, 289.1, 278.4), (8192, 1.2, 4, 291.9, 278.7)])
def test_order_that_measured_fast(rule, tokens, s, seed, own, turns):
    counts = zipf(128, 8, tokens, s, seed)
    several = [r for r in counts if r > 256]
    taken = rule.lib.turns(sum(-(-r // 256) for r in several), len(several), sum(0 < r <= 256 for r in counts))
    assert (turns if taken else own) <= 1.01 * min(own, turns)


def test_order_of_groups_of_one_kind(rule):
    assert rule.lib.turns(2 ** 31, 1, 0) and rule.lib.turns(256, 128, 0) and not rule.lib.turns(1, 1, 1000)


def test_tiles_stay_within_32_bits(rule):
    """Whatever the groups: where the largest tiles are at most 2^30, those of the choice are."""
    r = random.Random(3)
    worst = 0
    for _ in range(20000):
        parts0 = int(2 ** r.uniform(0, 23))
        tiles = int(2 ** r.uniform(0, 30)) // parts0 + 1
        if parts0 * tiles > 2 ** 30:
            continue
        longest = int(2 ** r.uniform(0, 12)) if r.random() < 0.5 else r.randint(1, 300)
        # each group's rows between one more than a multiple of 256 and the multiple: up to two and four times the parts
        parts = (parts0, r.randint(parts0, 2 * parts0), 0)
        parts = (parts[0], parts[1], r.randint(parts[1], 2 * parts[1]))
        rows16 = r.randint(parts0, 16 * parts0)
        for slope in (0, 1):
            c = rule.lib.choose((ctypes.c_uint * 3)(*parts), rows16, longest, tiles, int(2 ** r.uniform(0, 10)), min(76, parts[2] * tiles), slope)
            worst = max(worst, parts[c] * tiles)
    assert 2 ** 28 < worst <= 2 ** 30
