"""The barrier model of the shared-prefix decode where a CTA has more than two
segments (its queries are loaded again in every phase), where key tiles fold as
well, and where four fold into the smallest ring; and the host's rules that the model repeats,
as the source states them.  SHAPES is also what the GPU runs."""
import os
import random
import re

import pytest

from test_shared_protocol import Cta, _grid

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "integer_only_quantized_b200", "csrc")

# B, Hkv, G, Lp, Lmax, d -> what it is for: fold, ring stages, segments of a CTA, tiles of a
# segment among more than two (0: at most two segments, the queries stay)
SHAPES = {
    (1, 512, 1, 1000, 20, 64): (4, 14, 4, 2),
    (2, 600, 1, 600, 0, 64): (4, 18, 5, 2),
    (3, 600, 1, 600, 10, 128): (4, 7, 5, 2),
    (33, 600, 1, 300, 3, 64): (2, 14, 5, 2),
    (40, 400, 1, 600, 9, 128): (2, 5, 3, 3),
    (300, 90, 2, 260, 4, 64): (1, 10, 4, 3),
    (129, 100, 3, 390, 6, 128): (1, 5, 3, 4),
    (129, 128, 1, 900, 3, 128): (1, 7, 3, 8),
    (30, 32, 1, 2400, 100, 128): (4, 5, 1, 0),
}


def plan(case):
    """(fold, ring stages, most segments of a CTA, most tiles of a segment
    among more than two) of a call."""
    grid = _grid(case)
    ctas = [Cta(case, i, grid) for i in range(grid)]
    assert all(c.q_stays == (0 < len(c.segs) < 3) for c in ctas)
    return (ctas[0].F, ctas[0].stages, max(len(c.segs) for c in ctas),
            max((n for c in ctas if len(c.segs) > 2 for _, n in c.segs), default=0))


def name(case):
    return "B{}k{}G{}p{}m{}d{}".format(*case)


@pytest.mark.parametrize("case", SHAPES, ids=name)
def test_shapes_are_what_they_are_for(case):
    assert plan(case) == SHAPES[case]


@pytest.mark.parametrize("slow", [None, "producer", "qk", "pv", "team 0", "team 1", "q"])
@pytest.mark.parametrize("case", SHAPES, ids=name)
def test_no_order_blocks(case, slow):
    rng = random.Random(str((case, slow)))
    grid = _grid(case)
    for cta in {0, grid - 1, *(rng.randrange(grid) for _ in range(12))}:
        for _ in range(4):
            Cta(case, cta, grid).run(rng, slow)


def test_drawn_cases():
    """Many heads, few tiles: more than two segments in most."""
    rng = random.Random(12)
    reloads = 0
    for _ in range(300):
        case = (rng.choice([1, 3, 9, 31, 64, 70, 130]), rng.randrange(100, 900), rng.choice([1, 1, 2, 4]),
                rng.randrange(1, 1500), rng.choice([0, 9, 100]), rng.choice([64, 128]))
        grid = _grid(case)
        cta = Cta(case, rng.randrange(grid), grid)
        reloads += not cta.q_stays
        cta.run(rng, rng.choice([None, "team 0", "team 1", "pv", "q", "qk"]))
    assert reloads > 150


@pytest.mark.parametrize("file,rule", [
    ("shared_api.cuh", "a.fold = 1; for (int f = 2; f <= 4; f *= 2) if (a.R <= intattn::shared::kBM / f && "
                       "static_cast<long long>(Hkv) * ((a.key_tiles + f - 1) / f) >= sms) a.fold = f;"),
    ("shared_api.cuh", "a.seg_tiles = (a.key_tiles + a.fold - 1) / a.fold;"),
    ("shared_api.cuh", "own_keys = static_cast<long long>(B) * Hkv * Lmax, prefix_keys = static_cast<long long>(Hkv) * Lp; "
                       "a.own_slots = Lmax == 0 ? 0 : 2 * own_keys <= prefix_keys ? 1 : 2;"),
    ("shared_api.cuh", "a.stages = (intattn::shared::kRingBytes - a.own_slots * intattn::shared::kOwnWarps * "
                       "intattn::shared::kOwnBytes) / (intattn::shared::kBN * d);"),
    ("shared_api.cuh", "const long long own = static_cast<long long>(B) * Hkv * ((Lmax + 127) / 128); const int grid = "
                       "static_cast<int>(std::min<long long>(sms, std::max<long long>(std::max(tiles, own), 1)));"),
    ("shared_api.cuh", "a.seg_cost = tiles > grid ? 4 : 0;"),
    ("shared_kernel.cuh", "constexpr int kBM = 128;"), ("shared_kernel.cuh", "constexpr int kBN = 128;"),
    ("shared_kernel.cuh", "constexpr int kRingBytes = 144 * 1024;"), ("shared_kernel.cuh", "constexpr int kOwnWarps = 8;"),
    ("shared_kernel.cuh", "constexpr int kOwnBytes = 4096;"), ("shared_kernel.cuh", "constexpr int kPBufs = 4;"),
    ("shared_kernel.cuh", "const int p = a.cta_cost * i + min(i, a.cta_more); const int u = p / each; "
                          "return u * a.seg_tiles + min(p - u * each, a.seg_tiles);"),
    ("shared_kernel.cuh", "q_stays = t0 < t1 && (t1 - 1) / args.seg_tiles - t0 / args.seg_tiles < 2;"),
])
def test_the_model_follows_the_rules_in_the_source(file, rule):
    """A changed rule has to be changed in the model (here and in test_shared_protocol.py) too."""
    with open(os.path.join(CSRC, file)) as f:
        code = re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", f.read()))
    assert rule in code
