"""The shared-memory plan of the layer for a few tokens, compiled by the host compiler: every part
lies in the CTA's memory, none on another one, and the sizes that are taken have two stages."""
import itertools
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_expert_layer_gb300", "csrc")
FIELDS = ("xpitch hpitch hrest sum_at unit_at row_at red_at queue_at ring_at swords zwords whole "
          "sub_bytes stages bytes block step_k").split()
ROOM = 226 * 1024


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("few_plan")
    src, exe = d / "main.cc", d / "main"
    prints = " ".join(["%d"] * len(FIELDS))
    src.write_text('#include <cstdio>\n#include "few_plan.h"\n' + """
int main() {
  int T, H, inter, units, rows, four, group, sb, zeros, as, az, whole;
  while (scanf("%d %d %d %d %d %d %d %d %d %d %d %d", &T, &H, &inter, &units, &rows, &four, &group,
               &sb, &zeros, &as, &az, &whole) == 12) {
    const moe::FewPlan p = moe::few_plan(T, H, inter, units, rows, four, group, sb, zeros, as, az, whole);
    printf("PRINTS\\n", ARGS);
  }
}
""".replace("PRINTS", prints).replace("ARGS", ", ".join("p." + f for f in FIELDS)))
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o",
                    str(exe)], check=True)

    def run(cases):
        r = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, c)) for c in cases),
                           text=True, capture_output=True)
        assert r.returncode == 0
        return [dict(zip(FIELDS, map(int, line.split()))) for line in r.stdout.splitlines()]

    return run


def up(v, to):
    return -(-v // to) * to


def cases(four):
    for T, H, inter, k in itertools.product((1, 2, 5, 8), (32, 288, 2304, 7168, 8192),
                                            (32, 736, 2048, 65536), (1, 8, 32)):
        units, rows = T * k + 1, T * (k + 1)
        if not four:
            yield T, H, inter, units, rows, 0, 0, 2, 0, 1, 1, 0
            continue
        for group, sb, zeros in itertools.product((0, 32, 64, 128), (2, 4), (0, 1)):
            if group and (H % group or inter % group):
                continue
            sizes = [n // group if group else 1 for n in (H, inter)]
            yield (T, H, inter, units, rows, 1, group, sb, zeros,
                   int(all(n * sb % 4 == 0 for n in sizes)), int(all(n % 4 == 0 for n in sizes)),
                   int(group > 0 and H % 256 == 0 and inter % 256 == 0))


@pytest.mark.parametrize("four", [False, True])
def test_parts_lie_apart(plans, four):
    made = list(cases(four))
    taken = 0
    for c, p in zip(made, plans(made), strict=True):
        T, H, inter, units, rows, _, group, sb, zeros, *_, whole = c
        step = 256 if four else 64
        assert p["step_k"] == step
        # x, its block sums; h over both where it fits
        blocks = up(H, step) // p["block"] if four else 0
        assert p["xpitch"] >= 2 * up(H, step) and p["xpitch"] % 16 == 0
        assert p["sum_at"] >= T * p["xpitch"]
        front = p["sum_at"] + blocks * 8 * 4
        if p["hpitch"]:
            assert p["hpitch"] >= 2 * up(inter, step) and p["hpitch"] % 16 == 0
            assert p["hrest"] >= rows * p["hpitch"]
            front = max(front, rows * p["hpitch"] * (1 if four else 2))
            assert p["stages"] in (0, 4)
        assert p["unit_at"] >= front and p["unit_at"] % 8 == 0
        assert p["row_at"] >= p["unit_at"] + units * 8
        assert p["red_at"] >= p["row_at"] + (units + 1 + rows) * 4 and p["red_at"] % 16 == 0
        assert p["queue_at"] >= p["red_at"] + 2 * 16 * 128 * 4
        assert p["ring_at"] >= p["queue_at"] + 4 * 16 * 4 and p["ring_at"] % 128 == 0
        # a stage: sixteen rows of 128 bytes, then their scales and zero points
        groups = 16 * 4 * (p["swords"] + p["zwords"])
        assert p["sub_bytes"] >= 2048 + groups and p["sub_bytes"] % 16 == 0
        if four:
            n = step // group if group else 1
            assert 4 * p["swords"] >= n * sb and (4 * p["zwords"] >= n if zeros else True)
            if whole:
                assert 4 * p["swords"] == n * sb
        if p["stages"] < 2:
            continue
        taken += 1
        assert p["bytes"] == p["ring_at"] + 16 * p["stages"] * p["sub_bytes"] <= ROOM
        # the parts of down lie over the rings: 16 warps, 64 channels, 8 tokens
        assert 16 * 64 * 8 * 4 <= 16 * p["stages"] * p["sub_bytes"]
    assert taken > len(made) * 3 // 4


def test_the_largest_batches_have_four_stages(plans):
    got = plans([(8, 8192, 2048, 65, 72, 0, 0, 2, 0, 1, 1, 0), (8, 4096, 1024, 49, 56, 1, 128, 2, 0, 1, 1, 1),
                 (1, 7168, 2048, 9, 9, 1, 128, 2, 0, 1, 1, 1)])
    assert [p["stages"] for p in got][1:] == [4, 4] and got[0]["stages"] >= 2
