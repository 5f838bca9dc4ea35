"""The launch rules of the 4-bit products, compiled by the host compiler."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_expert_layer_gb300", "csrc")


def compiled(tmp_path_factory, name, body):
    d = tmp_path_factory.mktemp(name)
    src, exe = d / "main.cc", d / "main"
    src.write_text('#include <cstdio>\n#include "w4_plan.h"\n' + body)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o",
                    str(exe)], check=True)
    return str(exe)


@pytest.fixture(scope="module")
def splits(tmp_path_factory):
    """(SMs, tiles, panels) -> split, for lines of three numbers."""
    exe = compiled(tmp_path_factory, "split", """
int main() {
  long long tiles;
  int sms, panels;
  while (scanf("%d %lld %d", &sms, &tiles, &panels) == 3)
    printf("%d\\n", moe::w4_choose_split(tiles, panels, sms));
}
""")

    def run(cases):
        r = subprocess.run([exe], input="\n".join("%d %d %d" % c for c in cases), text=True,
                           capture_output=True)
        assert r.returncode == 0, f"ended with {r.returncode}"
        return [int(v) for v in r.stdout.split()]

    return run


def test_a_split_exists_for_every_device(splits):
    # partitions of a few SMs too: the count of a GPC's clusters must not be zero
    cases = [(sms, tiles, panels) for sms in list(range(1, 40)) + [76, 132, 152, 160]
             for tiles in (1, 7, 56, 1000, 2**31) for panels in (1, 2, 3, 4, 8, 14, 8192)]
    got = splits(cases)
    assert len(got) == len(cases)
    for (sms, tiles, panels), split in zip(cases, got):
        assert split in (1, 2, 4, 8) and split <= panels


def test_splits_of_a_full_device(splits):
    # one row tile: as many CTAs as there are panels; thousands: none
    assert splits([(152, 1, 1), (152, 1, 4), (152, 1, 14), (152, 48, 12), (152, 5000, 14)]) == \
        [1, 4, 8, 4, 1]


FIXED = {2: 98304, 1: 82944}  # rings and x panels for 16-bit and int8 x


@pytest.fixture(scope="module")
def memory(tmp_path_factory):
    """(fixed bytes, groups, groups a panel, scale bytes, zeros) -> the layout."""
    exe = compiled(tmp_path_factory, "memory", """
int main() {
  int fixed, groups, panel, es, zeros;
  while (scanf("%d %d %d %d %d", &fixed, &groups, &panel, &es, &zeros) == 5) {
    const moe::W4Memory m = moe::w4_memory(fixed, groups, panel, es, zeros != 0);
    printf("%d %d %d %d %d %d\\n", m.sunit, m.sstride, m.zunit, m.zstride, m.bytes, m.per_sm);
  }
}
""")

    def run(cases):
        r = subprocess.run([exe], input="\n".join("%d %d %d %d %d" % c for c in cases), text=True,
                           capture_output=True, check=True)
        return [dict(zip(("sunit", "sstride", "zunit", "zstride", "bytes", "per_sm"),
                         map(int, line.split()))) for line in r.stdout.splitlines()]

    return run


ALL = [(FIXED[x], groups, panel, es, zeros) for x in (1, 2) for groups in range(1, 260)
       for panel in (4, 8, 16) for es in (2, 4) for zeros in (0, 1)]


def test_two_ctas_fit_an_sm(memory):
    # 228 KB an SM, 1 KB a CTA besides its own; 16-bit scales fit for every count
    # of groups (groups of 32 with zero points at K = 256, 768, 2304, ... had not)
    for (fixed, groups, panel, es, zeros), m in zip(ALL, memory(ALL)):
        assert m["bytes"] == fixed + 256 * (m["sstride"] + m["zstride"]) <= 227 * 1024
        assert m["per_sm"] == (2 if 2 * (m["bytes"] + 1024) <= 228 * 1024 else 1)
        if es == 2 or fixed == FIXED[1] or panel < 16:
            assert m["per_sm"] == 2, (fixed, groups, panel, es, zeros)


def test_row_strides_hold_a_panel_from_any_start(memory):
    for (_, groups, panel, es, zeros), m in zip(ALL, memory(ALL)):
        for unit, stride, size in ((m["sunit"], m["sstride"], es), (m["zunit"], m["zstride"], 1)):
            if size == 1 and not zeros:
                assert stride == 0
                continue
            assert unit in (4, 8, 16) and stride % unit == 0
            start = max(r * groups * size % unit for r in range(16))  # inside its unit
            assert start + panel * size <= stride
            if start == 0 and unit > 4:
                assert groups * size % unit == 0 and panel * size % unit == 0
            # rows that are whole numbers of a stage's groups are read in one load
            gps = panel // 4
            if gps > 1 and groups % gps == 0 and size < 4:
                load = min(gps * size, 8)
                assert unit % load == 0 or unit % 4 == 0 and load <= 4
            # eight rows' words in different banks
            words = [r * stride // 4 % 32 for r in range(8)]
            assert len(set(words)) == 8


def test_a_lone_cta_an_sm_halves_the_slots(tmp_path_factory):
    exe = compiled(tmp_path_factory, "slots", """
int main() {
  // 144 tiles of 12 panels fill 152 SMs once when one CTA fits, half when two do
  printf("%d %d\\n", moe::w4_choose_split(144, 12, 152, 1), moe::w4_choose_split(144, 12, 152, 2));
}
""")
    one, two = map(int, subprocess.check_output([exe], text=True).split())
    assert one == 1 and two == 2
