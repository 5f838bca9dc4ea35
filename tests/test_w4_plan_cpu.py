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
