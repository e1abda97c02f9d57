"""The entries that lead the tree attention's join to its partial sums, checked on
the host: the rule of csrc/tree_parts.h is compiled as plain C++ and given entries
that a run wrote and entries that no run wrote (whatever bytes a workspace holds)."""

import os
import random
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "local_moe_route_b200", "csrc")
PROGRAM = r"""
#include <cstdio>
#include "tree_parts.h"
using namespace strata::ta;
int main() {
  int run, follow;
  while (std::scanf("%d %d", &run, &follow) == 2) {
    const Head h = {run, follow};
    if (!parts_within(h)) { std::puts("no"); continue; }
    std::printf("%d %d", part_slot(h, 0), follow ? part_slot(h, follow) : part_slot(h, 0));
    for (int i = 0; i <= follow; ++i)
      if (part_slot(h, i) < 0 || part_slot(h, i) >= 2 * MAX_CTAS) std::printf(" outside");
    std::puts("");
  }
}
"""


@pytest.fixture(scope="module")
def answers(tmp_path_factory):
    at = tmp_path_factory.mktemp("parts")
    (at / "parts.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-fsanitize=undefined",
                    "-fno-sanitize-recover", "-I", CSRC, str(at / "parts.cpp"), "-o",
                    str(at / "parts")], check=True)

    def ask(heads):
        text = "".join(f"{r} {f}\n" for r, f in heads)
        out = subprocess.run([str(at / "parts")], input=text, capture_output=True, text=True,
                             check=True).stdout.splitlines()
        assert len(out) == len(heads)
        return out
    return ask


def test_every_entry_a_run_writes_is_followed(answers):
    ctas = 296
    heads = [(r, f) for r in range(ctas) for f in (0, 1, 2, 73, ctas - 1 - r) if r + f < ctas]
    for (r, f), got in zip(heads, answers(heads)):
        # the run that begins the unit leaves its part in its second slot, the others
        # in their first
        assert got == f"{2 * r + 1} {2 * (r + f) if f else 2 * r + 1}", (r, f)


def test_entries_that_no_run_wrote_are_not_followed(answers):
    top, low = 2 ** 31 - 1, -2 ** 31
    bad = [(-1, 1), (0, -1), (296, 0), (295, 1), (0, 296), (top, top), (top, 1), (1, top), (low, low),
           (low, 1), (5, low), (-1, -1), (148, 148), (top, low), (low, top)]
    assert set(answers(bad)) == {"no"}


def test_any_bytes_lead_only_to_slots_of_the_workspace(answers):
    rng = random.Random(5)
    heads = [struct.unpack("<ii", rng.randbytes(8)) for _ in range(20000)]
    heads += [(rng.randint(-600, 600), rng.randint(-600, 600)) for _ in range(20000)]
    heads += [struct.unpack("<ii", struct.pack("<ff", rng.gauss(0, 1), rng.gauss(0, 1)))
              for _ in range(20000)]
    for (r, f), got in zip(heads, answers(heads)):
        assert "outside" not in got
        assert (got != "no") == (r >= 0 and f >= 0 and r + f < 296), (r, f)


def test_the_join_asks_before_it_follows():
    """The check stands between the entry's read and the first read of a part."""
    src = open(os.path.join(CSRC, "tree_attn.cu")).read()
    join = src[src.index("tree_attn_combine_kernel(const TreeArgs a) {"):]
    read, check, part = (join.index(x) for x in ("a.heads[unit]", "if (!parts_within(hd))",
                                                 "a.parts + "))
    assert read < check < part
