"""The order of what the softmax warpgroups exchange, on the host.

csrc/softmax_exchange.h is compiled with an Io that writes down what each of the
eight warps does (one thread a warp: the others do the same at their own places),
through items of given numbers of tiles, in the order of softmax() in latent_mla.cu.
The warps are then run in many orders with the barriers' rules (a barrier opens when
as many threads as it names have arrived or wait), and each access is compared with
the earlier ones of its place: a write has to be ordered behind every earlier read
and write, a read behind the last write, by the program or by barriers.  A missing
order shows in every schedule, not only in the unlucky one.
"""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include "softmax_exchange.h"

struct Trace {
  void store(uint32_t at, uint32_t) const { printf("w %u 0\n", at); }
  uint32_t load(uint32_t at) const { printf("r %u 0\n", at); return 0; }
  void sync(int id, int n) const { printf("s %d %d\n", id, n); }
  void arrive(int id, int n) const { printf("a %d %d\n", id, n); }
};

int main(int argc, char** argv) {
  for (uint32_t group = 0; group < 2; ++group)
    for (int warp = 0; warp < 4; ++warp) {
      misa::SoftmaxExchange<Trace> x = {{}, group, warp * 32};
      uint32_t n = 0, items = 0;
      printf("warp 0 0\n");
      for (int i = 1; i < argc; ++i) {
        const uint32_t tiles = (uint32_t)atoi(argv[i]);
        if (tiles == 0) continue;
        const uint32_t first = n, end = n + tiles;
        for (n += (n ^ group) & 1; n < end; n += 2) {
          x.other_half(0);
          x.reference_before(n, first, 0);
          x.set_reference(0);
        }
        n = end;
        const uint32_t turn = items++ & 1;
        if (((end - 1) & 1) != group) {
          x.hand_over(turn, 0);
          continue;
        }
        x.other_half_sum(turn, 0);
        if (tiles > 1) {
          x.handed_over(turn, 0);
          x.handed_over(turn, 1);
        }
      }
    }
  return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("exchange")
    (d / "trace.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "sparse_attention_token_misa_b200", "csrc"), str(d / "trace.cpp"), "-o",
                    str(d / "trace")], check=True)
    return str(d / "trace")


def _traces(program, items):
    warps = []
    for line in subprocess.run([program, *map(str, items)], capture_output=True, text=True, check=True).stdout.split("\n"):
        if line.startswith("warp"):
            warps.append([])
        elif line:
            op, x, n = line.split()
            warps[-1].append((op, int(x), int(n)))
    assert len(warps) == 8
    return warps


def unordered(warps, rng):
    """Runs the warps in an order that rng draws; the accesses that nothing orders."""
    W = len(warps)
    at = [0] * W
    clock = [[int(i == j) for j in range(W)] for i in range(W)]
    bars, asleep, found = {}, [None] * W, set()
    writes, reads = {}, {}          # place -> (warp, its time), place -> {warp: its time}

    def behind(w, other):           # does warp w know that `other` = (warp, time) has happened
        return clock[w][other[0]] >= other[1]

    def count(w, bar, n, waits):
        b = bars.setdefault(bar, {"threads": 0, "sleepers": [], "known": [0] * W, "n": n})
        assert b["n"] == n, f"barrier {bar} used with {b['n']} and {n} threads"
        b["threads"] += 32
        b["known"] = [max(x, y) for x, y in zip(b["known"], clock[w])]
        clock[w][w] += 1
        if waits:
            b["sleepers"].append(w)
            asleep[w] = bar
        if b["threads"] == n:
            for u in b["sleepers"]:
                clock[u] = [max(x, y) for x, y in zip(clock[u], b["known"])]
                asleep[u] = None
            del bars[bar]

    while True:
        ready = [w for w in range(W) if asleep[w] is None and at[w] < len(warps[w])]
        if not ready:
            break
        w = rng.choice(ready)
        for _ in range(rng.choice((1, 1, 4, 1000))):        # some warps run far ahead
            if asleep[w] is not None or at[w] == len(warps[w]):
                break
            op, x, n = warps[w][at[w]]
            at[w] += 1
            if op in "sa":
                count(w, x, n, op == "s")
                continue
            if x in writes and not behind(w, writes[x]):
                found.add((x, "write", op))
            if op == "r":
                reads.setdefault(x, {})[w] = clock[w][w]
            else:
                found |= {(x, "read", op) for r in reads.get(x, {}).items() if not behind(w, r)}
                writes[x], reads[x] = (w, clock[w][w]), {}
    assert asleep == [None] * W and all(a == len(t) for a, t in zip(at, warps)), "warps wait for ever"
    return found


def test_the_check_finds_a_missing_barrier():
    """Two warps: a place is read behind a barrier and written again without one."""
    sync = ("s", 1, 64)
    reader = [sync, ("r", 0, 0)]
    writer = [("w", 0, 0), sync, ("w", 0, 0)]
    assert unordered([writer, reader], random.Random(0)) and unordered([writer, reader], random.Random(1))
    assert not unordered([writer[:2] + [sync] + writer[2:], reader + [sync]], random.Random(0))
    assert unordered([[("w", 0, 0)], [("r", 0, 0)]], random.Random(0))
    with pytest.raises(AssertionError, match="wait for ever"):
        unordered([[sync], []], random.Random(0))


@pytest.mark.parametrize("items", [[1], [2], [3], [8], [1] * 7, [2] * 5, [3] * 5, [1, 2, 3, 4, 5], [2, 1, 2, 1, 1], [0, 1, 0, 4],
                                   [2, 4, 2, 6, 1, 1, 2]])
def test_accesses_are_ordered(program, items):
    warps = _traces(program, items)
    for seed in range(20):
        assert not unordered(warps, random.Random(seed))


def test_accesses_are_ordered_in_drawn_lists(program):
    rng = random.Random(7)
    for _ in range(40):
        items = [rng.choice((0, 1, 1, 2, 2, 3, 4, 7)) for _ in range(rng.randint(1, 9))]
        warps = _traces(program, items)
        for _ in range(4):
            assert not unordered(warps, rng), items
