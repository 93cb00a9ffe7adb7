"""The host side of the 8-bit linear's launchers (csrc/i8_plan.h), compiled for the CPU with the undefined-behaviour
checks on: integer division by zero and overflow end the program."""
import os
import subprocess

import pytest

from i8_cases import GROUPS, HELD, SPLITS, TILES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_block_scaled_18_b200", "csrc")


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    """ask(lines) -> the answers, one a line."""
    exe = str(tmp_path_factory.mktemp("i8_plan") / "i8_plan_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fsanitize=integer-divide-by-zero,signed-integer-overflow",
                    "-fno-sanitize-recover=all", "-I" + CSRC, os.path.join(ROOT, "tests", "i8_plan_check.cpp"), "-o", exe],
                   check=True)

    def run(lines):
        r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        out = r.stdout.splitlines()
        assert len(out) == len(lines)
        return out

    return run


def test_every_tile_once(ask):
    """The walk of the CTA pairs over the tiles, each looking up its next place while it works on the present one, as the
    loads' issuer does: also where the last tile ends a group, and where the last group is short."""
    lines = [f"order {tok} {ch} {size} {grid}"
             for tok in (1, 2, 3, 5, 16, 17, 32, 65) for ch in (1, 2, 7, 43, 112)
             for size in (4096, 256 * 8192, 256 * 65536, 256 * 131056) for grid in (1, 2, 66, 74)]
    for line, answer in zip(lines, ask(lines)):
        assert answer.split()[1:] == ["ok"], (line, answer)


def test_token_groups(ask):
    """Groups of at most 32 MB, as even as they come, and one block at least."""
    assert [a.split()[0] for a in ask(["order 32 112 2097152 74", "order 5 10 16777216 74", "order 3 2 67108864 74"])] == ["16", "2", "1"]


def test_cases_reach_every_width(ask):
    """The GPU tests' shapes: every width that the estimate takes, from either side, and short last groups."""
    got = [[int(v) for v in a.split()] for a in ask([f"tiles {m} {n} {k} 148" for m, n, k, _, _ in TILES])]
    assert [(g[0], bool(g[1])) for g in got] == [(bn, swap) for *_, bn, swap in TILES]
    assert {bn for *_, bn, swap in TILES if not swap} == set(range(32, 257, 32))
    assert {bn for *_, bn, swap in TILES if swap} == set(range(64, 225, 32))
    got = [[int(v) for v in a.split()] for a in ask([f"tiles {m} {n} {k} 148" for m, n, k, _, _ in GROUPS])]
    assert [(g[2], g[3]) for g in got] == [(tok, group) for *_, tok, group in GROUPS]
    assert all(tok > group and tok % group for *_, tok, group in GROUPS)


def test_widths_taken(ask):
    """Over the whole range of sizes no other width is taken than those the cases have."""
    sizes = [(m, n, k) for m in range(257, 8200, 379) for n in range(64, 28700, 1237) for k in (64, 528, 1552, 4096, 8192, 27648)]
    taken = {tuple(a.split()[:2]) for a in ask([f"tiles {m} {n} {k} 148" for m, n, k in sizes])}
    assert taken <= {(str(bn), str(int(swap))) for *_, bn, swap in TILES}


def test_failed_query_is_asked_again(ask):
    """A query that fails gives a guess for that call alone; an answer is kept."""
    assert ask(["held 33 7", "held -1 33", "held -1 -1"]) == ["33 33 33 1", "5 33 33 2", "5 5 5 3"]
    assert ask(["held 0 0"]) == ["0 0 0 3"]              # none is an answer too


def test_split_runs_in_one_wave(ask):
    """K is split as far as the clusters of all tiles are held at once, with the numbers of clusters of 2 to 8 that 148
    SMs held at one CTA per SM and at two."""
    for at_once in HELD.values():
        lines = [f"split {t} 112 1 8 " + " ".join(map(str, at_once)) for t in range(1, 160)]
        for tiles, answer in enumerate(ask(lines), 1):
            ks, held = map(int, answer.split())
            assert ks == max([1] + [k for k in range(2, 9) if tiles <= at_once[k - 2]])
            assert ks == 1 or tiles <= held
    held = " " + " ".join(map(str, HELD[2]))
    # 46 to 48 tiles: 45 clusters of six are held, so five parts; few steps, and partial sums that do not fit, split less
    assert ask([f"split {t} 112 1 8{held}" for t in (45, 46, 48)] + [f"split 10 35 10 8{held}", f"split 10 112 1 4{held}"]) == [
        "6 45", "5 56", "5 56", "3 93", "4 71"]


def test_cases_reach_every_split(ask):
    """The GPU tests' shapes of 129 to 256 tokens take the split-K kernel, in the parts that they name; no other split is
    taken over the whole range."""
    held = " ".join(map(str, HELD[1]))
    assert ask([f"few {m} {n} {k} 148 {held}" for m, n, k, _ in SPLITS]) == [f"1 {ks}" for *_, ks in SPLITS]
    sizes = [(m, n, k) for m in range(129, 257, 9) for n in range(64, 28700, 613) for k in (64, 1040, 4096, 9008, 14336, 27648)]
    taken = {a for a in ask([f"few {m} {n} {k} 148 {held}" for m, n, k in sizes]) if a[0] == "1"}
    assert taken <= {f"1 {ks}" for *_, ks in SPLITS}
