"""The walk of a tile of tokens over a batch's sequences, compiled for the host from the library's
header and run over many tables: right ones give every token and every empty sequence once, and no
table, however wrong, gives a span from which a kernel could leave its tensors."""
import os
import random
import subprocess

import pytest

from gated_delta_rule_gdn_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("walk") / "span_walk")
    subprocess.run([build._hipcc(), *build.FLAGS, "-I", build.CSRC, os.path.join(HERE, "span_walk.hip"), "-o", exe],
                   check=True, capture_output=True)

    def run(tables):
        """tables of (offsets or sequence length, total, tile, n) -> their spans, as tuples."""
        text = "".join(f"{-1 if isinstance(cu, list) else cu} {total} {tile} {n} "
                       + " ".join(map(str, cu if isinstance(cu, list) else [])) + "\n"
                       for cu, total, tile, n in tables)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        parts = out.split(".\n")[:-1]
        assert len(parts) == len(tables)
        return [[tuple(map(int, line.split())) for line in p.splitlines()] for p in parts]

    return run


def draw(rng, wrong):
    total, tile = rng.choice((0, 1, 7, 64, 200, 1000)), rng.choice((1, 5, 16, 64, 300))
    n = rng.choice((1, 2, 4, 9, 63, 64, 65, 130, 200))
    if wrong:
        return [rng.randint(-total - 2, 2 * total + 2) for _ in range(n + 1)], total, tile, n
    used = rng.choice((total, total, rng.randint(0, total)))
    cu = [0] + sorted(rng.choice((0, used, rng.randint(0, used), rng.randint(0, used)))
                      for _ in range(n - 1)) + [used]
    return cu, total, tile, n


def held(spans, total, tile, n):
    """What keeps every access in bounds. The W - 1 inputs before a span's first token are rows
    [lo - first, W - 2] of its sequence's state or tokens from `first` on, so first <= lo; tokens
    are read up to `end`; states are those of sequence i."""
    for k, i, first, end, lo, hi, starts, ends in spans:
        t0, t1 = k * tile, min(k * tile + tile, total)
        assert 0 <= i < n, (i, n)
        assert 0 <= first <= lo <= hi <= total and t0 <= lo and hi <= t1, (first, lo, hi, t0, t1)
        assert first <= end <= total and (hi <= end or hi == lo), (first, end, lo, hi)


def test_right_tables(walk):
    rng = random.Random(1)
    tables = [draw(rng, False) for _ in range(400)]
    tables += [(T, B * T, tile, B) for B in (1, 3, 70) for T in (0, 1, 9, 64) for tile in (1, 16, 64, 500)]
    for (cu, total, tile, n), spans in zip(tables, walk(tables)):
        at = cu if isinstance(cu, list) else [i * cu for i in range(n + 1)]
        held(spans, total, tile, n)
        tokens, starts, ends = [], [], []
        for k, i, first, end, lo, hi, s, e in spans:
            assert (first, end) == (at[i], at[i + 1])
            tokens += range(lo, hi)
            starts += [i] * s
            ends += [i] * e
        assert tokens == list(range(at[0], at[n]))          # each once, in order
        assert starts == list(range(n)) and ends == list(range(n))


def test_wrong_tables_stay_inside_the_tensors(walk):
    """Offsets that decrease, are negative or lie behind the batch."""
    rng = random.Random(2)
    tables = [([0, 150, 120, 20, 200], 200, 64, 4)] + [draw(rng, True) for _ in range(2000)]
    for (cu, total, tile, n), spans in zip(tables, walk(tables)):
        held(spans, total, tile, n)
