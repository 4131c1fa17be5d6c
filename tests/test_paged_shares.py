"""How the paged decode cuts its work (paged_shares.cuh, compiled for the host): no pair into more parts than the limit,
no share without work, and no fewer shares than the limit asks for."""
import os
import random
import re
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mixed_head_kv_b200", "csrc")


def test_no_pair_is_cut_into_more_parts_than_the_limit():
    limit = int(re.search(r"kPartsPerPair = (\d+)", open(os.path.join(CSRC, "paged_shares.cuh")).read()).group(1))
    rng = random.Random(5)
    cases = [(296, [2049] + [6] * 7), (296, [2049]), (296, [7813] + [6] * 7), (296, [2] * 200 + [1 << 21] + [2] * 600),
             (296, [(1 << 21) + 1] * 4096), (296, [1]), (296, [0, 0]), (296, [1] * 295), (296, [limit]), (296, [limit + 1]), (2, [900, 1])]
    for _ in range(400):
        n = rng.choice([1, 2, 7, 40, 700])
        units = [int(2 ** rng.uniform(0, rng.choice([1, 4, 8, 14]))) for _ in range(n)]
        if rng.random() < 0.5:
            units[rng.randrange(n)] = int(2 ** rng.uniform(8, 21))
        cases.append((rng.choice([1, 132, 296, 320]), units))
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "paged_shares_check")
        subprocess.check_call(["g++", "-O1", "-std=c++17", "-I", CSRC, os.path.join(HERE, "paged_shares_check.cpp"), "-o", exe])
        text = "".join(f"{c} {len(u)} {' '.join(map(str, u))}\n" for c, u in cases)
        out = [tuple(map(int, x.split())) for x in subprocess.check_output([exe], input=text, text=True).splitlines()]
    assert len(out) == len(cases)
    for (ctas, units), (shares, most) in zip(cases, out):
        total, longest = sum(units), max(units)
        assert min(1, total) <= shares <= min(ctas, total)
        assert most <= limit + 1, (ctas, shares, most, longest)
        least = max(1, -(-longest // limit))  # units that every share has to hold
        assert shares == ctas or (shares + 1) * least > total
