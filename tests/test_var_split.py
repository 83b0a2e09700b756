"""How the packed backward cuts a batch into work items (csrc/var_split.h), on the CPU:
every chunk of every key tile is one item, in both numberings; partial tiles fit their
workspace; and no launch has fewer blocks than SMs while it has that many items."""
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SMS = 152


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("var_split") / "check")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", os.path.join(ROOT, "tests", "c_client", "var_split_check.cpp"),
                    "-I" + os.path.join(ROOT, "exact_tiled_attention_22_gb300", "csrc"), "-o", exe], check=True)

    def run(batches):
        text = "\n".join(" ".join(map(str, [int(c), hq, h, SMS, len(lq), *lq, *lk])) for c, hq, h, lq, lk in batches)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr
        out = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
        assert len(out) == len(batches)
        return out
    return run


@pytest.mark.parametrize("causal,hq,h,lq,lk,items", [
    (True, 1, 1, [8192], [8192], 160),        # one head: 64 key tiles, most of them cut
    (False, 4, 4, [65536], [128], 128),       # many queries on one key tile of each head
    (False, 8, 8, [16384], [128], 64),
])
def test_a_block_for_every_item(walk, causal, hq, h, lq, lk, items):
    (n, _, ctas), = walk([(causal, hq, h, lq, lk)])
    assert n == items and ctas >= min(SMS, n)


def test_groups_up_to_the_largest(walk):
    """Every group size at which the least chunk changes, and the largest ones."""
    batches = []
    for g in (1, 2, 3, 5, 8, 9, 15, 16, 17, 64, 65, 127, 128, 256, 1000, 1024):
        for causal in (False, True):
            batches += [(causal, g, 1, [n], [m]) for n, m in ((1, 1), (130, 129), (1000, 1000), (700, 3000), (3000, 500))]
            batches.append((causal, 2 * g, 2, [100, 0, 2000, 65], [100, 40, 2500, 0]))
    walk(batches)


def test_drawn_batches(walk):
    rng = random.Random(5)
    batches = []
    for _ in range(300):
        top = int(2 ** rng.uniform(0, 14))
        lq = [rng.randint(0, top) for _ in range(int(2 ** rng.uniform(0, 6)))]
        lk = [rng.choice([n, rng.randint(0, top), n + rng.randint(0, top)]) for n in lq]
        h = rng.choice([1, 1, 2, 3, 8])
        batches.append((rng.random() < 0.6, h * rng.choice([1, 1, 2, 3, 4, 7, 16, 40]), h, lq, lk))
    walk(batches)
