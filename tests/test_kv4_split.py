"""What the decodes from the paged caches do before and around their tiles, on the CPU."""
import os
import random
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_tiled_attention_22_gb300", "csrc")


def test_dependents_may_start_when_tensor_memory_is_there():
    """A kernel that takes the tensor memory of an SM before a block of the kernel it waits for has its own would wait
    for ever: the thread that lets the next kernel start belongs to the warp that allocates, and comes behind it."""
    with open(os.path.join(CSRC, "attn_kv4.cu")) as f:
        kernel = f.read().split("attn_kv4_split_kernel(")[1].split("launch_split_t(")[0]
    kernel = re.sub(r"//.*", "", kernel)
    alloc, trigger = (re.search(r"if \((.*?)\)\s*(\{[^}]*)?%s\(" % f, kernel)
                      for f in ("tmem_alloc", "griddep_launch_dependents"))
    assert kernel.count("griddep_launch_dependents(") == kernel.count("tmem_alloc(") == 1
    assert alloc.group(1) == "warp == kWarpMma" and trigger.group(1) == "threadIdx.x == kWarpMma * 32"
    assert alloc.start() < trigger.start()


def host_program(tmp_path_factory, name):
    exe = str(tmp_path_factory.mktemp(name) / "check")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", os.path.join(ROOT, "tests", "c_client", name + ".cpp"),
                    "-I" + CSRC, "-o", exe], check=True)

    def run(calls):
        text = "\n".join(" ".join(str(int(x)) for x in c) for c in calls)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr
        got = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
        assert len(got) == len(calls)
        return got
    return run


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    return host_program(tmp_path_factory, "kv4_rules_check")


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    return host_program(tmp_path_factory, "kv_split_check")


def test_clusters_of_eight_where_none_of_sixteen_fits(rules):
    """Every call that would take clusters of 16 has a form without them: clusters of 8, or dealt tiles."""
    rng = random.Random(3)
    calls, sixteen = [], 0
    for _ in range(20000):
        calls.append((int(2 ** rng.uniform(0, 8)), rng.random() < 0.5, rng.choice([152, 148, 16, 8]), int(2 ** rng.uniform(0, 4)),
                      rng.choice([1, 2, 3, 4, 5, 8]), int(2 ** rng.uniform(0, 12)), 16))
    with16, with8 = rules(calls), rules([(*c[:-1], 8) for c in calls])
    for (R, bf16, sms, B, H, tiles, _), a, b in zip(calls, with16, with8):
        rp, segs = a[0], B * H * -(-R // a[0])
        resident = sms * (1 if rp == 16 else 3 if rp == 4 and bf16 else 2)
        assert a[1] in (0, 2, 4, 8, 16) and b[1] in (0, 2, 4, 8)
        for _, cluster, grid, _ in (a, b):
            assert grid == segs * cluster if cluster else 1 <= grid <= min(resident, segs * tiles)
            assert grid <= resident
        if a[1] == 16:
            sixteen += 1
            assert b[1] in (0, 8)
        else:
            assert a == b
    assert sixteen > 100


SMS = 152
# (grid, CTAs with a full share): each number of CTAs to an SM, 8 to 7 shares where there are three
GRIDS = [(SMS, 0), (2 * SMS, 0), (3 * SMS, 0), (3 * SMS, 2 * SMS)]


@pytest.mark.parametrize("lens,Hr", [
    ([1], 1), ([0], 3), ([0, 0, 5, 0], 2), ([1000], 8), ([17001, 9000, 2300, 130, 1, 0, 4000], 8), ([8192] * 64, 8),
    ([50001, 131072, 70000, 99999], 8), ([60000] * 4, 8), ([200, 0, 100000], 1), ([300] * 200, 3), ([128] * 1000, 5),
    ([2 ** 31 - 1, -5, 2 ** 31 - 1], 2), ([2 ** 31 - 1], 16), ([2 ** 31 - 256] * 40, 64)])
def test_every_tile_is_dealt_once_and_every_part_is_found(walk, lens, Hr):
    calls = [(ts, sc, Hr, grid, full, len(lens), *lens) for ts in (7, 8) for sc in (1, 2) for grid, full in GRIDS]
    out = walk(calls)
    if sum(lens) > 40 * 128 * 3 * SMS:     # (many tiles a CTA: segments are cut)
        assert all(cut for _, _, cut, _ in out)


def test_drawn_deals(walk):
    rng = random.Random(11)
    calls = []
    for _ in range(1500):
        top = int(2 ** rng.uniform(0, 31 if rng.random() < 0.2 else 16))
        lens = [rng.choice([0, 1, rng.randint(0, top), int(2 ** rng.uniform(0, 16))]) for _ in range(int(2 ** rng.uniform(0, 9)))]
        grid, full = rng.choice(GRIDS + [(rng.randint(1, 640), 0)])
        calls.append((rng.choice([7, 8]), rng.choice([1, 2]), int(2 ** rng.uniform(0, 6)), grid, full, len(lens), *lens))
    out = walk(calls)
    weighted = [o for o, c in zip(out, calls) if c[4] and o[0] >= 4 * c[3]]
    assert len(weighted) > 100 and {o[3] for o in weighted} == {0, 1}


def test_clusters_of_sixteen(rules):
    """By the block table's width: 17 tiles and more of one to nine segments."""
    calls = [(4, 1, SMS, 1, 1, 16, 16), (4, 1, SMS, 1, 1, 17, 16), (7, 0, SMS, 2, 1, 18, 16), (16, 1, SMS, 2, 1, 21, 16),
             (4, 1, SMS, 1, 8, 128, 16), (4, 1, SMS, 1, 8, 129, 16), (4, 1, SMS, 10, 1, 17, 16)]
    assert [o[1] for o in rules(calls)] == [8, 16, 16, 16, 16, 0, 8]
