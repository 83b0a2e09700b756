"""What the decode from the 4-bit cache does before and around its tiles, on the CPU."""
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


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("kv4_rules") / "check")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", os.path.join(ROOT, "tests", "c_client", "kv4_rules_check.cpp"),
                    "-I" + CSRC, "-o", exe], check=True)

    def run(calls):
        text = "\n".join(" ".join(str(int(x)) for x in c) for c in calls)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60, check=True).stdout
        got = [tuple(map(int, line.split())) for line in out.splitlines()]
        assert len(got) == len(calls)
        return got
    return run


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
