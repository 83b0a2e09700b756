"""What the decode from the 4-bit cache does before and around its tiles, on the CPU."""
import os
import re

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
