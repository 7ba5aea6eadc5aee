"""Orders in the kernels' sources that a run on a GPU cannot be made to break: what hangs on timing alone shows in the
text, seldom in an output."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "causal_gqa_attention_fwd_gb300", "csrc")


def source(name):
    """The file's text without comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_each_warp_of_the_4_bit_decode_clears_its_own_piece_records():
    """A warp records its pieces as soon as it has them, in the cluster path before any barrier of the block: an entry that
    another warp clears may be lost.  So each entry is written by one thread alone, lane 0 of the warp whose it is."""
    text = source("attn_decode_q4.cu")
    indexes = re.findall(r"\brec_kind\[([^\]]+)\] [|&]?= ", text)
    assert sorted(indexes) == ["2 * warp", "2 * warp + 1", "slot"]
    assert re.search(r"const int slot = 2 \* warp \+ \(ta == 0\);", text)
    assert re.search(r"if \(lane == 0\) rec_kind\[2 \* warp\] = rec_kind\[2 \* warp \+ 1\] = 0;", text)
    assert re.search(r"if \(lane == 0\) \{\s*rec_unit\[slot\] = cu;\s*rec_kind\[slot\] = ", text)


def bodies(text):
    """{kernel: its body} of a file's __global__ functions."""
    out = {}
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\([^()]*\)\s*)?(\w+)\s*\((?=[^;{]*\)\s*\{)", text):
        i = start = text.index("{", m.end())
        depth = 0
        while True:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
            if depth == 0:
                break
        out[m.group(1)] = text[start:i]
    return out


def test_every_programmatic_dependent_waits_for_the_grid_before_it():
    """A kernel that is launched while the one before drains has to wait for it at some point: a kernel behind both waits
    for the last of them alone, and takes what the other has written, and the memory it used, for finished."""
    launched = set()
    kernels = {}
    for name in sorted(os.listdir(CSRC)):
        if name.endswith(".cu"):
            text = source(name)
            launched |= set(re.findall(r"launch_programmatic\(\s*(\w+)", text))
            launched |= set(re.findall(r"launch_programmatic_clusters\(\s*(\w+)", text))
            launched |= set(re.findall(r"cudaLaunchKernelEx\(&cfg,\s*(\w+)", text))
            kernels.update(bodies(text))
    assert len(launched) >= 12 and launched <= set(kernels), launched - set(kernels)
    for k in sorted(launched):
        assert re.search(r"griddep_wait\(\)|griddepcontrol\.wait", kernels[k]), f"{k} never waits for the grid before it"


def test_the_dq_kernel_ends_after_the_dkdv_kernel():
    """It runs beside the dK/dV grid; on each way out it waits for that grid's end."""
    body = bodies(source("attn_bwd_split.cu"))["bwd_dq_kernel"]
    assert body.rstrip("} \n").endswith("griddep_wait();")
    for m in re.finditer(r"\breturn;", body):
        assert body[:m.start()].rstrip().endswith("griddep_wait();")
