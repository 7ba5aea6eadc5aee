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
