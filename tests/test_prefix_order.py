"""Orders within attn_prefix's warps, in its source: what hangs on the lanes' timing shows in the text, seldom in an output."""
import re

from test_kernel_order import bodies, source


def test_a_partial_is_read_back_before_the_next_queries_overwrite_it():
    """A warp's lanes write their rows' outputs into the warp's rows of the query tile and read other lanes' from there; the
    next piece's queries go into the same rows.  Between the last of the reads and those writes the warp has to meet."""
    body = bodies(source("attn_prefix.cu"))["attn_prefix_kernel"]
    read = body.rindex("ld_shared_v4(buf")
    assert body.index("*reinterpret_cast<uint4*>(sQ + x * C::kTileBytes") < read      # the queries', earlier in the loop
    # behind the read-back loops (k over the parts, q over 32 features), still where all lanes pass
    tail = body[read:body.index("if (mine) a.ws_ml[wr]")]
    assert re.search(r"=\s*v;\s*\}\s*\}\s*__syncwarp\(\);\s*tc_fence_before\(\);", tail)


def test_a_buffer_of_a_partial_is_read_before_it_is_written_again():
    """Heads of 64 have one box to stage 32 features in: the warp meets before each further use of it; those of 128 have two
    and meet once between two uses of one."""
    body = bodies(source("attn_prefix.cu"))["attn_prefix_kernel"]
    stage = body[body.index("const uint32_t buf"):body.rindex("ld_shared_v4(buf")]
    at = [stage.index(x) for x in ("if (C::kBoxes == 1) __syncwarp();", "st_shared_v4(buf", "__syncwarp();\n")]
    assert at[0] < at[1] and stage.index("__syncwarp();", at[1]) > at[1]
