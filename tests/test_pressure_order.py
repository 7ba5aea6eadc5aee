"""Orders in the sources of shared-prefix attention and of cached keys' weights that a run on a GPU cannot be made to
break."""
import re

from test_kernel_order import bodies, source


def test_a_window_has_its_tensor_memory_before_the_next_kernel_may_start():
    """The next kernel's CTAs may take tensor memory before they wait for the grid before them: a CTA that took its own
    only then would wait for theirs, and they for it.  So a CTA takes it after it has waited and before it lets them start."""
    body = bodies(source("cache_evict.cu"))["cache_weights_window_kernel"]
    at = [body.index(x) for x in ("griddep_wait()", "tmem_alloc(", "__syncthreads();", "griddep_launch()")]
    assert at == sorted(at) and body.count("griddep_launch()") == 1 and body.count("tmem_alloc(") == 1


def test_a_prefix_leaves_no_room_beside_it():
    """attn_prefix lets the next kernel start before it takes its tensor memory: no CTA with tensor memory of its own fits
    beside one of its, which hold most of an SM's shared memory (and it waits for the grid before it first)."""
    text = source("attn_prefix.cu")
    body = bodies(text)["attn_prefix_kernel"]
    assert body.index("griddep_wait()") < body.index("tmem_alloc(")
    stages = {int(d): int(n) for d, n in [("128", re.search(r"kStages = D == 128 \? (\d+) : (\d+);", text)[1]),
                                          ("64", re.search(r"kStages = D == 128 \? (\d+) : (\d+);", text)[2])]}
    for D, n in stages.items():
        assert (2 + n) * 128 * D * 2 > 190 << 10       # of 228 KB; the others take 40 KB or more
