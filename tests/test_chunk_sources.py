"""What the chunk kernels' sources keep to where a run could only show a fault by a hang."""
from __future__ import annotations

import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_tensor_memory_is_taken_after_the_previous_kernel_has_ended():
    """A block that holds its TMEM while it waits for the previous kernel in the stream could
    wait for a kernel whose own blocks wait for that TMEM."""
    with open(os.path.join(ROOT, "collective_kv_cache_gb300", "csrc", "k_chunk_tc.cu")) as f:
        text = f.read()
    body = text[text.index("chunk_tc_kernel(const"):]
    body = body[body.index("return;"):]                  # past the empty parts' way out
    wait, alloc = body.index("pdl_wait()"), body.index("tcgen05.alloc")
    assert wait < alloc < body.index("pdl_trigger()")
