"""CPU checks of draft verification: what its source and its entry point promise without a GPU."""
import os
import re

import megatron_tensor_transformer_colwise_gb300 as tp

CSRC = os.path.join(os.path.dirname(os.path.abspath(tp.__file__)), "csrc")


def kernel_source():
    """verify_kernel without its comments."""
    with open(os.path.join(CSRC, "tp_verify.cu"), encoding="utf-8") as f:
        src = re.sub(r"//[^\n]*", "", f.read())
    return src[src.index("verify_kernel("):src.index("int verify_launch")]


def test_the_cluster_has_started_before_a_store_into_another_block():
    # Shared memory of another block of the cluster may be touched once that block is known to run, which a
    # cluster barrier tells.  Every thread passes it: nothing returns before it.
    src = kernel_source()
    barrier = min(src.index(w) for w in ("cluster_wait()", "cluster_sync_all()") if w in src)
    assert barrier < src.index("store_cluster(")
    assert "return" not in src[:barrier]
