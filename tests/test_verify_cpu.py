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


def test_warps_meet_before_a_barrier_of_the_cluster():
    # The barrier's instructions are for whole warps; behind code of some lanes alone the warp is brought together.
    src = kernel_source()
    for of_some in (src.index("if (tid == 0) {"), src.index("if (tid < CS) {")):
        barrier = min(x for x in (src.find("cluster_arrive()", of_some), src.find("cluster_sync_all()", of_some)) if x > 0)
        assert src.rindex("__sync", 0, barrier) > of_some


def test_no_sequences_need_no_addresses():
    # Nothing is launched for them, and empty tensors have no address.
    L, p = tp.lib(), 1 << 20

    def verify(M, n, x, accepted):
        return L.tp_vocab_verify_drafts(x, None, M, 64, 4, x, p, n, None, x, None, accepted, x, None)

    assert verify(0, 0, None, None) == tp.TP_OK, tp.tp_last_error()
    assert verify(3, 0, p, None) == tp.TP_OK, tp.tp_last_error()
    assert verify(3, 0, None, None) == tp.TP_ERR_INVALID_ARG
    assert verify(0, 2, None, None) == tp.TP_ERR_INVALID_ARG
    assert verify(0, 0, p + 4, None) == tp.TP_ERR_INVALID_ARG


def test_the_self_test_refuses_places_that_are_not_there():
    p = 1 << 20
    for where in (-1, 0, 3):
        assert tp.lib().tp_selftest_verify_timeout(p, 4, 64, p, p, 2, p, p, p, where, None) == tp.TP_ERR_INVALID_ARG
    assert tp.lib().tp_selftest_verify_timeout(p, 4, 66, p, p, 2, p, p, p, 1, None) == tp.TP_ERR_INVALID_ARG


def test_nothing_is_armed_or_left_behind_once_a_wait_gave_up():
    # The producer looks at the word that every wait sets when it gives up, after the wait for a free stage and
    # before it arms the stage's barrier again; and the copies in flight are waited for by that word too, not by
    # what the producer itself met.
    src = kernel_source()
    produce = src[src.index("auto produce ="):]
    produce = produce[:produce.index("advance();")]
    assert produce.index("wait(empty0") < produce.index("abort_word") < produce.index("mbar_arrive_expect_tx")
    assert re.search(r"if \(abort_word && tid == VT\)\s*for [^;]*;[^;]*;[^)]*\) drain\(", src)
