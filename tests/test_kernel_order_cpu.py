"""Orders inside kernels that no run can show to be missing, read from their sources: a violation faults or hangs only
when CTAs happen to start in an unlucky order, so it is not to be found out on a GPU."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "offline_rl_step_gb300", "csrc")


def kernel_body(file, name):
    """The kernel's text from its opening brace to the closing one, without comments."""
    text = open(os.path.join(CSRC, file)).read()
    text = re.sub(r"//[^\n]*", "", text)
    at = re.search(r"__global__[^;{]*?\b" + name + r"\s*\(", text, re.S).end()
    at = text.index("{", at)
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError(f"{name}: no closing brace")


def test_cluster_runs_before_its_shared_memory_is_written_from_outside():
    body = kernel_body("norm.cu", "norm_cluster_kernel")
    first = body.index("st.shared::cluster")
    before = body[:first]
    assert "barrier.cluster.arrive" in before and "barrier.cluster.wait" in before
    assert before.index("barrier.cluster.arrive") < before.index("barrier.cluster.wait")
    # and once more after it, before the parts are read
    assert "barrier.cluster.arrive" in body[first:] and "barrier.cluster.wait" in body[first:]


def test_tmem_is_not_taken_ahead_of_a_kernel_that_still_needs_it():
    """A kernel that takes TMEM before it waits for its predecessor may share an SM with CTAs of the predecessor: those
    have to have theirs before they let it start, or each waits for the other."""
    for file, name in (("delta_chain_tc.cu", "delta_reverse_tc_kernel"), ("delta_grad_tc.cu", "delta_grad_tc_kernel"),
                       ("delta_prep.cu", "delta_prep_kernel")):
        body = kernel_body(file, name)
        assert body.index("pdl_wait()") < body.index("tmem_alloc("), name
    forward, prep = kernel_body("delta_chain_tc.cu", "delta_forward_tc_kernel"), kernel_body("delta_prep.cu", "delta_prep_kernel")
    if forward.index("tmem_alloc(") < forward.index("pdl_wait()"):
        assert prep.count("pdl_trigger()") == 1
        assert prep.index("tmem_alloc(") < prep.index("pdl_trigger()")
        # the same warp does both, one after the other
        assert re.search(r"if \(warp == 3\) \{\s*umma::tmem_alloc\([^;]*;\s*pdl_trigger\(\);\s*\}", prep)


def function_body(file, name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, file)).read())
    at = re.search(r"__device__ __forceinline__ \w+ " + name + r"\s*\(", text).end()
    return text[text.index("{", at):text.index("\n}", at)]


def test_lanes_give_up_together():
    """`dead` may be set by another warp between two lanes' reads of it: a lane that leaves on its own leaves the rest of
    its warp in a vote over all lanes."""
    for name in ("copy_chunk", "stage_ready"):
        body = function_body("delta_chain.cu", name)
        vote = body.index("__any_sync(0xffffffffu")
        assert not re.search(r"if \([^;{]*\bdead\b[^;{]*\)\s*\{?\s*return", body[:vote]), name


def test_nothing_is_in_flight_when_a_chain_that_gave_up_ends():
    """After a wait that ran out of time, copies into shared memory and products into TMEM are waited for before the CTA
    gives either back."""
    end = function_body("delta_chain.cu", "ring_end")
    assert "mbar_wait(&r.full" in end and "cp.async.wait_all" in end
    for name in ("delta_forward_kernel", "delta_reverse_kernel"):
        assert kernel_body("delta_chain.cu", name).rstrip("}\n ").endswith("ring_end(a, ring, stages);")
    end = function_body("delta_chain_tc.cu", "finish")
    assert end.index("umma::commit(") < end.index("mbar_wait(&b.full") < end.index("tmem_dealloc(")
    for name in ("delta_forward_tc_kernel", "delta_reverse_tc_kernel"):
        body = kernel_body("delta_chain_tc.cu", name)
        assert "tmem_dealloc(" not in body and body.rstrip("}\n ").endswith("finish(a, b, tmem);")
    prep = kernel_body("delta_prep.cu", "delta_prep_kernel")
    assert re.search(r"mbar_wait\([^;]*;\s*umma::tmem_dealloc\(", prep)
