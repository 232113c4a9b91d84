"""Orders inside the kernels that no run can be made to break on purpose, read off the sources."""
import os
import re

import prefix_shared_kv_ra_gb300 as ra

CSRC = os.path.join(os.path.dirname(ra.__file__), "csrc")


def kernels():
    """The kernels' bodies by name, without comments."""
    found = {}
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh")):
            continue
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\(", text):
            start = i = text.index("{", m.end())
            depth = 0
            while i == start or depth > 0:
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                i += 1
            found[m.group(1)] = text[start:i]
    return found


def test_stores_into_other_ctas_come_behind_a_cluster_barrier():
    """A CTA of a cluster has to have started before another one accesses its shared memory."""
    users = {k: body for k, body in kernels().items() if re.search(r"\bst_cluster_\w+\(", body)}
    assert set(users) >= {"tree_verify_kernel", "tree_verify_greedy_kernel", "tree_commit_kernel"}
    for k, body in users.items():
        remote = re.search(r"\bst_cluster_\w+\(", body).start()
        before = body[:remote]
        assert before.count("cluster_arrive();") == 1, k
        # one wait on the way to the store, and one on every way out before it
        before = before.split("cluster_arrive();")[1]
        assert before.count("cluster_wait();") == before.count("return;") + 1, k


def test_stored_weights_are_complete_before_they_are_read_back():
    """Loads and stores of tensor memory are asynchronous: a raised reference scales weights that the same tile has stored."""
    body = kernels()["attn_tc_kernel"]
    loop = body.index("for (int k = 0; k < 2 * c; ++k)")
    stores = [m.start() for m in re.finditer(r"tmem_st\d+\(", body) if m.start() < loop]
    assert "tmem_ld8(" in body[loop:loop + 300]
    assert "tc_wait_st();" in body[stores[-1]:loop]


def test_planning_kernels_read_lengths_through_l2():
    """They read lengths before they wait for the kernel before them, which may have written them and still run."""
    found = kernels()
    for k in ("decode_plan_kernel", "extend_plan_kernel", "extend_mod_plan_kernel"):
        assert "__ldcg(" in found[k] and "__ldg(" not in found[k], k
    with open(os.path.join(CSRC, "decode_internal.h")) as f:
        text = f.read()
    start = text[text.index("int32_t mod_start("):]
    assert "__ldg(" not in start[:start.index("}")]
    # and those that write lengths let the next kernel launch behind a fence only
    for k in ("step_slots_kernel", "tree_commit_kernel", "tree_verify_kernel", "tree_verify_greedy_kernel"):
        assert "griddep_launch();" not in found[k] and "launch_behind_writes();" in found[k], k
