"""Rules of the CUDA sources that a run cannot show: what they guard against
would be a race or a fault on the GPU, so they are checked in the text."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_weight_matvec_hq_gb300", "csrc")


def source(name):
    """A source file without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def device_functions(name):
    """(name, body) of each kernel and device function with a body of its own."""
    text = re.sub(r"__launch_bounds__\((?:[^()]|\((?:[^()]|\([^()]*\))*\))*\)", "", source(name))
    for m in re.finditer(r"^(?:template <[^\n]*>\s*)?(?:static )?__(?:global|device)__[^;{]*?(\w+)\s*\([^;{]*\)[^;{]*\{", text, flags=re.M):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield m.group(1), text[m.end():i]


REMOTE = r"\b(?:st_shared_cluster_\w+|ld_shared_cluster_\w+|mbar_arrive_remote)\s*\("


def test_peers_have_started_before_their_shared_memory_is_accessed():
    """Distributed shared memory may be accessed only once every block of the
    cluster runs: a cluster barrier comes before the first such access."""
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        for name, body in device_functions(os.path.basename(path)):
            first = re.search(REMOTE, body)
            if first:
                found.append(name)
                assert re.search(r"\bcluster_(?:sync|wait)\s*\(\)", body[:first.start()]), name
    assert {"softmax_kernel", "verify_kernel", "adapter_down", "matmul_tc_kernel", "plan_slots", "matvec_tma_kernel"} <= set(found)


def test_no_load_writes_to_more_than_one_block():
    """Cluster multicast is for a GPU's own memory; a caller's x or W may be mapped from elsewhere."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        assert "multicast" not in source(os.path.basename(path)), path


def test_weights_are_copied_early_only_behind_a_kernel_that_has_waited():
    """The many-token product may copy weights before its own wait, so the
    kernel in front of it lets it start only after that kernel's wait: what
    wrote the weights, one kernel further back, is then done."""
    bodies = dict(device_functions("hq_matmul.cu"))
    for name in ("prepare_kernel", "prepare_adapters_kernel"):
        assert bodies[name].index("griddep_wait()") < bodies[name].index("griddep_launch_dependents()"), name
    first = bodies["matmul_tc_kernel"].index("griddep_wait()")
    assert bodies["matmul_tc_kernel"][:first].endswith("if (!z.early || warp != kWarpW) ")
    assert "z.early = !a.moe && prep_grid > 0;" in source("hq_matmul.cu")


def test_tensor_memory_loads_are_in_no_branch_of_their_own():
    """A load from tensor memory is under way until it is waited for.  Under a
    condition its registers could be copied where the branches join, before
    the wait."""
    text = source("hq_matmul.cu")
    assert len(re.findall(r"\btmem_ld8\(", text)) > 3
    assert not re.findall(r"\b(?:if|else)\b[^;{}]*\btmem_ld8\(", text)
