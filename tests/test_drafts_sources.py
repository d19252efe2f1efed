"""Rules that the drafted-token kernels' sources keep because no run can show a breach of them.
CPU only."""
import os
import re

from paged_kv_cache_split_gb300 import build as pkv_build

FILES = ["rotated_write.cu", "accept.cu", "tree_attn.cu", "tree_attn.cuh", "drafts.cuh"]


def sources():
    return {f: re.sub(r"//[^\n]*|/\*.*?\*/", "", open(os.path.join(pkv_build.CSRC, f)).read(), flags=re.S) for f in FILES}


def test_no_non_coherent_loads():
    """The kernels are resident while the stream's previous kernel may still write what they read
    after their wait: loads of data that has to stay constant for a kernel's lifetime are not
    allowed there."""
    for name, text in sources().items():
        assert not re.search(r"__ldg|\.nc\b|__restrict", text), name


def test_every_kernel_waits_before_it_reads():
    """Launched with programmatic dependence, each kernel waits for the previous one before its
    first global access, and lets the next one start only after that."""
    found = 0
    for name, text in sources().items():
        for m in re.finditer(r"__global__.*?\{", text, flags=re.S):
            body = text[m.end():]
            body = body[:body.index("\n}")]
            wait, go = body.index("griddepcontrol.wait"), body.index("griddepcontrol.launch_dependents")
            assert wait < go, name
            assert not re.search(r"\b(P\.a|P|a)\.\w+\s*\[|\bstart_walk\b|\blength\(", body[:wait]), name
            found += 1
    assert found == 5


def test_whole_warps_meet_the_tensor_memory_loads():
    """Loads from and stores to tensor memory want a converged warp: a warp barrier, or a wait that
    ends in one, lies between them and any branch by lane before them."""
    text = sources()["tree_attn.cuh"]
    body = text[text.index("if (warp < 8) {"):]
    body = body[:body.index("if (warp < L::kFeeder0 / 32)")]
    for m in re.finditer(r"tc_(ld|st)_rows", body):
        before = body[:m.start()]
        synced = max(before.rfind(x) for x in ("__syncwarp()", "wait_or_die(", "tc_wait_ld()", "tc_wait_st()"))
        lanes = max(before.rfind(x) for x in ("if (mine", "if (lane", "threadIdx.x == 0"))
        assert synced > lanes, body[m.start() - 200:m.end()]


def test_the_powers_of_two_segments_queries_lie_apart():
    """With more than 128 rows a warpgroup's part of a segment of few tiles hangs on nothing that the
    other does: it may load the next segment's queries before the other has read the powers of this
    one.  Two copies in turns are enough: a barrier lies in every segment."""
    text = sources()["tree_attn.cuh"]
    assert re.search(r"\w+ q_pow\[2\]\[2 \* kRows\];", text)
    uses = re.findall(r"sm\.q_pow\b[^;,]*", text)
    assert uses and all(u.startswith("sm.q_pow[n_seg & 1]") for u in uses), uses
    body = text[text.index("load_queries<D, KB>(P"):]
    body = body[:body.index("q_pow[rr]")]
    assert body.index("named_barrier_sync(1, kSoftmaxThreads)") < body.index("++n_seg")


def block(text, head):
    """The braces that follow the first `head` in text, and what lies between them."""
    at = text.index("{", text.index(head))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError(head)


def test_a_rescaled_output_is_stored_before_it_is_loaded_again():
    """Both halves of a tile may rescale O.  Stores to tensor memory are not ordered before later
    loads of the same columns without a wait for them, so the rescaling itself ends in one."""
    body = block(sources()["tree_attn.cuh"], "if (job > before)")
    assert "tc_ld_rows<32>(tm_o(t)" in body
    assert "tc_wait_st()" in body[body.index("tc_st_rows<32>(tm_o(t)"):]
