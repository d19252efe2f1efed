"""Rules that the latent kernels' sources keep because no run can show a breach of them.
CPU only."""
import glob
import os
import re

from paged_kv_cache_split_gb300 import build as pkv_build


def sources():
    paths = glob.glob(os.path.join(pkv_build.CSRC, "latent*.cu*")) + [os.path.join(pkv_build.CSRC, "tcgen05.cuh")]
    assert len(paths) == 5
    return {os.path.basename(p): re.sub(r"//[^\n]*|/\*.*?\*/", "", open(p).read(), flags=re.S) for p in paths}


def test_no_non_coherent_loads():
    """The kernels are resident while the stream's previous kernel may still write what they
    read after their wait (context lengths, value exponents): loads of data that has to
    stay constant for a kernel's lifetime are not allowed there."""
    for name, text in sources().items():
        assert not re.search(r"__ldg|\.nc\b|__restrict", text), name


def test_every_kernel_waits_before_it_reads():
    """Launched with programmatic dependence, each kernel waits for the previous one before
    its first global access: the wait comes before any use of the parameters' pointers."""
    for name, text in sources().items():
        for m in re.finditer(r"__global__.*?\{", text, flags=re.S):
            body = text[m.end():]
            body = body[:body.index("\n}")]
            assert "griddepcontrol.wait" in body, name
            before = body[:body.index("griddepcontrol.wait")]
            assert not re.search(r"\b(P\.a|P|a)\.\w+\s*\[|\bstart_walk\b|\bcontext\(|\bvisible\b", before), name


def test_acquired_maps_are_ordered_before_the_copies():
    """Lanes look blocks up and acquire their slabs' tensor maps, an elected lane copies through
    them: a warp barrier lies between every lookup and the copies after it."""
    text = sources()
    body = text["latent_attn.cu"]
    calls = [m.start() for m in re.finditer(r"latent_maps_acquire\(map\);", body)]
    assert len(calls) == 1
    prefill = text["latent_prefill.cu"]
    lookups = [m.start() for m in re.finditer(r"\? block_map\(", prefill)]
    assert len(lookups) == 2
    for src, at in [(body, calls[0])] + [(prefill, x) for x in lookups]:
        rest = src[at:]
        assert rest.index("__syncwarp();") < re.search(r"latent_copy_\w+\(", rest).start()
