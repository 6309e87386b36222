"""Rules of the memory model that no run of a kernel can show to be broken, held to the sources."""
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "jacobi_speculative_decode_gb300", "csrc")


def source(name):
    """A source without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def body(text, name):
    """What stands between the braces of the function `name`."""
    at = text.index("{", re.search(r"\b%s\s*\([^;{]*\)\s*\{" % name, text).start())
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at + 1:i]
    raise ValueError(name)


def test_peers_have_started_before_their_shared_memory_is_written():
    # a CTA's shared memory may be reached by its cluster only once that CTA is known to run: every
    # table kernel arrives on the cluster's barrier before all else, and the first remote store
    # waits for it
    text = source("k_cache.cu")
    kernels = re.findall(r"__cluster_dims__\([^)]*\)[^{;]*?(\w+_kernel)\s*\(", text)
    assert sorted(kernels) == ["compact_kernel", "fork_kernel", "resize_kernel"]
    for k in kernels:
        b = body(text, k)
        first = b.index("cluster_base(")
        assert -1 < b.find("cluster_arrive()") < first, k
        assert re.match(r"cluster_base\(cl, 0,", b[first:]), k          # the use that waits
        assert "map_shared_rank" not in b, k
    base = body(text, "cluster_base")
    assert -1 < base.find("if (use == 0) cluster_wait()") < base.index("map_shared_rank")
    assert text.count("map_shared_rank") == 1


def test_one_lane_reads_what_a_whole_warp_decides_by():
    # marks change while the streaming warp reads them: lanes that read for themselves could decide
    # differently before full-mask shuffles, so one lane reads and all take its value
    b = body(source("k_verify.cu"), "verify_stats_kernel")
    reads = [m.start() for m in re.finditer(r"__ldcg\(&a\.marks", b)]
    assert len(reads) == 1
    assert re.search(r"lane == 0[^;?]*\? \(int\)$", b[:reads[0]])
    for name in ("mark", "seen"):       # every use but its assignments goes through lane 0's value
        uses = [m for m in re.finditer(r"\b%s\b(?!\s*=[^=])" % name, b)]
        shuffled = re.findall(r"__shfl_sync\(0xFFFFFFFFu, %s, 0\)" % name, b)
        assert len(uses) == len(shuffled) == 1, name


def test_every_device_helper_is_called():
    text = {name: source(name) for name in sorted(os.listdir(CSRC))}
    everything = "".join(text.values())
    idle = [(name, f) for name, t in text.items()
            for f in re.findall(r"__device__ (?:__forceinline__|__noinline__|inline) [\w:<> *&]+?\b(\w+)\(", t)
            if len(re.findall(r"\b%s\b" % f, everything)) < 2]
    assert not idle


def test_an_error_word_is_cleared_in_the_callers_stream():
    # a clear in the default stream may run after the call returned, over what a kernel of a
    # non-blocking stream has recorded since
    text = "".join(source(name) for name in sorted(os.listdir(CSRC)))
    assert not re.search(r"\bcudaMem(set|cpy)\s*\(", text)
    take = body(text, "xp_take_error")
    order = [take.index(x) for x in ("cudaMemcpyAsync(", "cudaMemsetAsync(", "cudaStreamSynchronize(")]
    assert order == sorted(order)
    for f in ("xp_get_error", "xp_cache_get_error"):
        assert "xp_take_error(" in body(text, f), f
