"""Orderings that a run cannot show to be missing, read from the CUDA sources."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "means_clustering_gmm_b200", "csrc")


def code(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"/\*.*?\*/", " ", f.read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def test_lanes_meet_before_they_overwrite_a_tiles_biases():
    """An epilogue warp keeps a tile's biases in shared memory: a warp barrier
    stands between the last tile's reads and the next tile's writes, and one
    between the writes and their reads."""
    text = code("experts_tc.cu")
    loop = text.index("for (int idx = first", text.index("float *gate_b"))
    write = text.index("gate_b[i] =", loop)
    read = text.index("reinterpret_cast<const float4 *>(gate_b", write)
    assert "__syncwarp()" in text[loop:write]
    assert "__syncwarp()" in text[write:read]


def test_guarded_elements_are_read_by_ordinary_loads():
    """`p < N ? load_elem(...) : 0` reads behind its test only if the load is
    one the compiler may not move above it, which __ldg of 16-bit types is not."""
    text = code("common.cuh")
    assert "load_elem" in text and "__ldg" not in text
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".h")):
            # every __ldg left names a 32- or 128-bit array, none a generic element
            for arg in re.findall(r"__ldg\(([^;]*)", code(name)):
                assert not re.match(r"\(?(const )?(T|XT|__half|__nv_bfloat16)\b", arg), (name, arg)


def test_shared_memory_limits_do_not_depend_on_the_call():
    """A kernel's limit of dynamic shared memory is process-wide: set to one
    call's own size it can be lowered by another thread before the launch."""
    for name, own in (("kmeans.cu", "sc_smem"), ("gmm_simt.cu", "smem")):
        calls = re.findall(r"cudaFuncSetAttribute\(([^;]*);", code(name))
        assert calls
        for c in calls:
            assert not re.search(rf"\b{own}\b", c), (name, c)


def test_no_plain_static_is_written_by_the_calls():
    """What launches ask a device for once is kept per device, in atomics."""
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".h")):
            assert not re.findall(r"^\s+static (?:int|unsigned|size_t|int64_t) \w+ = 0;", code(name),
                                  re.M), name
