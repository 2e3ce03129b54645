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
