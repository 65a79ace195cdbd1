"""Order of the programmatic-launch instructions, read from the kernels' sources.  The sparse attention reads q before it
waits for the kernel before it, so that kernel may let it start only when everything earlier in the stream is complete:
a kernel that goes out as a dependent launch waits first.  Exempt are kernels whose next launch is always their own
combine, which waits before it reads anything."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp4_compressed_sparse_kv_b200", "csrc")
FOLLOWED_BY_THEIR_COMBINE = {"attn_split_tc_kernel", "dense_attn_kernel"}


def kernels(text):
    """(name, body) of every __global__ function of a source."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__global__[^;{]*?\b(\w+_kernel)\s*\(", text):
        at = text.index("{", m.end())
        depth, end = 1, at + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
        yield m.group(1), text[at:end]


def test_dependent_launches_wait_before_they_release():
    found = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = open(path).read()
        for name, body in kernels(text):
            # launched with <<<>>> alone: the kernel starts when everything before it is complete
            plain = re.search(r"\b%s\b(<[^;]*?>)?\s*<<<" % name, text) is not None
            release, wait = body.find("grid_dep_launch()"), body.find("grid_dep_wait()")
            if release >= 0 and not plain:
                found[name] = 0 <= wait < release
    assert FOLLOWED_BY_THEIR_COMBINE < set(found)
    assert {"kv_append_kernel", "kv_unpack_kernel", "topk_kernel", "reuse_kernel", "select_kernel"} < set(found)
    assert {n for n, ok in found.items() if not ok} == FOLLOWED_BY_THEIR_COMBINE
