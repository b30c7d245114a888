"""What reading the kernels' sources shows and running them does not."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_rank_kv_gb300", "csrc")
BUILTIN = r"(?:blockIdx|threadIdx|gridDim|blockDim)\.[xyz]"


def comparisons(text):
    """(built-in, the other side's first word) of the comparisons that have one of CUDA's unsigned numbers,
    itself and not cast, on one side."""
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    right = re.findall(rf"({BUILTIN})\s*(?:<=|>=|<(?!<)|>(?!>))\s*([\w.]+)", text)
    left = re.findall(rf"([\w.\]]+)\s*(?:<=|>=|(?<!<)<|(?<!>)>)\s*({BUILTIN})", text)
    return right + [(b, a) for a, b in left]


def test_no_signed_number_is_compared_with_an_unsigned_one():
    """blockIdx.x < n with an int n = -1 ("nothing to do") is true: the int becomes 2^32 - 1.  Constants and other
    built-ins are on the other side of such a comparison, or the built-in is cast."""
    found = []
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh")):
            with open(os.path.join(CSRC, name)) as f:
                found += [(name, a, b) for a, b in comparisons(f.read())
                          if not re.fullmatch(rf"{BUILTIN}|\d\w*|k[A-Z]\w*", b)]
    assert not found


def test_the_rule_sees_both_sides():
    assert comparisons("x = blockIdx.x < n ? 1 : 0;") == [("blockIdx.x", "n")]
    assert comparisons("if (a.count >= gridDim.y) f<<<1, 2>>>();") == [("gridDim.y", "a.count")]
    assert comparisons("static_cast<int>(blockIdx.x) < n; for (int i = blockIdx.x; i < n;)  // blockIdx.x < n") == []
