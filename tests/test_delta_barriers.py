"""The order of workgroup memory in the delta rule's gradients, read from the source: a sum that lacks the
part of a slower wave is rare and silent on the card, so no run of the kernel shows that nothing orders it."""
import re

from nonlinear_rnn_solve_newton_amd import build


def kernel(name):
    """The text of a kernel of delta_rule.h, without comments."""
    s = re.sub(r"//[^\n]*", "", (build.CSRC / "delta" / "delta_rule.h").read_text())
    at = s.index(f" {name}(")
    return s[at:s.index("\n}\n", at)]


def test_pair_matrix_is_whole_before_its_columns_are_summed():
    """W = D0 q.k + D1 k.k: one half of the waves stores its part, the other adds to it, then every wave sums 8 rows
    that are other waves' and, after their sums are joined, reads them again."""
    s = kernel("delta_grad_kernel")
    stored = [m.start() for m in re.finditer(r"mt\.w\[[^\]]*\] = ", s)]
    added = [m.start() for m in re.finditer(r"mt\.w\[[^\]]*\] \+= ", s)]
    read = [m.start() for m in re.finditer(r"(?<!\+= )v \+= mt\.w\[", s)]
    assert len(stored) == 2 and len(added) == 1 and len(read) == 2
    assert max(stored) < added[0] < min(read)
    for a, b in ((max(stored), added[0]), (added[0], min(read))):
        assert "__syncthreads();" in s[a:b]
    # and they have been read before the next value head's stage or matrices take their place
    assert "__syncthreads();" in s[max(read):]
