"""Which rotary kernels are built: the ones that some call reaches, and no others."""
import os
import re

import pytest

from speculative_verify_gdn_amd import gdn

HALVES, NEIGHBOURS, PART = 0, 1, 2


def reached():
    """(bf16, elements of a piece, how pairs lie) over every size of head and of what turns in it."""
    kinds = set()
    for bf16 in (0, 1):
        whole = 8 if bf16 else 4                                  # elements of 16 bytes
        for pairs in (HALVES, NEIGHBOURS):
            for D in range(16, 513, 16):
                for rot in range(0, D + 1, 2):
                    of = rot if pairs == NEIGHBOURS else rot // 2   # made of pieces
                    e = next(n for n in (whole, whole // 2, 1) if of % n == 0)
                    kinds.add((bf16, e, PART if pairs == NEIGHBOURS and e > 1 and rot < D else pairs))
    return kinds


def test_no_kernel_without_a_call():
    if not os.path.exists(gdn.LIB_PATH):
        pytest.skip("libgdn.so not built")
    code = open(gdn.LIB_PATH, "rb").read()
    built = {(int(b), 8 if int(b) else 4, int(p)) for b, p in re.findall(rb"11rope_kernelILb([01])ELNS0_5PairsE([012])E", code)}
    built |= {(int(b), int(e), int(p))
              for b, e, p in re.findall(rb"18rope_narrow_kernelILb([01])ELi(\d)ELi\dELNS0_5PairsE([012])E", code)}
    assert built == reached()
