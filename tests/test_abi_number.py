"""The ABI number names one set of entry points: a library with others has another."""
import hashlib

import w8a8_int8_quantized_qk_amd as qk

# number: (entry points, the first digits of the SHA-256 of their sorted names, one per line)
SETS = {8: (30, "a3cc2047284d0397"), 9: (38, "56711fc9ca7fd1de")}


def test_the_number_names_this_set():
    count, digest = SETS[qk.ABI_VERSION]
    assert len(qk.EXPORTED) == len(set(qk.EXPORTED)) == count
    assert digest == hashlib.sha256("\n".join(sorted(qk.EXPORTED)).encode()).hexdigest()[:16]


def test_no_two_sets_share_a_number():
    assert len({v[0] for v in SETS.values()}) == len(SETS)
