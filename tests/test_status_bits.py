"""The binding's names of row_status bits against the header's list."""
import os
import re

import speculative_decoding_verification_57_gb300 as sv

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "specv.h")


def _header_bits():
    """Every bit that the header's declarations tell of."""
    text = open(HEADER).read()
    return {int(n) for n in re.findall(r"\b(\d+)\b", text) if int(n) in {2 ** i for i in range(14)}}


def test_every_bit_has_a_name():
    named = {v for k, v in vars(sv).items() if k.startswith("ST_") and k != "ST_ERROR_MASK"}
    assert named == {2 ** i for i in range(14)}
    assert named <= _header_bits()
    assert {k for k in vars(sv) if k.startswith("ST_")} <= set(sv.__all__)


def test_the_mask_takes_no_refused_row_for_a_good_one():
    """What the calls on the cache, the rollback and the verify calls report
    of a row that they refuse; a zero residual is information."""
    for bit in (sv.ST_ACCEPTED, sv.ST_NO_ROOM, sv.ST_PARENT, sv.ST_LENGTH, sv.ST_BLOCK, sv.ST_PATH, sv.ST_TIMEOUT,
                sv.ST_NONFINITE, sv.ST_TOKEN_RANGE, sv.ST_UNIFORM_RANGE, sv.ST_TEMPERATURE, sv.ST_Q_INVALID,
                sv.ST_FILTER):
        assert sv.ST_ERROR_MASK & bit
    assert (sv.ST_ACCEPTED, sv.ST_NO_ROOM, sv.ST_LENGTH, sv.ST_BLOCK, sv.ST_PATH) == (128, 256, 2048, 4096, 8192)
    assert not sv.ST_ERROR_MASK & sv.ST_ZERO_RESIDUAL
