"""CPU checks of the appends' outputs against their inputs: a block of threads writes lens_out,
key_pos and scores while others read lens, cu_new, the table and the positions."""
import pytest

from test_cache_abi import append, lib  # noqa: F401
from test_cache_more_abi import append8

LENS, CU, TABLE, POS, FREQ, KP, SC, LO = (0x30000 + 0x1000 * i for i in range(8))


def call(f, lib, **over):
    """Two sequences, one head, 32 slots a row; refused (-3) for a stride of K when all else is well."""
    a = dict(khs=164, lens=LENS, cu=CU, table=TABLE, trs=6, pos=POS, freq=FREQ, kp=KP, kprs=64, kphs=64, lo=LO)
    if f is append:
        a.update(sc=SC, scrs=64, schs=64)
    return f(lib, **{**a, **over})


# (outputs at these places, of sizes in bytes: lens 8, cu_new 12, a table row 8 of 24, positions 12, inv_freq 640)
MEET = [dict(lo=LENS), dict(lo=LENS + 4), dict(lo=LENS - 4), dict(lo=CU + 4), dict(lo=CU + 8), dict(lo=CU - 4), dict(lo=TABLE + 4), dict(lo=TABLE + 20),
        dict(lo=TABLE + 28), dict(lo=POS + 8), dict(lo=POS - 4), dict(lo=FREQ + 636), dict(lo=KP + 124), dict(lo=KP + 256), dict(lo=KP + 380),
        dict(kp=LENS - 124), dict(kp=LENS - 256 - 124), dict(kp=CU), dict(kp=TABLE - 20 - 256), dict(kp=POS - 8), dict(kp=FREQ),
        dict(axes=3, axs=16, lo=POS + 72), dict(kp=TABLE - 124)]
APART = [dict(), dict(lo=LENS + 8), dict(lo=LENS - 8), dict(lo=CU + 12), dict(lo=CU - 8), dict(lo=TABLE + 8), dict(lo=TABLE + 16), dict(lo=TABLE + 32),
         dict(lo=POS + 12), dict(lo=FREQ + 640), dict(lo=KP + 128), dict(lo=KP + 248), dict(lo=KP + 384), dict(kp=LENS - 128), dict(kp=LENS - 248),
         dict(kp=LENS - 384), dict(kp=TABLE - 128, trs=2), dict(kp=None), dict(lo=None), dict(axes=3, axs=16, lo=POS + 52)]


@pytest.mark.parametrize("f", [append, append8])
def test_outputs_that_meet_inputs_are_refused(lib, f):
    for over in MEET:
        assert call(f, lib, **over) == -1, over
    for over in APART:
        assert call(f, lib, **over) == -3, over


def test_scores_that_meet_other_arrays_are_refused(lib):
    for at in (LENS, LENS - 124, CU + 8, TABLE - 256 - 8, KP + 64, KP - 128 + 4, LO - 256):
        assert call(append, lib, sc=at) == -1, hex(at)
    for at in (KP + 128, LENS - 200, LO + 8):  # (side by side, and between the rows)
        assert call(append, lib, sc=at) == -3, hex(at)
