"""StepState's host side: what upload takes (no GPU needed)."""
import ctypes as C
import warnings

import numpy as np
import pytest


@pytest.fixture(scope="module")
def zf():
    import fsdp_sharded_mixed_flatparameter_amd as m
    return m


@pytest.mark.parametrize("kind", [lambda st: st, bytes, bytearray, lambda st: memoryview(bytes(st)),
                                  lambda st: np.frombuffer(bytes(st), np.uint8), lambda st: list(bytes(st))],
                         ids=["struct", "bytes", "bytearray", "memoryview", "array", "list"])
def test_upload_takes_saved_states(zf, kind):
    """A state saved as bytes in any form, read-only or not, comes back without
    a warning."""
    a = zf.StepState(1024.0, True, window=7, device="cpu")
    st = a.read()
    st.step, st.beta1_pow, st.good_steps = 12, 0.25, 3
    b = zf.StepState(1.0, False, device="cpu")
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        b.upload(kind(st))
    got = b.read()
    assert bytes(got) == bytes(st) and got.step == 12 and C.sizeof(got) == zf.STATE_BYTES
