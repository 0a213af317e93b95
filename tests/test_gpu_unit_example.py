"""The example of a unit applies every one of its steps: nothing in it overflows."""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_every_step_is_applied():
    import unit_saved8
    assert torch.cuda.is_available()
    losses, unit = unit_saved8.train(steps=12, batch=8, length=16)
    st = unit.opt.state.read()
    assert st.step == 12 and st.last_skipped == 0 and st.overflow == 0
    assert all(math.isfinite(v) for v in losses) and bool(torch.isfinite(unit.opt.master).all())
