"""The checkpoint's error by the size of a run: half a step always, relative to the run's largest value only where the
step follows it.  CPU only."""
import numpy as np
import pytest

import oracle as O


@pytest.mark.parametrize("top", [2.0 ** -149, 2.0 ** -130, 127 * 2.0 ** -128, 127 * 2.0 ** -127, 128 * 2.0 ** -127,
                                 127 * 2.0 ** -126, 1.0, 3.4e38])
def test_error_of_a_run(top):
    x = np.random.default_rng(1).uniform(-1, 1, (200, 32)) * top
    x[:, 0] = top
    q, s = O.ckpt_pack(x)
    off = np.abs(O.ckpt_unpack(q, s) - x)
    assert (off <= 2.0 ** (s.astype(np.float64) - 128)).all()
    if top > 127 * 2.0 ** -127:
        assert (off <= top / 127).all()
    else:
        assert (s == 1).all() and (off <= 2.0 ** -127).all()
    if top <= 2.0 ** -130:  # less than half a step: all of it is lost
        assert (q == 0).all() and (off[:, 0] == top).all()
