"""The example that trains and serves an RNN head runs, and learns."""

import numpy as np
import pytest

from examples import rnn_head

pytestmark = pytest.mark.gpu


def test_training_lowers_the_loss_and_raises_the_accepted_length():
    out = rnn_head.run(300)
    first, last = np.mean(out["losses"][:10]), np.mean(out["losses"][-10:])
    assert np.isfinite(out["losses"]).all()
    assert last < 0.85 * first
    assert out["after"] > out["before"]
