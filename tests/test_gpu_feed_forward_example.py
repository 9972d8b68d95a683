"""The feed-forward example at a small size: it learns, and single tokens agree with the batch."""
import os
import sys

import pytest

from conftest import ROOT, log

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,width,hidden", [(256, 192, 320), (2100, 264, 1040)])
def test_feed_forward(fqlib, tokens, width, hidden):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import w4_feed_forward
    log(f"feed-forward example {tokens} {width} {hidden}")
    losses, apart = w4_feed_forward.run(tokens, width, hidden, steps=6)
    assert losses[-1] < 0.8 * losses[0], losses
    # h of one token and of the batch round alike but for sums in another order: a bfloat16
    # step (2^-7) of some h, carried by a row of the down weight, and one of y itself
    assert apart < 2 * 2.0 ** -7, apart
