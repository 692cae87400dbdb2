"""GPU tests of the many-adapter entry points where values are not finite and
where sizes pass a launch's reach.

An infinity or NaN of one adapter or of one row changes that adapter's rows, or
that row, alone: everything else keeps its bits. What it does change follows
the formula: an infinity times a finite nonzero number is an infinity of their
sign.
"""

import numpy as np
import pytest

from gpu_util import require_gpu, say
from test_gpu_multi import Case

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def api():
    return require_gpu()


def set_ids(c, ids):
    c.ids = np.asarray(ids, np.int32)
    c.d["ids"].copy_(c.d["ids"].new_tensor(c.ids.tolist()))


# ---- a single token -------------------------------------------------------------------

@pytest.mark.parametrize("K,N,r", [(512, 512, 64), (512, 264, 16), (320, 72, 8)])
@pytest.mark.parametrize("bare", [-1, 3])
@pytest.mark.parametrize("what", ["L1", "L2", "scale"])
def test_bare_token_beside_a_diverged_adapter(api, K, N, r, bare, what):
    """A token without an adapter is the base alone, whatever adapter 0 holds."""
    import torch

    say(f"multi bare token K={K} N={N} r={r} id={bare} {what}")
    c = Case(api, 1, K, N, r, 3, "one")
    set_ids(c, [bare])
    Y, T = c.fwd(want_T=True)
    assert torch.isfinite(Y).all() and (T == 0).all()
    for value in (INF, -INF, NAN):
        if what == "scale":
            c.d["scale"][:] = value
        else:
            c.d[what][0, ::3, ::5] = value
            c.d[what][2, ::3, ::5] = value
        Y2, T2 = c.fwd(want_T=True)
        assert torch.equal(Y2, Y) and (T2 == 0).all(), value
