"""The gated delta recurrence at the ends of its gates' range (signs, reflections) and with growing states, on both
sides of the length at which it goes from tokens to chunks.  Tolerances as derived in test_gpu_gdn.py, with these
factors: with beta up to 2 what is rounded is up to twice as large; where decays exceed 1 a chunk's terms are as
large as the state would be had no update taken anything away from it, G |S0| + (G + G/alpha + ...) |v| with
G = alpha^tokens, and the bound follows that instead of the state's own size."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_03_amd as nv
from gpu_util import DEV, say
from oracle import gdn
from test_gpu_gdn import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [8, 9, 64, 150])
def test_signs_and_reflections(t):
    """alpha of both signs and of magnitude 1; beta |k|^2 of nearly 2, which turns a key's component round."""
    say(f"gdn, alpha in -1 .. 1 and beta up to 2, {t} tokens")
    rng = np.random.default_rng(t)
    alpha = rng.choice([-1.0, 1.0, -0.9, 0.97, 0.0], (2, t, 2), p=[0.3, 0.3, 0.2, 0.18, 0.02])
    c = Case(60 + t, 2, t, 1, 2, 64, 48, alpha=alpha, beta=rng.choice([0.0, 1.0, 1.5, 2.0], (2, t, 2)))
    c.e *= 2
    o, s = nv.gdn_forward(*c.dev(), **c.kw())
    grads = nv.gdn_backward(*c.dev(), c.do.to(DEV), c.ds.to(DEV), **c.kw())
    torch.cuda.synchronize()
    assert all(bool(torch.isfinite(x).all()) for x in (o, s, *grads))
    c.check_forward(o, s, f"{t} tokens")
    c.check_backward(grads, f"{t} tokens")


@pytest.mark.parametrize("state", [True, False], ids=["state", "no_state"])
@pytest.mark.parametrize("alpha,t", [(4.0, 8), (4.0, 9), (4.0, 14), (1.25, 8), (1.25, 64)])
def test_growing_states(alpha, t, state):
    say(f"gdn, alpha = {alpha}, {t} tokens, state {state}")
    c = Case(70 + t, 1, t, 1, 1, 64, 32, alpha=alpha, state=state)
    o, s = nv.gdn_forward(*c.dev(), **c.kw())
    torch.cuda.synchronize()
    if t > 8:                                    # by chunks
        size = gdn.forward(*c.host(), **c.okw())[2].item()
        free = alpha ** t * ((np.linalg.norm(c.state.numpy()) if state else 0.0)
                             + alpha / (alpha - 1) * np.linalg.norm(c.v.float().numpy(), axis=-1).max())
        c.e *= max(1.0, free / size)
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(s).all())
    c.check_forward(o, s, f"alpha {alpha}, {t} tokens")
