"""A sequence given in parts: the state handed on from part to part, its gradient handed back."""
import pytest
import torch

import nvfp4_block_scaled_03_amd as nv
from gpu_util import DEV, say
from test_gpu_gdn import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cuts", [[0, 64, 300], [0, 5, 133, 134, 300]], ids=["2_parts", "4_parts"])
def test_parts_make_the_whole(cuts):
    say(f"gdn forward and backward in parts {cuts}")
    c = Case(31, 2, cuts[-1], 2, 2, 64, 48)
    parts = [[x[:, a:b] for x in c.dev()] for a, b in zip(cuts, cuts[1:])]
    do, states, outs, grads = c.do.to(DEV), [c.state.to(DEV)], [], []
    for p in parts:
        o, s = nv.gdn_forward(*p, scale=c.scale, state=states[-1])
        outs.append(o)
        states.append(s)
    d_state = c.ds.to(DEV)
    for p, s, a, b in reversed(list(zip(parts, states, cuts, cuts[1:]))):
        *g, d_state = nv.gdn_backward(*p, do[:, a:b], d_state, scale=c.scale, state=s)
        grads.append(g)
    torch.cuda.synchronize()
    c.check_forward(torch.cat(outs, 1), states[-1], "parts")
    c.check_backward((*[torch.cat(x, 1) for x in zip(*grads[::-1])], d_state), "parts")
