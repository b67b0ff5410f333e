"""The gated delta recurrence with enough heads for 32 state columns per workgroup: every k_dim, state widths that end
inside a workgroup's columns, ragged lengths, and inputs and outputs with the heads before the tokens."""
import pytest
import torch

import nvfp4_block_scaled_03_amd as nv
from gpu_util import DEV, say
from test_gpu_gdn import Case

pytestmark = pytest.mark.gpu
SHAPES = [  # b, t, hk, group, dk, dv, lens
    (32, 70, 4, 2, 96, 48, None),
    (16, 129, 8, 2, 64, 16, [129, 128, 65, 64, 63, 1, 0, 129] * 2),
    (33, 66, 4, 2, 32, 80, [66, 65, 1] * 11),
    (16, 100, 4, 2, 128, 112, None),
]


@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s[:6])) for s in SHAPES])
def test_odd_widths(shape):
    say(f"gdn, 32 columns per workgroup, {shape[:6]}")
    c = Case(sum(shape[:6]), *shape)
    dev, kw = c.dev(), c.kw()
    want = [*nv.gdn_forward(*dev, **kw), *nv.gdn_backward(*dev, c.do.to(DEV), c.ds.to(DEV), **kw)]
    torch.cuda.synchronize()
    c.check_forward(*want[:2], str(shape))
    c.check_backward(want[2:], str(shape))

    def turned(x):                                   # [b, t, h, ...] in memory as [b, h, t, ...]
        return x.transpose(1, 2).contiguous().transpose(1, 2)

    views = [turned(x) for x in dev]
    g = nv.gdn_desc(*views, **kw)
    fill = lambda x: turned(torch.full_like(x, 3.0, memory_format=torch.contiguous_format))   # noqa: E731
    o, grads = fill(dev[2]), [fill(x) for x in dev]
    s, d0 = torch.empty_like(want[1]), torch.empty_like(want[1])
    size = max(nv.nvfp4_gdn_forward_workspace_bytes(g), nv.nvfp4_gdn_backward_workspace_bytes(g))
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
    nv.nvfp4_gdn_forward(g, o, s, ws)
    nv.nvfp4_gdn_backward(g, turned(c.do.to(DEV)), c.ds.to(DEV), *grads, d0, ws)
    torch.cuda.synchronize()
    there = torch.from_numpy(c.there()).to(DEV)
    assert torch.equal(s, want[1]) and torch.equal(d0, want[7])
    for x, y in zip([o, *grads], [want[0], *want[2:7]]):
        assert torch.equal(x[there], y[there]) and bool((x[~there] == 3.0).all())
