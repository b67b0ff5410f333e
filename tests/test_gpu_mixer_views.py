"""Views whose axes of one entry have strides of their own: calls on them are the calls on their contents."""
import pytest
import torch

import nvfp4_block_scaled_03_amd as nv
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _odd(x, axes):
    """x, with strides of 4099 and 1 on axes of one entry."""
    assert all(x.shape[a] == 1 for a in axes)
    stride = list(x.stride())
    for a, s in zip(axes, (4099, 1)):
        stride[a] = s
    return torch.as_strided(x, x.shape, stride, x.storage_offset())


def test_one_sequence_of_one_head():
    say("attention, cache and recurrence on views with arbitrary strides where an axis has one entry")
    gen = torch.Generator(device=DEV).manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(BF16)   # noqa: E731
    caches = [nv.KVCache.allocate(4, 16, 1, 64, device=DEV) for _ in range(2)]
    k, v, at = rnd(20, 1, 64), rnd(20, 1, 64), torch.arange(20, device=DEV)
    nv.kv_cache_write(k, v, caches[0], at)
    nv.kv_cache_write(_odd(k, [1]), _odd(v, [1]), caches[1], at)
    assert torch.equal(caches[0].k_codes, caches[1].k_codes) and torch.equal(caches[0].v_scale, caches[1].v_scale)
    pages, lens = torch.arange(4, dtype=torch.int32, device=DEV).view(1, 4), torch.full((1,), 20, dtype=torch.int32, device=DEV)
    for shape, axes in (((1, 1, 64), (0, 1)), ((1, 3, 64), (0,)), ((3, 1, 64), (1,))):
        q = rnd(*shape)
        args = (caches[0], None, 0, pages.expand(shape[0], 4).contiguous(), lens.expand(shape[0]).contiguous())
        assert torch.equal(nv.prefix_attention(q, *args), nv.prefix_attention(_odd(q, axes), *args))
        out = torch.zeros_like(q)
        nv.prefix_attention(q, *args, out=_odd(out, axes))
        assert torch.equal(out, nv.prefix_attention(q, *args))
    for t in (1, 70):
        q, k = (torch.nn.functional.normalize(rnd(1, t, 1, 64).float(), dim=-1).to(BF16) for _ in range(2))
        v, alpha, beta = rnd(1, t, 1, 32), torch.rand(1, t, 1, device=DEV), torch.rand(1, t, 1, device=DEV)
        odd = [_odd(x, [0, 2]) for x in (q, k, v, alpha, beta)]
        a, b = nv.gdn_forward(q, k, v, alpha, beta), nv.gdn_forward(*odd)
        g, h = nv.gdn_backward(q, k, v, alpha, beta, v), nv.gdn_backward(*odd, _odd(v, [2]))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((*a, *g), (*b, *h)))
