"""Attention over a cache with a scale per slot whose scales lie far apart: rows of zeros (which the write gives the
scale 1) among small ones, rows that are large and hardly count, scales at the ends of their range.  Each against the
FP64 oracle within its derived bound, which does not know the scales: a token's precision must not depend on another's."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_03_amd as nv
from gpu_util import DEV, say
from oracle import fp8_kv, kv_cache

pytestmark = pytest.mark.gpu
F32 = np.float32

# batch, kv_heads, group, dim, prefix, longest own, page: every way a call is split
LAYOUTS = {
    "joint": (3, 2, 4, 64, 100, 150, 16),              # a short prefix, walked by each sequence itself
    "joint_256": (2, 1, 3, 256, 33, 300, 32),
    "ranges": (4, 1, 4, 128, 3000, 1500, 64),          # prefix and own tokens in several ranges, joined
    "ranges_256": (5, 1, 4, 256, 2100, 40, 64),
    "own_only": (2, 2, 2, 128, 0, 1300, 16),
    "panels": (1, 1, 128, 128, 57411, 300, 64),        # codes of the prefix widened once for 128 rows
    "panels_64": (2, 1, 64, 64, 57411, 290, 16),
}


def _encode(x):
    """E4M3 codes of rows [n, heads, dim] as they stand."""
    return fp8_kv.quantize_kv(x.reshape(-1, x.shape[-1]).astype(F32), "given", 1.0)[0].reshape(x.shape)


def _case(layout, kind):
    batch, hk, group, dim, prefix, longest, page = LAYOUTS[layout]
    rng = np.random.default_rng(sum(map(ord, layout + kind)))
    n_pre, n_seq = -(-prefix // page), -(-longest // page)
    total = n_pre + batch * n_seq
    order = rng.permutation(total).astype(np.int32)
    prefix_pages, pages = order[:n_pre], order[n_pre:].reshape(batch, n_seq)
    lens = rng.integers(0, longest + 1, batch).astype(np.int32)
    lens[0] = longest
    shape = (total * page, hk)
    # queries near a direction of +-1, keys along it: a slot's score is about what `score` asks for
    u = rng.choice([-1.0, 1.0], (hk, dim))
    q = np.repeat(u, group, 0)[None] * (1 + 0.05 * rng.standard_normal((batch, hk * group, dim)))
    q = torch.from_numpy(q.astype(F32)).to(torch.bfloat16)
    v = (1.5 + rng.standard_normal((*shape, dim))) * 80
    score = rng.uniform(-1, 1, shape)                   # natural logarithm of a slot's weight
    vs = np.exp(rng.uniform(-1, 1, shape)) * 1e-5
    if kind == "zero_rows":                             # as the write leaves them
        zero = rng.random(shape) < 0.02
        v[zero], vs[zero] = 0.0, 1.0
    elif kind == "zero_rows_tiny":
        zero = rng.random(shape) < 0.02
        v[zero], vs[zero] = 0.0, 1.0
        vs[~zero] *= 2.0 ** -70
    elif kind == "far_apart":                           # the larger a scale, the less it counts
        power = rng.uniform(-40, 40, shape)
        vs, score = 2.0 ** power, -1.5 * np.log(2) * power
    elif kind == "one_large":
        big = rng.random(shape) < 0.01
        vs[big], score[big] = 2.0 ** 24 * 1e-5, -40.0
    elif kind == "dominant_small":
        one = rng.random(shape) < 0.002
        score[one], vs[one] = 9.0, 1e-9
        zero = rng.random(shape) < 0.01
        v[zero], vs[zero] = 0.0, 1.0
    elif kind == "floor":
        vs = np.full(shape, 2.0 ** -100)
    elif kind == "ceiling":                             # values to 2^110; the sums stay in FP32's range
        vs = 2.0 ** rng.uniform(80, 101, shape)
    k = np.broadcast_to(np.sign(score)[..., None] * u * 16.0, v.shape)
    ks = np.maximum(np.abs(score), 1e-3) / (16.0 * dim ** 0.5)
    codes = [_encode(x).reshape(total, page, hk, dim) for x in (k, v)]
    scales = [x.astype(F32).reshape(total, page, hk) for x in (ks, vs)]
    dev = [torch.from_numpy(np.ascontiguousarray(a)).to(DEV) for a in (*codes, *scales, prefix_pages, pages, lens)]
    want = kv_cache.attention(q.float().numpy(), *codes, *scales, prefix_pages, prefix, pages, lens, dim ** -0.5)
    got = nv.prefix_attention(q.to(DEV), nv.KVCache(*dev[:4]), dev[4], prefix, dev[5], dev[6])
    torch.cuda.synchronize()
    return got.float().cpu().numpy().astype(np.float64), *want


KINDS = ["zero_rows", "zero_rows_tiny", "far_apart", "one_large", "dominant_small", "floor", "ceiling"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout", sorted(LAYOUTS))
def test_scales_far_apart(layout, kind):
    say(f"attention, a scale per slot, {kind}, {layout} {LAYOUTS[layout]}")
    got, want, tol = _case(layout, kind)
    assert np.all(np.isfinite(got)), f"{np.sum(~np.isfinite(got))} outputs are not finite"
    off = np.abs(got - want)
    i = np.unravel_index(np.argmax(off / tol), off.shape)
    assert np.all(off <= tol), f"{np.sum(off > tol)} of {off.size} outputs off, worst at {i}: gpu {got[i]} want {want[i]} tol {tol[i]}"


def test_written_zero_rows():
    """Through the write itself: padding rows of zeros among rows of 1e-5, K and V from the same projection."""
    say("attention over a cache whose write met rows of zeros, V of 1e-5")
    b, hk, g, d, page, n = 2, 2, 2, 128, 16, 250
    gen = torch.Generator(device=DEV).manual_seed(7)
    k, v = (torch.randn(b * n, hk, d, generator=gen, device=DEV) for _ in range(2))
    v *= 1e-5
    v[torch.rand(b * n, generator=gen, device=DEV) < 0.05] = 0.0
    cache = nv.KVCache.allocate(b * 16, page, hk, d, device=DEV)
    pages = torch.arange(b * 16, dtype=torch.int32, device=DEV).view(b, 16)
    slots = (pages.long()[:, :, None] * page + torch.arange(page, device=DEV)).view(b, -1)[:, :n].reshape(-1).contiguous()
    nv.kv_cache_write(k, v, cache, slots)
    q = torch.randn(b, hk * g, d, generator=gen, device=DEV).to(torch.bfloat16)
    lens = torch.full((b,), n, dtype=torch.int32, device=DEV)
    o = nv.prefix_attention(q, cache, None, 0, pages, lens)
    torch.cuda.synchronize()
    host = [x.cpu().numpy() for x in (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale)]
    want, tol = kv_cache.attention(q.float().cpu().numpy(), *host, None, 0, pages.cpu().numpy(), lens.cpu().numpy(), d ** -0.5)
    assert np.all(np.abs(o.float().cpu().numpy() - want) <= tol)
