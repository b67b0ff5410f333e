"""Where the tensors of the cache, attention and the recurrence are: calls that would give a kernel addresses that are
not the GPU's are refused before anything is launched."""
import weakref

import pytest
import torch

import nvfp4_block_scaled_03_amd as nv

BF16 = torch.bfloat16


def _cache():
    return nv.KVCache.allocate(4, 16, 2, 64, device="cpu")


def _gdn(t):
    q, v = torch.zeros(2, t, 1, 32).to(BF16), torch.zeros(2, t, 2, 16).to(BF16)
    return q, q, v, torch.zeros(2, t, 2), torch.zeros(2, t, 2)


HOST_CALLS = {
    "write": lambda: nv.kv_cache_write(torch.zeros(3, 2, 64), torch.zeros(3, 2, 64), _cache(), torch.arange(3)),
    "read": lambda: nv.kv_cache_read(_cache(), torch.arange(3)),
    "attention": lambda: nv.prefix_attention(torch.zeros(2, 4, 64).to(BF16), _cache(), torch.zeros(1, dtype=torch.int32), 5,
                                             torch.ones(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32)),
    "step": lambda: nv.gdn_forward(*_gdn(1)),
    "forward": lambda: nv.gdn_forward(*_gdn(70)),
    "backward": lambda: nv.gdn_backward(*_gdn(70), _gdn(70)[2]),
}


@pytest.mark.parametrize("name", sorted(HOST_CALLS))
def test_host_tensors_are_refused(name):
    with pytest.raises(ValueError, match="GPU"):
        HOST_CALLS[name]()


@pytest.mark.parametrize("workspace", [torch.empty(1 << 22, dtype=torch.uint8, device="meta"),
                                       torch.empty(1, dtype=torch.uint8).expand(1 << 22)], ids=["elsewhere", "one_byte"])
def test_workspaces_elsewhere_or_not_whole_are_refused(workspace):
    cache, t = _cache(), _gdn(70)
    table, lens = torch.ones(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="workspace"):
        nv.prefix_attention(torch.zeros(2, 4, 64).to(BF16), cache, torch.zeros(1, dtype=torch.int32), 5, table, lens,
                            workspace=workspace)
    with pytest.raises(ValueError, match="workspace"):
        nv.gdn_forward(*t, workspace=workspace)
    with pytest.raises(ValueError, match="workspace"):
        nv.gdn_backward(*t, t[2], workspace=workspace)


def test_strides_of_single_entries_do_not_count():
    """An axis of one entry may have any stride; what the kernels are told for it is the row's size."""
    one = torch.as_strided(torch.zeros(64).to(BF16), (1, 1, 64), (4099, 3, 1))
    assert nv._rows3(one, "q")[1:] == (64, 64)
    rows = torch.as_strided(torch.zeros(4096).to(BF16), (3, 1, 64), (128, 68, 1))
    assert nv._rows3(rows, "q")[1:] == (128, 64)
    x = torch.as_strided(torch.zeros(4096).to(BF16), (1, 3, 1, 64), (9, 128, 68, 1))
    assert nv._gdn_rows(x, "q", (1, 3, 1, 64), BF16, x.device)[2:] == (128, 64)
    gates = torch.as_strided(torch.zeros(64), (1, 3, 1), (0, 5, 0))
    assert nv._gdn_rows(gates, "alpha", (1, 3, 1), torch.float32, gates.device)[2:] == (5, 1)


def test_a_descriptor_holds_what_it_points_to():
    """Made from temporaries, it must not be left with addresses that the allocator hands out again."""
    q, k, v, alpha, beta = _gdn(5)
    state, lens = torch.zeros(2, 2, 32, 16), torch.zeros(2, dtype=torch.int32)
    alive = [weakref.ref(x) for x in (q, v, alpha, beta, state, lens)]
    g = nv.gdn_desc(q, k, v, alpha, beta, state=state, lens=lens)
    del q, k, v, alpha, beta, state, lens
    assert all(r() is not None for r in alive)
    del g
    assert all(r() is None for r in alive)


def test_missing_tables_are_named():
    cache, q = _cache(), torch.zeros(2, 4, 64).to(BF16)
    table, lens = torch.ones(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    for pre, pages, n, name in ((None, table, lens, "prefix_pages"), (table[0], table, None, "lens")):
        with pytest.raises(TypeError, match=name):
            nv.prefix_attention(q, cache, pre, 5, pages, n)
    with pytest.raises(TypeError, match="slots"):
        nv.kv_cache_write(q[:, :2], q[:, :2], cache, [0, 1])


def test_a_stream_waits_for_its_own_device(monkeypatch):
    """A stream of another device than the current one waits for what produced the inputs there."""
    class Stream:
        device, waited = torch.device("cuda:1"), []

        def wait_stream(self, other):
            self.waited.append(other)

    s = Stream()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: ("current", device))
    monkeypatch.setattr(torch.cuda, "stream", lambda x: ("on", x))
    assert nv._on_stream(s) == ("on", s) and s.waited == [("current", torch.device("cuda:1"))]


def test_panels_pay_earlier_beside_own_tokens():
    """The split of a prefix, as its workspace shows it: many rows take panels (ranges of 256 tokens, one workgroup for
    128 rows) from 12 << 20 products of rows, heads and tokens on, from 7 << 20 with 256 own tokens or more."""
    def ranges(rows, prefix, max_len, dim=128):
        cache = nv.KVCache.allocate(1, 16, 8, dim, device="cpu")
        size = nv.nvfp4_prefix_attention_workspace_bytes(cache, rows // 4, 32, prefix, max_len)
        own = 0 if max_len == 0 else max(1, min(1024 // (8 * rows // 4), -(-max_len // 512)))
        for n in range(1, 600):
            ml = -(-rows * 8 * n * 8 // 256) * 256
            if n > 1 and size == ml + rows * 8 * n * dim * 4:
                return n - own
        return 1

    tiles = {rows: max(1, 512 // (8 * -(-rows // 16))) for rows in (64, 80, 96, 256)}
    for rows, max_len, least in ((96, 0, 12), (256, 0, 12), (96, 255, 12), (96, 256, 7), (256, 512, 7)):
        edge = -(-(least << 20) // (rows * 8))
        assert ranges(rows, edge, max_len) > ranges(rows, edge - 1, max_len) == tiles[rows], (rows, max_len)
    for rows in (64, 80):                                   # less than three quarters of a panel
        assert ranges(rows, 65536, 0) == tiles[rows]
    assert ranges(256, 65536, 0, dim=256) == tiles[256]
