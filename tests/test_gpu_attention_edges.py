"""Attention on both sides of what makes a prefix go by panels instead of tiles: 96 rows, and 7 << 20 products of rows,
heads and prefix tokens beside 256 own tokens or more (12 << 20 beside fewer)."""
import pytest

from gpu_util import say
from test_gpu_attention import MODES, Case

pytestmark = pytest.mark.gpu
OWN = [260, 0, 1, 17, 255]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("batch,group,prefix,lens", [
    (6, 16, 76458, OWN + [64]), (6, 16, 76459, OWN + [64]),      # one token short of 7 << 20, and there
    (5, 19, 77300, OWN),                                         # 95 rows
    (4, 32, 57344, [0, 1, 17, 240]), (4, 32, 57344, [0, 1, 17, 241]),   # a table of 240, of 256 own tokens
    (2, 64, 98304, [5, 0]), (2, 64, 98303, [5, 0])])             # 12 << 20
def test_both_sides(batch, group, prefix, lens, mode):
    lens = lens[:batch]
    say(f"attention {mode} {batch * group} rows, prefix {prefix}, own {lens}")
    c = Case(batch * group + prefix, batch, 1, group, 64, prefix, lens, 16, mode)
    c.check(c.run(), f"{mode} {batch * group} rows {prefix}")
