"""More of what the paged cache's calls refuse on the host, each refusal told by its own message or
status; on the CPU, where nothing is launched."""
import pytest

from test_paged_cpu import POOL, TABLE, lib


@pytest.mark.parametrize("want,pos", [
    (1, 1024), (1, 1024 - 12), (1, 1024 + 12),          # delta: 4 rows, from 1024 on
    (1, 2048), (1, 2048 + 12), (1, 4096), (1, 4096 + 396),      # seq_lens; ref, of 100 pages
])
def test_resize_pos_of_its_own(want, pos):
    """pos is written while delta, seq_lens and ref are still read: it cannot be one of them."""
    G = lib()
    a = dict(delta=1024, lens=2048, S=4, **TABLE, ref=4096, **POOL, H=8, d=128, pos=pos, status=None,
             ws=8192, wsb=16, stream=None)
    assert G._lib.gret_paged_resize(*a.values()) == want
