"""The operators around the cache where calls that their documentation allows lie at a border: blocks of cached heads that are
not full, pages that two sequences name, groups without values, scales far apart, long moves."""

import functools

import numpy as np
import pytest

import _cache_ops as R
from test_cache_ops_gpu import Setup, random_trees

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- blocks of heads


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,D,bits,group", [(9, 128, 4, 128), (11, 64, 8, 64), (13, 128, 4, 32), (20, 64, 4, 64), (9, 80, 3, 40),
                                                (11, 24, 8, 8), (5, 256, 8, 64), (7, 256, 8, 256)])
def test_attention_blocks_of_heads_that_are_not_full(heads, D, bits, group, dtype, monkeypatch):
    """Numbers of cached heads whose last block has fewer than the others, in a pool whose every slot is used: the last block
    takes nothing from behind the last token."""
    monkeypatch.setattr(R, "shuffled_table", functools.partial(R.shuffled_table, spare=0))
    key = f"{heads}-{D}-{bits}-{group}-{dtype}"
    for new, grp in ((1, 1), (3, 2)):
        s = Setup(f"blocks{key}{new}", [15, 160, 33, 0], [new] * 4, heads=heads, grp=grp, D=D, bits=bits, group=group, dtype=dtype, room=1 << 20,
                  page_size=1, tree=random_trees if new > 1 else None)
        assert s.kv[0].n_slots == sum(s.past) + 4 * new  # no page is left over
        s.check()
