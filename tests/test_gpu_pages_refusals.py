"""Page calls on a table whose lengths cannot be: compact and free change nothing."""
import numpy as np
import pytest
import torch

import fp8_mla_latent_gb300 as pkg
from pages_ref import Pool
from test_gpu_pages import Dev

pytestmark = pytest.mark.gpu


def pool(B=4, wide=4, n_blocks=20):
    p = Pool(B, wide, n_blocks)
    p.append([70, 130, 64] + [3] * (B - 3), 264 + 3 * (B - 3))
    p.free([0])
    return p


@pytest.mark.parametrize("length", [-1, 4 * 64 + 1, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("B,n_blocks", [(4, 20), (700, 9000)])  # (one CTA, and a cluster)
def test_compact_with_a_bad_length_changes_nothing(B, n_blocks, length):
    """A sequence that holds a page which would move, and whose length is out of range."""
    p = pool(B, 4, n_blocks)
    assert p.copy().compact()[0], "there is something to move"
    for b in (1, B - 1):
        q = p.copy()
        q.lens[b] = length
        d = Dev(q)
        moves = torch.full((n_blocks // 2, 2), -9, dtype=torch.int32, device="cuda")
        n_moves, live = (torch.full((1,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
        pkg.kv8_pages_compact(*d.state(), moves=moves, n_moves=n_moves, n_live=live, err_word=d.err)
        d.same(q, 1)
        assert int(n_moves[0]) == 0 and int(live[0]) == n_blocks and (moves == -9).all()
        d.lens[b] = int(p.lens[b])  # mended, the call does what it does
        want = p.copy()
        assert d.compact() == want.compact()
        d.same(want)


@pytest.mark.parametrize("length", [-1, 4 * 64 + 1, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("B", [4, 3000])  # (one CTA, and a cluster)
def test_free_with_a_bad_length_changes_nothing(B, length):
    """A row's entries behind the held ones may say anything, another sequence's pages among them:
    with a length that cannot be, none of them is given back, nor any other sequence of the list."""
    p = pool(B, 4, B + 60)
    p.table[2, 1:] = p.table[1, :3]  # (left from an earlier use of the row)
    q = p.copy()
    q.lens[2] = length
    everyone = list(range(B))
    for seq in ([2], [1, 2, 3], everyone):
        d = Dev(q)
        d.free(seq)
        d.same(q, 1)
    d = Dev(p)
    d.free(everyone)
    assert int(d.err[0]) == 0 and not d.refs.any() and not d.lens.any()
