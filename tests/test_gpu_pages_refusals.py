"""Page calls on a table whose lengths cannot be: compact and free change nothing.  And a captured
serving step against an eager one."""
import numpy as np
import pytest
import torch

import fp8_mla_latent_gb300 as pkg
from chunk_helpers import D, DL, DR, SM_SCALE
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


def test_a_captured_step_gives_what_an_eager_one_gives():
    """append, quantize, attention in one graph; after every replay the new rows of every sequence lie in
    its slots, and the attention is that of an eager call on the same state, bit for bit."""
    H, mb, nb, B = 16, 4, 12, 3
    p = Pool(B, mb, nb)
    p.append([63, 10, 64], 137)
    d = Dev(p)
    g = torch.Generator(device="cuda").manual_seed(6)
    codes = torch.randint(0, 0x7F, (nb * 64, D), dtype=torch.uint8, device="cuda", generator=g)
    scales = 0.002 + 0.003 * torch.rand((nb * 64, 2), device="cuda", generator=g)
    rows = torch.randn((B, D), device="cuda", generator=g)
    n_new = torch.ones(B, dtype=torch.int32, device="cuda")
    q_start = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    slots = torch.zeros(B, dtype=torch.int64, device="cuda")
    ql = torch.randn((B, H, DL), device="cuda", generator=g).bfloat16()
    qr = torch.randn((B, H, DR), device="cuda", generator=g).bfloat16()
    out = torch.empty((B, H, DL), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((B, H), device="cuda")
    ws = pkg.alloc_workspace(pkg.mla_absorb_chunk_fp8_batch_workspace_size(B, H, B, mb))

    def step():
        pkg.kv8_pages_append(*d.state(), n_new, q_start=q_start, dst_slot=slots, err_word=d.err)
        pkg.kv8_quantize_rows(rows, codes, scales, dst_slot=slots)
        pkg.mla_absorb_chunk_fp8_batch(ql, qr, codes, scales, d.table, d.lens, q_start, SM_SCALE, out=out, lse=lse,
                                       workspace=ws)

    step()
    p.append([1, 1, 1], 3)
    d.same(p)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(5):
        rows.copy_(torch.randn((B, D), device="cuda", generator=g) * (1 + i))
        ql.copy_(torch.randn((B, H, DL), device="cuda", generator=g).bfloat16())
        out.fill_(float("nan"))
        lse.fill_(float("nan"))
        graph.replay()
        _, s, _ = p.append([1, 1, 1], 3)
        d.same(p)
        assert np.array_equal(slots.cpu().numpy(), s)
        c2, s2 = torch.zeros_like(codes[:B]), torch.zeros_like(scales[:B])
        pkg.kv8_quantize_rows(rows, c2, s2)
        assert torch.equal(codes[slots], c2) and torch.equal(scales[slots], s2)
        lse2 = torch.empty_like(lse)
        want = pkg.mla_absorb_chunk_fp8_batch(ql, qr, codes, scales, d.table, d.lens,
                                              torch.arange(B + 1, dtype=torch.int32, device="cuda"), SM_SCALE, lse=lse2)
        assert torch.equal(out, want) and torch.equal(lse, lse2)
        assert torch.isfinite(lse).all() and pkg.kv8_workspace_error(ws) == 0
