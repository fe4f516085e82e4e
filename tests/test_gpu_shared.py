"""Attention of sequences that share prefixes, against its definition in 64 bits."""
import math

import pytest
import torch

import fp8_mla_latent_gb300 as pkg
from chunk_helpers import DL, PAGE, SM_SCALE
from more_helpers import SharedCase

pytestmark = pytest.mark.gpu


def workspace(c):
    return pkg.alloc_workspace(pkg.mla_absorb_shared_fp8_batch_workspace_size(
        len(c.nq), c.H, c.q_lat.shape[0], c.max_blocks, c.shared_len.numel()))


ALWAYS, AUTO = pkg.KV8_SHARE_ALWAYS, pkg.KV8_SHARE_AUTO


def run(c, causal=True, lse=True, ws=None, share=ALWAYS):
    rows = c.q_lat.shape[0]
    ws = workspace(c) if ws is None else ws
    out = torch.full((rows, c.H, DL), 7.0, dtype=torch.bfloat16, device="cuda")
    l = torch.full((rows, c.H), 7.0, device="cuda") if lse else None
    got = pkg.mla_absorb_shared_fp8_batch(*c.args(), SM_SCALE, c.group_start, c.shared_len, causal=causal, out=out,
                                          lse=l, workspace=ws, share=share)
    assert got is out
    return out, l, pkg.kv8_workspace_error(ws)


def check(c, causal=True, lse=True):
    """Where every prefix that can be is shared, and as the call decides by itself."""
    for share in (AUTO, ALWAYS):
        out, l, err = run(c, causal, lse, share=share)
        assert err == 0
        c.check(out, l, causal)
        assert (out[sum(c.nq):] == 7).all() and (l is None or (l[sum(c.nq):] == 7).all()), "rows behind the last"
    return out, l


def run_with(c, shared_len, group_start=None):
    old = c.shared_len, c.group_start
    c.shared_len, c.group_start = shared_len, old[1] if group_start is None else group_start
    try:
        return run(c)
    finally:
        c.shared_len, c.group_start = old


def check_with(c, shared_len):
    out, l, err = run_with(c, shared_len)
    assert err == 0
    c.check(out, l)
    return out, l


def chunk(c, causal=True):
    l = torch.full(c.q_lat.shape[:2], 7.0, device="cuda")
    out = torch.full((*c.q_lat.shape[:2], DL), 7.0, dtype=torch.bfloat16, device="cuda")
    pkg.mla_absorb_chunk_fp8_batch(*c.args(), SM_SCALE, causal=causal, out=out, lse=l)
    return out, l


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H", [1, 3, 16, 64, 128, 130])
def test_one_group(H, causal):
    nq = [1, 1, 3, 1, 2, 1, 1, 5, 1, 1, 1, 1]
    lens = [900 + (97 * i) % 300 for i in range(12)]
    check(SharedCase(H, nq, lens, [12], [850], seed=H, pad=3), causal)


@pytest.mark.parametrize("shared", [0, 1, 63, 64, 65, 127, 128, 640, 700, 704, 5000])
def test_shared_lengths(shared):
    """Around pages and tiles, and over the members' lengths; the shortest rows see no more than the prefix."""
    lens = [704, 705, 768, 1000, 704, 720, 1500, 710]
    check(SharedCase(16, [1] * 8, lens, [8], [shared], seed=shared))


@pytest.mark.parametrize("H", [4, 20, 128])
def test_several_groups_and_sequences_in_none(H):
    sizes, shared = [3, 1, 0, 7, 9], [700, 900, 50, 1999, 1300]
    lens = [750, 800, 702, 1000, *[2000 + 31 * i for i in range(7)], *[1301 + 64 * i for i in range(9)], 40, 300]
    nq = [1 + (5 * i) % 4 for i in range(len(lens))]
    check(SharedCase(H, nq, lens, sizes, shared, seed=H + 1, pad=5))


def test_members_without_queries_or_tokens():
    """The first member has neither: the prefix is read through the row of one that has queries."""
    c = SharedCase(16, [0, 2, 0, 1, 1, 1, 2, 1], [0, 900, 70, 880, 900, 1000, 860, 990], [8], [850], seed=2)
    check(c)


def test_a_prefix_that_some_row_does_not_see():
    """A chunk that begins inside the prefix: what every row of the group sees is computed once, no more."""
    check(SharedCase(16, [1, 1, 300, 1, 1, 1], [900, 910, 1000, 920, 930, 940], [6], [850], seed=3))


def test_prompts_that_fill_their_row_tiles():
    check(SharedCase(128, [130, 70, 40], [700, 800, 900], [3], [600], seed=4))


def test_long_prefix_over_all_clusters():
    check(SharedCase(128, [1, 1, 2], [9000, 9100, 9050], [3], [8990], seed=5))


def test_rows_that_see_nothing():
    check(SharedCase(16, [5, 1, 1, 3], [2, 900, 900, 0], [4], [850], seed=6))


@pytest.mark.parametrize("H", [1, 128])
def test_more_sequences_than_the_plans_keep_near(H):
    lens = [65 + (37 * i) % 60 for i in range(1400)]
    check(SharedCase(H, [1] * 1400, lens, [7] * 200, [64] * 200, seed=32), lse=False)


def test_many_sequences_in_many_groups():
    lens = [500 + (37 * i) % 300 for i in range(300)]
    check(SharedCase(4, [1] * 300, lens, [5] * 60, [490] * 60, seed=7), lse=False)


@pytest.mark.parametrize("H", [1, 4, 16, 17, 20, 32, 64])
def test_single_tokens_behind_a_long_prefix(H):
    """Prefix and rest are different kernels' parts, cut by the borders of either's ranges."""
    lens = [5000 + (613 * i) % 1500 for i in range(40)]
    check(SharedCase(H, [1] * 40, lens, [25, 15], [4999, 3000], seed=H, pad=2))


@pytest.mark.parametrize("causal", [True, False])
def test_few_rows_in_groups_of_every_kind(causal):
    """Groups that share and that do not, sequences without queries, some with several tokens, some in none."""
    nq = [1, 0, 2, 1, 1, 1, 0, 0, 3, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 0, 4, 1, 1]
    lens = [800, 900, 801, 1000, 850, 900, 640, 0, 700, 70, 64, 1, 128] + [2000 + 65 * i for i in range(11)]
    check(SharedCase(16, nq, lens, [5, 4, 4, 8], [790, 640, 60, 1990], seed=30, pad=7), causal)


def test_a_prefix_is_computed_once():
    """The other members' entries for it are not looked up: wherever it can be, and where it is found to pay."""
    for c, share in ((SharedCase(16, [1] * 16, [2000] * 16, [16], [1984], seed=8), ALWAYS),
                     (SharedCase(128, [1] * 16, [2000] * 16, [16], [1984], seed=8), ALWAYS),
                     (SharedCase(64, [1] * 24, [9000] * 24, [24], [8960], seed=8, rows=lambda b, t, g: torch.rand((t, 576)) - 0.5), AUTO)):
        want, want_l, err = run(c, share=share)
        assert err == 0
        c.table[1:, : int(c.shared_len[0]) // PAGE] = 2 ** 30
        out, l, err = run(c, share=share)
        assert err == 0 and torch.equal(out, want) and torch.equal(l, want_l)


def test_a_short_prefix_is_left_where_it_is():
    """Too little to pay for a kernel more: the members' own entries are read."""
    c = SharedCase(16, [1] * 6, [300] * 6, [6], [256], seed=31)
    c.table[3, 1] = 2 ** 30
    assert run(c, share=AUTO)[2] == -5 and run(c, share=ALWAYS)[2] == 0


@pytest.mark.parametrize("groups", [[0, 3, 2, 8], [-1, 4, 8, 8], [0, 4, 8, 9], [5, 4, 3, 2]])
def test_groups_that_cannot_be_are_told_and_share_nothing(groups):
    c = SharedCase(16, [1] * 8, [900] * 8, [8], [850], seed=9)
    c.group_start = torch.zeros(4, dtype=torch.int32, device="cuda")
    c.shared_len = torch.zeros(3, dtype=torch.int32, device="cuda")
    want = check(c)
    c.group_start = torch.tensor(groups, dtype=torch.int32, device="cuda")
    c.shared_len = torch.tensor([850] * 3, dtype=torch.int32, device="cuda")
    out, l, err = run(c)
    assert err == -5 and torch.equal(out, want[0]) and torch.equal(l, want[1])


@pytest.mark.parametrize("B", [2, 8])
def test_a_negative_length_is_told_and_shares_nothing(B):
    c = SharedCase(4, [1] * B, [900] * B, [B], [850], seed=10)
    shared = c.shared_len.clone()
    want = check_with(c, shared * 0)
    out, l, err = run_with(c, shared * 0 - 5)
    assert err == -5 and torch.equal(out, want[0]) and torch.equal(l, want[1])
    assert run_with(c, shared, c.group_start + 1)[2] == -5


def test_without_groups_the_bits_of_chunk_attention():
    c = SharedCase(128, [1, 40, 3], [900, 300, 70], [], [], seed=11, pad=4)
    out, l, err = run(c)
    want = chunk(c)
    assert err == 0 and torch.equal(out, want[0]) and torch.equal(l, want[1])


def test_a_bad_query_range_is_told():
    """Its sequence has no query, the group shares nothing, and the others are right."""
    c = SharedCase(16, [1] * 6, [900] * 6, [6], [850], seed=12)
    c.start[3] = 10 ** 6
    out, l, err = run(c)
    assert err == -5
    c.start[3] = 3
    for b in (0, 1, 4, 5):
        ref, ref_l, tol, tol_l = c.reference(b)
        assert ((out[b: b + 1].double() - ref).abs() <= tol).all() and ((l[b: b + 1] - ref_l).abs() <= tol_l).all()


@pytest.mark.parametrize("H,n", [(16, 1), (20, 3), (128, 2), (128, 60)])
def test_query_ranges_that_overlap_are_told_and_stay_in_the_workspace(H, n):
    """Every second sequence has the same n tokens, far more in all than the arrays hold."""
    B = 90
    c = SharedCase(H, [n] + [0] * (B - 1), [400] * B, [40, 50], [320, 320], seed=34)
    want, _ = check(c)
    c.start.copy_(torch.tensor([0, n] * (B // 2) + [0]))
    size = pkg.mla_absorb_shared_fp8_batch_workspace_size(B, H, n, c.max_blocks, 2)
    for share in (AUTO, ALWAYS):
        room = torch.full((size + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
        out = torch.full((n, H, DL), 7.0, dtype=torch.bfloat16, device="cuda")
        pkg.mla_absorb_shared_fp8_batch(*c.args(), SM_SCALE, c.group_start, c.shared_len, out=out, workspace=room[:size],
                                        share=share)
        assert pkg.kv8_workspace_error(room) == -5
        assert (room[size:] == 0xA5).all()
    c.start.copy_(torch.tensor([0] + [n] * B))
    assert torch.equal(run(c)[0], want)


def test_nan_in_the_prefix_and_in_one_sequence():
    c = SharedCase(16, [1, 2, 1, 1, 1, 1, 1, 1], [1000] * 8, [8], [960], seed=13)
    clean, clean_l = check(c)
    slot = int(c.slots[2][990])
    c.codes[slot] = 0x7F
    c.scales[slot] = math.nan
    out, l, _ = run(c)
    hit = torch.zeros(9, dtype=torch.bool, device="cuda")
    hit[3] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(l[hit]).all()
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(l[~hit], clean_l[~hit])
    c.codes[int(c.slots[0][100])] = 0x7F
    out, l, _ = run(c)
    assert torch.isnan(out).all() and torch.isnan(l).all()


def test_a_dominant_token_in_the_prefix_or_behind_it():
    """Parts of very different size are joined: 2^30 and more between their maxima."""
    def rows(b, t, g):
        x = 0.3 * torch.randn((t, 576), generator=g) + 0.5
        x[5] *= 9 if b < 8 else 1
        x[t - 3] *= 1 if b < 8 else 9
        return x
    c = SharedCase(32, [1] * 16, [1000 + i for i in range(16)], [8, 8], [970, 980], seed=14, rows=rows)
    c.q_lat.copy_((c.q_lat.float() * 0.4 + 0.3).bfloat16())
    check(c)


def test_captured_and_replayed_with_lengths_that_change():
    """One captured step over 5 more tokens of every sequence, the lengths read on the device."""
    c = SharedCase(16, [1] * 10, [1100 + 7 * i for i in range(10)], [10], [1088], seed=15)
    ws, full = workspace(c), c.lens.clone()
    out, l = (torch.zeros_like(x) for x in check(c))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkg.mla_absorb_shared_fp8_batch(*c.args(), SM_SCALE, c.group_start, c.shared_len, out=out, lse=l, workspace=ws,
                                        share=ALWAYS)
    for back in (5, 3, 0):
        c.lens.copy_(full - back)
        g.replay()
        want, want_l, err = run(c)
        assert err == 0 and pkg.kv8_workspace_error(ws) == 0
        assert torch.equal(out, want) and torch.equal(l, want_l)


@pytest.mark.parametrize("H,P", [(16, 8000), (128, 4000)])
def test_two_calls_at_once_and_groups_that_change_in_a_graph(H, P):
    """Two streams with a workspace each, and a captured call (where sharing pays) whose groups are made anew."""
    B = 64
    c = SharedCase(H, [1] * B, [P + 9 + 3 * i for i in range(B)], [32, 32], [P, P], seed=33)
    want, want_l = check(c)
    ws, outs = [workspace(c) for _ in range(3)], [torch.zeros_like(want) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]

    def call(i):
        pkg.mla_absorb_shared_fp8_batch(*c.args(), SM_SCALE, c.group_start, c.shared_len, out=outs[i], workspace=ws[i])
    torch.cuda.synchronize()
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].zero_()
                call(i)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(2)
    groups = c.group_start.clone()
    for edge, P1 in ((groups, P), (torch.zeros_like(groups), P), (groups // 2, 640), (groups, P)):
        c.group_start.copy_(edge)
        c.shared_len.fill_(P1)
        outs[2].zero_()
        g.replay()
        assert pkg.kv8_workspace_error(ws[2]) == 0
        for b in (0, 15, 16, 31, 32, 63):
            ref, _, tol, _ = c.reference(b)
            assert ((outs[2][b].double() - ref[0]).abs() <= tol[0]).all(), (b, P1)
    assert torch.equal(outs[2], outs[0])
    for o in outs:
        c.check(o)


@pytest.mark.parametrize("H", [16, 128])
def test_queries_of_wider_arrays(H):
    c = SharedCase(H, [1, 2, 1, 3, 1, 1, 1, 1], [700 + 9 * i for i in range(8)], [8], [640], seed=35)
    want, want_l = check(c)
    wide = torch.full((11, H + 1, 640), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:, 32:608] = torch.cat([c.q_lat, c.q_rope], -1)
    c.q_lat, c.q_rope = wide[:, 1:, 32:544], wide[:, 1:, 544:608]
    out, l, err = run(c)
    assert err == 0 and torch.equal(out, want) and torch.equal(l, want_l)


def test_fork_append_and_attend():
    """Sequences made by the page calls: a prompt forked eight times, tokens appended, one step of attention."""
    T, n, H = 1000, 8, 16
    n_blocks, mb = 64, 24
    g = torch.Generator().manual_seed(16)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.full((n + 1, mb), -1, dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(n + 1, dtype=torch.int32, device="cuda"), torch.zeros(n_blocks, dtype=torch.int32, device="cuda")
    codes = torch.full((n_blocks * PAGE, 576), 0x7F, dtype=torch.uint8, device="cuda")
    scales = torch.full((n_blocks * PAGE, 2), math.nan, device="cuda")
    _, slots = pkg.kv8_pages_append(table, lens, refs, i32(T, *[0] * n), cap=T)
    pkg.kv8_quantize_rows(torch.randn((T, 576), generator=g).cuda(), codes, scales, slots)
    moves, n_moves = pkg.kv8_pages_fork(table, lens, refs, i32(*[0] * n), i32(*range(1, n + 1)))
    pkg.kv8_pages_copy(codes, scales, moves, n_moves)
    start, slots = pkg.kv8_pages_append(table, lens, refs, i32(0, *[2] * n), cap=2 * n)
    pkg.kv8_quantize_rows(torch.randn((2 * n, 576), generator=g).cuda(), codes, scales, slots)
    q_lat = torch.randn((2 * n, H, 512), generator=g).bfloat16().cuda()
    q_rope = torch.randn((2 * n, H, 64), generator=g).bfloat16().cuda()
    args = (q_lat, q_rope, codes, scales, table, lens, start)
    got = pkg.mla_absorb_shared_fp8_batch(*args, SM_SCALE, i32(1, n + 1), i32(T), share=ALWAYS)
    want = pkg.mla_absorb_chunk_fp8_batch(*args, SM_SCALE)
    # both are within 2^-9 + 3 2^-11 + 2^-8 (the weights, the rounding to bf16) of the exact value, up to
    # cancellation in the sum, which the largest magnitude stands for
    assert float((got.double() - want.double()).abs().max()) <= 2 * (2 ** -9 + 3 * 2 ** -11 + 2 ** -8) * float(want.abs().max())


@pytest.mark.parametrize("H,n,times,more", [(4, 60, 18, 40), (16, 60, 18, 40), (20, 30, 20, 70), (128, 60, 18, 2),
                                            (128, 200, 30, 3)])
def test_rows_that_no_other_range_touches_behind_ranges_that_overlap(H, n, times, more):
    """The same n rows named again and again, then ranges of their own, a group among them: these are in order, and
    computed as in any call, although there are more row tiles than of ranges that are apart."""
    B = 2 * times - 1 + more  # (the n rows' sequences, with ranges that turn back between them, then the others)
    nq = [n] + [0] * (2 * times - 2) + [1 + b % 2 for b in range(more)]
    c = SharedCase(H, nq, [400 + b % 7 for b in range(B)], [2 * times - 1, more], [0, 320], seed=36)
    check(c)
    c.start[: 2 * times] = torch.tensor([0, n] * times)
    for groups in ([0, 2 * times - 1, B], [0, 0, 0]):
        for share in (AUTO, ALWAYS):
            c.group_start.copy_(torch.tensor(groups))
            size = pkg.mla_absorb_shared_fp8_batch_workspace_size(B, H, sum(nq), c.max_blocks, 2)
            room = torch.full((size + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
            out, l, err = run(c, ws=room[:size], share=share)
            assert err == -5 and (room[size:] == 0xA5).all()
            for b in range(2 * times - 1, B):
                ref, ref_l, tol, tol_l = c.reference(b)
                rows = slice(int(c.start[b]), int(c.start[b + 1]))
                assert ((out[rows].double() - ref).abs() <= tol).all() and ((l[rows] - ref_l).abs() <= tol_l).all(), b


@pytest.mark.parametrize("H", [16, 128])
def test_far_pages(H):
    """Cache slots whose bytes lie behind 2^31 and 2^32, of the prefix and of what lies behind it."""
    c = SharedCase(H, [1, 2, 1, 1, 3, 1], [900 - 9 * b for b in range(6)], [6], [640], seed=37)
    n_blocks = 2 ** 32 // (PAGE * 576) + 800
    want = {share: run(c, share=share) for share in (AUTO, ALWAYS)}
    check(c)
    codes = torch.full((n_blocks * PAGE, 576), 0x7F, dtype=torch.uint8, device="cuda")
    scales = torch.full((n_blocks * PAGE, 2), math.nan, device="cuda")
    k = c.codes.shape[0]
    codes[-k:], scales[-k:] = c.codes, c.scales
    c.table = torch.where(c.table >= 0, c.table + (n_blocks - k // PAGE), c.table)
    c.codes, c.scales = codes, scales
    for share in (AUTO, ALWAYS):
        out, l, err = run(c, share=share)
        assert err == 0 and torch.equal(out, want[share][0]) and torch.equal(l, want[share][1])


@pytest.mark.parametrize("H,B", [(16, 16), (128, 2)])
@pytest.mark.parametrize("share", [AUTO, ALWAYS])
def test_lengths_near_2_to_the_31(H, B, share):
    """The longest table there is.  Of the prefix the first two pages and the last are there, of what lies behind it
    four; the others are told and left out."""
    mb = (1 << 25) - 1
    c = SharedCase(H, [1] * B, [7 * PAGE] * B, [B], [3 * PAGE], seed=38)
    table = torch.full((B, mb), -1, dtype=torch.int32, device="cuda")
    table[:, :2] = c.table[:, :2]
    table[:, mb - 5:] = c.table[:, 2:7]
    out, l = torch.empty(B, H, DL, dtype=torch.bfloat16, device="cuda"), torch.empty(B, H, device="cuda")
    ws = pkg.alloc_workspace(pkg.mla_absorb_shared_fp8_batch_workspace_size(B, H, B, mb, 1))
    pkg.mla_absorb_shared_fp8_batch(c.q_lat, c.q_rope, c.codes, c.scales, table, torch.full_like(c.lens, mb * PAGE), c.start,
                                    SM_SCALE, c.group_start, torch.full_like(c.shared_len, (mb - 4) * PAGE), out=out, lse=l,
                                    workspace=ws, share=share)
    assert pkg.kv8_workspace_error(ws) == -5
    c.check(out, l)


def test_a_group_with_room_for_its_parts_before_groups_without():
    """The rows of the second group are more than there is room for: its members read the prefix themselves.  The
    first one's is still computed once (the other members' entries for it are not looked up)."""
    c = SharedCase(128, [1, 1, 60, 60, 1, 1], [900, 950, 1000, 980, 870, 1010], [2, 2, 2], [832, 850, 800], seed=39)
    want, want_l, err = run(c)
    assert err == 0
    c.check(want, want_l)
    c.table[1, : 832 // PAGE] = 2 ** 30
    out, l, err = run(c)
    assert err == 0 and torch.equal(out, want) and torch.equal(l, want_l)
    c.table[3, 0] = 2 ** 30  # (not so the second one's)
    assert run(c)[2] == -5
