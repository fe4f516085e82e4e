"""Attention with a sliding window and first tokens that stay visible, against its definition in 64 bits."""
import math

import pytest
import torch

import fp8_mla_latent_gb300 as pkg
from chunk_helpers import DL, PAGE, SM_SCALE
from more_helpers import WindowCase

pytestmark = pytest.mark.gpu


def run(c, lse=True, ws=None, **kw):
    rows = c.q_lat.shape[0]
    if ws is None:
        ws = pkg.alloc_workspace(pkg.mla_absorb_window_fp8_batch_workspace_size(len(c.nq), c.H, rows, c.max_blocks,
                                                                                c.window, c.sinks))
    out = torch.full((rows, c.H, DL), 7.0, dtype=torch.bfloat16, device="cuda")
    l = torch.full((rows, c.H), 7.0, device="cuda") if lse else None
    got = pkg.mla_absorb_window_fp8_batch(*c.args(), SM_SCALE, c.window, c.sinks, out=out, lse=l, workspace=ws, **kw)
    assert got is out
    return out, l, pkg.kv8_workspace_error(ws)


def check(c, lse=True):
    out, l, err = run(c, lse)
    assert err == 0
    c.check(out, l)
    assert (out[sum(c.nq):] == 7).all() and (l is None or (l[sum(c.nq):] == 7).all()), "rows behind the last"
    return out, l


LENS = [1, 2, 63, 64, 65, 127, 128, 129, 192, 257, 300, 700]
NQ = [1, 2, 5, 1, 65, 3, 4, 129, 2, 1, 7, 33]


@pytest.mark.parametrize("sinks", [0, 1, 64, 70])
@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 200])
def test_windows_around_pages_and_tiles(window, sinks):
    check(WindowCase(16, NQ, [max(t, n) for t, n in zip(LENS, NQ)], window, sinks, seed=window + sinks, pad=3))


@pytest.mark.parametrize("H", [1, 3, 20, 128, 130])
def test_head_counts(H):
    check(WindowCase(H, NQ, [max(t, n) for t, n in zip(LENS, NQ)], 100, 4, seed=H))


@pytest.mark.parametrize("H,nq,T,window,sinks", [
    (128, 1, 4096, 1000, 64), (4, 1, 700, 128, 4), (16, 1, 9000, 4096, 4), (128, 130, 1500, 256, 128),
    (1, 700, 900, 33, 5), (1024, 2, 400, 70, 0), (128, 4, 3000, 1, 0), (20, 333, 1999, 777, 300), (16, 40, 3000, 8, 2000)])
def test_one_sequence(H, nq, T, window, sinks):
    check(WindowCase(H, [nq], [T], window, sinks, seed=T))


def test_many_single_tokens():
    lens = [1 + (37 * i) % 900 for i in range(200)]
    check(WindowCase(16, [1] * 200, lens, 150, 4, seed=5))


FEW_LENS = [1, 2, 63, 64, 65, 127, 128, 129, 192, 257, 300, 700, 1500, 2, 640, 3]


@pytest.mark.parametrize("sinks", [0, 1, 64, 70])
@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 200, 5000])
def test_single_tokens_around_pages_and_tiles(window, sinks):
    check(WindowCase(16, [1] * 16, FEW_LENS, window, sinks, seed=window + sinks, pad=3))


@pytest.mark.parametrize("H", [1, 3, 4, 8, 15, 16, 17, 20, 32])
def test_few_rows_a_sequence(H):
    """One to three tokens, some sequences with none, one with many: on average at most 32 rows."""
    nq = [1, 1, 0, 1, 0, 1, 1, 0, 1, 1, 0, 1, 1, 0, 3, 1]
    check(WindowCase(H, nq, FEW_LENS, 130, 5, seed=H, pad=2))
    check(WindowCase(H, [0] * 14 + [9, 0], FEW_LENS, 400, 70, seed=H + 1))


@pytest.mark.parametrize("H,T,window,sinks", [(16, 40000, 30000, 4), (1, 40000, 40000, 0), (4, 256, 100, 2), (32, 9000, 8000, 640),
                                              (16, 1, 1, 0), (20, 5000, 1, 0), (8, 20000, 64, 9000)])
def test_one_token(H, T, window, sinks):
    check(WindowCase(H, [1], [T], window, sinks, seed=T + H))


@pytest.mark.parametrize("B,T", [(300, 500), (152, 1000), (40, 3000)])
def test_single_tokens_of_many_sequences_in_ranges_that_cross_them(B, T):
    lens = [1 + (T * 7 * i) % T for i in range(B)]
    check(WindowCase(16, [1] * B, lens, T // 2, 4, seed=B))


@pytest.mark.parametrize("H,nq", [(128, 1), (100, 1), (65, 1), (33, 3), (20, 6), (4, 30)])
@pytest.mark.parametrize("window,sinks", [(70, 3), (1, 0), (300, 130)])
def test_65_to_128_rows_a_sequence(H, nq, window, sinks):
    """Row tiles of 128; more or fewer rows and none in some sequences."""
    n = [nq] * 96
    n[5:50:9] = [0] * len(n[5:50:9])
    n[3], n[70] = 2 * nq, 2 * nq
    lens = [max(n[i], 1 + (61 * i) % 450) for i in range(96)]
    check(WindowCase(H, n, lens, window, sinks, seed=H + window, pad=2))


def test_128_heads_in_ranges_that_cross_sequences():
    check(WindowCase(128, [1] * 40, [1500 + 37 * i for i in range(40)], 1000, 64, seed=40))
    check(WindowCase(128, [1, 1], [9000, 8500], 7000, 4, seed=41))


def test_keys_out_of_sight_never_reach_a_row_of_65_to_128():
    c = WindowCase(128, [1] * 70, [300 + i for i in range(70)], 100, 5, seed=42)
    clean, clean_l, err = run(c)
    for b in (0, 30, 69):
        for at in (5, 63, c.lens_list[b] - 101):
            slot = int(c.slots[b][at])
            c.codes[slot] = 0x7F
            c.codes[slot, ::2] = 0xFF
            c.scales[slot] = math.nan
    out, l, err = run(c)
    assert err == 0 and torch.equal(out, clean) and torch.equal(l, clean_l)
    c.codes[int(c.slots[7][250])] = 0x7F
    out, l, err = run(c)
    hit = torch.arange(70, device="cuda") == 7
    assert torch.isnan(out[hit]).all() and torch.isnan(l[hit]).all() and torch.equal(out[~hit], clean[~hit])


def test_few_rows_that_see_nothing_and_queries_with_nan():
    c = WindowCase(4, [3, 1, 4, 1], [2, 1, 0, 300], 40, 2, seed=17)
    out, l = check(c)
    c.q_lat[8, 2, 100] = math.nan
    c.q_rope[3, 1, 3] = math.inf
    got, gl, _ = run(c)
    hit = torch.zeros(9, 4, dtype=torch.bool, device="cuda")
    hit[8, 2] = hit[3, 1] = True
    assert torch.isnan(got[hit]).all() and torch.isnan(gl[hit]).all()
    assert torch.equal(got[~hit], out[~hit]) and torch.equal(gl[~hit], l[~hit])


def test_keys_out_of_sight_never_reach_a_single_token():
    """NaN behind a token's window, in pages that its window shares and in the last page behind its end."""
    c = WindowCase(16, [1, 1, 1], [700, 333, 90], 100, 5, seed=18)
    clean, clean_l, _ = run(c)
    for b, at in ((0, 599), (0, 5), (0, 63), (1, 232), (1, 10)):
        slot = int(c.slots[b][at])
        c.codes[slot] = 0x7F
        c.codes[slot, ::2] = 0xFF
        c.scales[slot] = math.nan
    out, l, err = run(c)
    assert err == 0 and torch.equal(out, clean) and torch.equal(l, clean_l)
    c.codes[int(c.slots[2][80])] = 0x7F
    out, l, err = run(c)
    assert torch.isnan(out[2]).all() and torch.isnan(l[2]).all() and torch.equal(out[:2], clean[:2])


def test_row_scales_of_every_size_and_dominant_keys_for_single_tokens():
    def rows(b, t, g):
        x = torch.randn((t, 576), generator=g) * 2.0 ** torch.randint(-4, 5, (t, 1), generator=g)
        x[::17] = 0
        x[5::31] *= 1e-38
        if b == 1:
            x = 0.3 * torch.randn((t, 576), generator=g) + 0.5
            x[2] *= 8
            x[t - 40] *= 6
        return x
    c = WindowCase(16, [1, 1, 1], [700, 1500, 260], 600, 4, seed=19, rows=rows)
    c.q_lat[1] = (c.q_lat[1].float() * 0.4 + 0.3).bfloat16()
    c.q_lat[2] *= 1e-30
    c.q_rope[2] *= 1e-30
    check(c)


def test_mixed_batch_with_sequences_that_have_no_query_or_no_token():
    check(WindowCase(16, [0, 3, 0, 1, 40, 0], [70, 500, 0, 1, 290, 64], 50, 3, seed=6, pad=9))


@pytest.mark.parametrize("H", [1, 16, 128])
def test_rows_that_see_nothing(H):
    """More queries than cached tokens: the first rows see no key; a sequence without a token."""
    check(WindowCase(H, [5, 3, 2, 170], [2, 0, 1, 103], 40, 2, seed=7))


def test_no_lse():
    check(WindowCase(64, [3, 9], [400, 700], 100, 10, seed=8), lse=False)


@pytest.mark.parametrize("window,sinks", [(5000, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1)])
def test_a_window_or_sinks_over_everything_give_the_bits_of_chunk_attention(window, sinks):
    c = WindowCase(16, [3, 40, 1], [300, 700, 90], window, sinks, seed=9)
    out, l, err = run(c)
    assert err == 0
    want_l = torch.empty_like(l)
    want = pkg.mla_absorb_chunk_fp8_batch(*c.args(), SM_SCALE, lse=want_l)
    assert torch.equal(out, want) and torch.equal(l, want_l)


def unseen_pages(c):
    for b in range(len(c.nq)):
        see = c.sees(b).any(0)
        for k in range((c.lens_list[b] + PAGE - 1) // PAGE):
            if not see[k * PAGE: (k + 1) * PAGE].any():
                yield b, k


def test_pages_out_of_sight_need_not_be_there():
    """Entries of pages that no row sees are free for anything, the pages hold NaN: no error, the same bits."""
    c = WindowCase(16, [1, 30, 200, 2], [900, 1500, 1300, 70], 130, 70, seed=10)
    want, want_l = check(c)
    n = 0
    for i, (b, k) in enumerate(unseen_pages(c)):
        page = int(c.table[b, k])
        c.codes[page * PAGE: (page + 1) * PAGE] = 0x7F
        c.scales[page * PAGE: (page + 1) * PAGE] = math.nan
        c.table[b, k] = (-1, 2 ** 31 - 1, -(2 ** 31), 10 ** 6)[i % 4]
        n += 1
    assert n > 20
    out, l, err = run(c)
    assert err == 0 and torch.equal(out, want) and torch.equal(l, want_l)


def test_keys_out_of_sight_never_reach_a_row():
    """NaN codes and scales behind a row's window and after it: rows that do not see them keep their
    bits, those that see them are NaN."""
    c = WindowCase(16, [60, 130], [400, 330], 90, 5, seed=11)
    clean, clean_l, _ = run(c)
    for b, at in ((0, 260), (0, 380), (1, 215), (1, 3)):
        slot = int(c.slots[b][at])
        c.codes[slot] = 0x7F
        c.codes[slot, ::2] = 0xFF
        c.scales[slot] = math.nan
    out, l, err = run(c)
    assert err == 0
    for b, bad in ((0, (260, 380)), (1, (215, 3))):
        first, n = int(c.start[b]), c.nq[b]
        hit = c.sees(b)[:, list(bad)].any(1)
        assert hit.any() and (b == 1 or not hit.all())
        got, gl = out[first: first + n], l[first: first + n]
        assert torch.equal(got[~hit], clean[first: first + n][~hit]) and torch.equal(gl[~hit], clean_l[first: first + n][~hit])
        assert torch.isnan(got[hit]).all() and torch.isnan(gl[hit]).all()


def test_a_bad_page_in_sight_is_told_and_left_out():
    c = WindowCase(16, [4], [600], 200, 3, seed=12)
    c.table[0, 8] = 10 ** 6  # tokens 512 .. 575
    out, l, err = run(c)
    assert err == -5
    keep = torch.ones(600, dtype=torch.bool)
    keep[512:576] = False
    c.check(out, l, keep=[keep])


@pytest.mark.parametrize("H,nq", [(16, 1), (128, 1), (16, 40)])
def test_lengths_that_cannot_be_are_told_and_clamped(H, nq):
    """A length over the table's room and one below 0, beside good ones."""
    B = 70
    c = WindowCase(H, [nq] * B, [300] * B, 100, 4, seed=43)
    check(c)
    c.lens[3], c.lens[5] = 10 ** 6, -7
    out, l, err = run(c)
    assert err == -5
    for b in set(range(B)) - {3, 5}:
        ref, ref_l, tol, tol_l = c.reference(b)
        rows = slice(b * nq, (b + 1) * nq)
        assert ((out[rows].double() - ref).abs() <= tol).all() and ((l[rows] - ref_l).abs() <= tol_l).all(), b
    assert (out[5 * nq: 6 * nq] == 0).all() and torch.isneginf(l[5 * nq: 6 * nq]).all()


@pytest.mark.parametrize("H,n", [(1, 3), (16, 1), (20, 5), (128, 1), (128, 70), (200, 40)])
def test_query_ranges_that_overlap_are_told_and_stay_in_the_workspace(H, n):
    """Every second sequence has the same n tokens, far more in all than the arrays hold."""
    B = 90
    c = WindowCase(H, [n] + [0] * (B - 1), [400] * B, 200, 4, seed=48)
    want, _ = check(c)
    c.start.copy_(torch.tensor([0, n] * (B // 2) + [0]))
    size = pkg.mla_absorb_window_fp8_batch_workspace_size(B, H, n, c.max_blocks, 200, 4)
    room = torch.full((size + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((n, H, DL), 7.0, dtype=torch.bfloat16, device="cuda")
    pkg.mla_absorb_window_fp8_batch(*c.args(), SM_SCALE, 200, 4, out=out, workspace=room[:size])
    assert pkg.kv8_workspace_error(room) == -5
    assert (room[size:] == 0xA5).all()
    c.start.copy_(torch.tensor([0] + [n] * B))
    assert torch.equal(run(c)[0], want)


@pytest.mark.parametrize("H", [16, 200])
def test_lengths_near_2_to_the_31(H):
    """The longest table there is, of whose pages only the last four, the window's, are there."""
    mb, k = (1 << 25) - 1, 4
    c = WindowCase(H, [1], [k * PAGE], 200, 0, seed=45)
    table = torch.full((1, mb), -1, dtype=torch.int32, device="cuda")
    table[0, mb - k:] = c.table[0, :k]
    got_l = torch.empty(1, H, device="cuda")
    ws = pkg.alloc_workspace(pkg.mla_absorb_window_fp8_batch_workspace_size(1, H, 1, mb, 200, 0))
    got = pkg.mla_absorb_window_fp8_batch(c.q_lat, c.q_rope, c.codes, c.scales, table,
                                          torch.tensor([mb * PAGE], dtype=torch.int32, device="cuda"), c.start, SM_SCALE,
                                          200, 0, lse=got_l, workspace=ws)
    assert pkg.kv8_workspace_error(ws) == 0
    ref, ref_l, tol, tol_l = c.reference(0)
    assert ((got.double() - ref).abs() <= tol).all() and ((got_l - ref_l).abs() <= tol_l).all()


@pytest.mark.parametrize("H", [1, 65])
def test_more_sequences_than_the_plan_keeps_near(H):
    lens = [1 + (37 * i) % 150 for i in range(4200)]
    check(WindowCase(H, [1] * 4200, lens, 70, 2, seed=46), lse=False)


def test_strided_queries():
    c = WindowCase(20, [7, 3], [190, 401], 64, 4, seed=14)
    want, want_l = check(c)
    both = torch.cat([c.q_lat, c.q_rope], -1)
    hm = both.transpose(0, 1).contiguous().transpose(0, 1)  # heads outermost in memory
    c.q_lat, c.q_rope = hm[..., :DL], hm[..., DL:]
    out, l, _ = run(c)
    assert torch.equal(out, want) and torch.equal(l, want_l)


@pytest.mark.parametrize("H,nq", [(16, [1] * 9), (20, [1, 0, 2, 1, 1]), (128, [1] * 70), (16, [40, 3])])
def test_queries_of_wider_arrays_and_one_head_for_all(H, nq):
    """In each of the kernels: rows of a wider array, heads outermost, and one head's query for every head."""
    c = WindowCase(H, nq, [500 + 3 * i for i in range(len(nq))], 200, 4, seed=49)
    want, want_l = check(c)
    wide = torch.full((sum(nq) + 2, H + 1, 640), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[1:-1, 1:, 32:608] = torch.cat([c.q_lat, c.q_rope], -1)
    c.q_lat, c.q_rope = wide[1:-1, 1:, 32:544], wide[1:-1, 1:, 544:608]
    for _ in range(2):
        out, l, err = run(c)
        assert err == 0 and torch.equal(out, want) and torch.equal(l, want_l)
        wide = wide.transpose(0, 1).contiguous().transpose(0, 1)
        c.q_lat, c.q_rope = wide[1:-1, 1:, 32:544], wide[1:-1, 1:, 544:608]
    c.q_lat, c.q_rope = c.q_lat[:, :1].expand(-1, H, -1), c.q_rope[:, :1].expand(-1, H, -1)
    check(c)


def test_workspaces_of_the_calls_own_on_a_given_stream_and_in_a_graph():
    c = WindowCase(16, [1] * 40, [900 + 7 * i for i in range(40)], 600, 4, seed=50)
    want, _ = check(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [pkg.mla_absorb_window_fp8_batch(*c.args(), SM_SCALE, 600, 4, stream=s) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    outs = [torch.zeros_like(want) for _ in range(2)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for o in outs:
            pkg.mla_absorb_window_fp8_batch(*c.args(), SM_SCALE, 600, 4, out=o)
    for _ in range(3):
        junk = [torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(20)]
        for o in outs:
            o.zero_()
        g.replay()
        junk += [torch.full((1 << 22,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(20)]
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
        assert torch.equal(pkg.mla_absorb_window_fp8_batch(*c.args(), SM_SCALE, 600, 4), want)


def test_dominant_keys_behind_the_window_and_among_the_first_tokens():
    """The rows' largest keys leave the window in the middle of the chunk; the first tokens' are larger still."""
    def rows(b, t, g):
        x = 0.3 * torch.randn((t, 576), generator=g) + 0.5
        x[2] *= 8
        x[500:520] *= 5
        return x
    c = WindowCase(32, [200], [700], 120, 4, seed=13, rows=rows)
    c.q_lat.copy_((c.q_lat.float() * 0.4 + 0.3).bfloat16())
    check(c)


def test_captured_and_replayed_on_another_stream():
    c = WindowCase(16, [3, 1, 70], [900, 65, 400], 100, 4, seed=15)
    want, want_l = check(c)
    ws = [pkg.alloc_workspace(pkg.mla_absorb_window_fp8_batch_workspace_size(3, 16, 74, c.max_blocks, 100, 4)) for _ in range(2)]
    out, l = torch.zeros_like(want), torch.zeros_like(want_l)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkg.mla_absorb_window_fp8_batch(*c.args(), SM_SCALE, 100, 4, out=out, lse=l, workspace=ws[0])
    s = torch.cuda.Stream()
    for _ in range(3):
        out.zero_()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g.replay()
        other = pkg.mla_absorb_window_fp8_batch(*c.args(), SM_SCALE, 100, 4, workspace=ws[1])
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(out, want) and torch.equal(l, want_l) and torch.equal(other, want)


@pytest.mark.parametrize("H,nq", [(16, 1), (32, 1), (128, 1), (128, 5)])
def test_two_calls_at_once(H, nq):
    c = WindowCase(H, [nq] * 70, [600 + 5 * i for i in range(70)], 300, 4, seed=47)
    want, _ = check(c)
    ws = [pkg.alloc_workspace(pkg.mla_absorb_window_fp8_batch_workspace_size(70, H, 70 * nq, c.max_blocks, 300, 4)) for _ in range(2)]
    outs, streams = [torch.zeros_like(want) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for w, o, s in zip(ws, outs, streams):
            with torch.cuda.stream(s):
                o.zero_()
                pkg.mla_absorb_window_fp8_batch(*c.args(), SM_SCALE, 300, 4, out=o, workspace=w)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


@pytest.mark.parametrize("H,B", [(16, 2), (200, 2), (128, 70)])
def test_far_pages(H, B):
    """Cache slots whose bytes lie behind 2^31 and 2^32, in each of the kernels."""
    c = WindowCase(H, [2 if H == 200 else 1] * B, [400 - b for b in range(B)], 150, 4, seed=16)
    n_blocks = 2 ** 32 // (PAGE * 576) + 800
    want, want_l = check(c)
    codes = torch.full((n_blocks * PAGE, 576), 0x7F, dtype=torch.uint8, device="cuda")
    scales = torch.full((n_blocks * PAGE, 2), math.nan, device="cuda")
    k = c.codes.shape[0]
    codes[-k:], scales[-k:] = c.codes, c.scales
    c.table = torch.where(c.table >= 0, c.table + (n_blocks - k // PAGE), c.table)
    c.codes, c.scales = codes, scales
    out, l, err = run(c)
    assert err == 0 and torch.equal(out, want) and torch.equal(l, want_l)


@pytest.mark.parametrize("H,n,times,more", [(1, 3, 60, 4), (16, 60, 18, 40), (20, 30, 20, 70), (128, 20, 40, 30), (128, 60, 18, 2),
                                            (200, 40, 30, 3)])
def test_rows_that_no_other_range_touches_behind_ranges_that_overlap(H, n, times, more):
    """The same n rows named again and again, then ranges of their own: these are computed as in any call, although
    there are more row tiles than of ranges that are apart."""
    B = 2 * times - 1 + more  # (the n rows' sequences, with ranges that turn back between them, then the others)
    nq = [n] + [0] * (2 * times - 2) + [1 + b % 2 for b in range(more)]
    c = WindowCase(H, nq, [400 + b % 7 for b in range(B)], 200, 4, seed=51)
    check(c)
    c.start[: 2 * times] = torch.tensor([0, n] * times)
    size = pkg.mla_absorb_window_fp8_batch_workspace_size(B, H, sum(nq), c.max_blocks, 200, 4)
    room = torch.full((size + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((sum(nq), H, DL), 7.0, dtype=torch.bfloat16, device="cuda")
    l = torch.full((sum(nq), H), 7.0, device="cuda")
    pkg.mla_absorb_window_fp8_batch(*c.args(), SM_SCALE, 200, 4, out=out, lse=l, workspace=room[:size])
    assert pkg.kv8_workspace_error(room) == -5 and (room[size:] == 0xA5).all()
    for b in range(2 * times - 1, B):
        ref, ref_l, tol, tol_l = c.reference(b)
        rows = slice(int(c.start[b]), int(c.start[b + 1]))
        assert ((out[rows].double() - ref).abs() <= tol).all() and ((l[rows] - ref_l).abs() <= tol_l).all(), b
