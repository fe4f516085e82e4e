"""Attention of a chunk of new tokens over the paged cache, against its definition in 64 bits."""
import math

import pytest
import torch

import fp8_mla_latent_gb300 as pkg
from chunk_helpers import D, DL, DR, PAGE, SM_SCALE, Case

pytestmark = pytest.mark.gpu


def run(c, causal=True, lse=True, **kw):
    rows = c.q_lat.shape[0]
    ws = pkg.alloc_workspace(pkg.mla_absorb_chunk_fp8_batch_workspace_size(len(c.nq), c.H, rows, c.max_blocks))
    out = torch.full((rows, c.H, DL), 7.0, dtype=torch.bfloat16, device="cuda")
    l = torch.full((rows, c.H), 7.0, device="cuda") if lse else None
    got = pkg.mla_absorb_chunk_fp8_batch(*c.args(), SM_SCALE, causal=causal, out=out, lse=l, workspace=ws, **kw)
    assert got is out
    return out, l, pkg.kv8_workspace_error(ws)


def check(c, causal=True, lse=True):
    out, l, err = run(c, causal, lse)
    assert err == 0
    worst = c.check(out, l, causal)
    assert (out[sum(c.nq):] == 7).all() and (l is None or (l[sum(c.nq):] == 7).all()), "rows behind the last"
    return worst


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H", [1, 3, 16, 64, 128, 130])
def test_lengths_around_pages_and_tiles(H, causal):
    lens = [1, 2, 63, 64, 65, 127, 128, 129, 192, 257, 300]
    nq = [1, 2, 5, 1, 65, 3, 4, 129, 2, 1, 7]
    lens = [max(t, n) for t, n in zip(lens, nq)]
    check(Case(H, nq, lens, seed=H, pad=3), causal)


@pytest.mark.parametrize("H,nq,T", [(128, 1, 4096), (128, 4, 1000), (16, 1, 2049), (4, 1, 256), (20, 33, 1999),
                                    (128, 130, 130), (1, 700, 700), (1024, 2, 150)])
def test_one_sequence(H, nq, T):
    check(Case(H, [nq], [T], seed=T))


def test_many_sequences_of_one_token():
    lens = [1 + (37 * i) % 500 for i in range(200)]
    check(Case(16, [1] * 200, lens, seed=5))


def test_mixed_batch_with_sequences_that_have_no_query_or_no_token():
    check(Case(16, [0, 3, 0, 1, 40, 0], [70, 200, 0, 1, 90, 64], seed=6, pad=9))


@pytest.mark.parametrize("H", [1, 16, 128])
def test_rows_that_see_nothing(H):
    """More queries than cached tokens: the first rows see no key; a sequence without a token."""
    check(Case(H, [5, 3, 2, 70], [2, 0, 1, 3], seed=7))


def test_no_lse():
    check(Case(64, [3, 9], [100, 400], seed=8), lse=False)


def test_keys_out_of_sight_never_reach_a_row():
    """NaN codes and scales of every kind in later tokens of the chunk: the rows before them are
    those of a cache without them, bit for bit; the rows that see them are NaN."""
    c = Case(16, [40, 130], [300, 130], seed=9)
    clean, clean_l, _ = run(c)
    for b, at in ((0, 271), (1, 65)):
        slot = int(c.slots[b][at])
        c.codes[slot] = 0x7F
        c.codes[slot, ::2] = 0xFF
        c.scales[slot] = math.nan
        slot = int(c.slots[b][at + 1])
        c.scales[slot] = math.inf
    out, l, err = run(c)
    assert err == 0
    for b, at in ((0, 271), (1, 65)):
        first, n, T = int(c.start[b]), c.nq[b], c.lens_list[b]
        seen_from = at - (T - n)  # the first query that sees the bad token
        assert torch.equal(out[first: first + seen_from], clean[first: first + seen_from])
        assert torch.equal(l[first: first + seen_from], clean_l[first: first + seen_from])
        assert torch.isnan(out[first + seen_from: first + n]).all()
        assert torch.isnan(l[first + seen_from: first + n]).all()


def test_a_query_with_nan_or_infinity_gives_nan_in_its_row_alone():
    c = Case(16, [20], [200], seed=10)
    clean, _, _ = run(c)
    c.q_lat[3, 5, 100] = math.nan
    c.q_rope[7, 15, 3] = math.inf
    out, l, _ = run(c)
    hit = torch.zeros(20, 16, dtype=torch.bool, device="cuda")
    hit[3, 5] = hit[7, 15] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(l[hit]).all()
    assert torch.equal(out[~hit], clean[~hit])


def test_zero_queries_and_large_ones():
    c = Case(16, [20], [200], seed=11)
    c.q_lat[2] = 0
    c.q_rope[2] = 0
    c.q_lat[3] *= 1e-30
    c.q_rope[3] *= 1e-30
    c.q_lat[4] *= 30
    check(c)


def test_row_scales_of_every_size():
    """Rows of very different size, zero rows and subnormal ones among them."""
    def rows(b, t, g):
        x = torch.randn((t, D), generator=g)
        e = torch.randint(-4, 5, (t, 1), generator=g)
        x = x * 2.0 ** e
        x[::17] = 0
        x[5::31] *= 1e-38
        return x
    check(Case(16, [33, 5], [700, 260], seed=12, rows=rows))


def test_a_dominant_token_over_a_bulk():
    """One token far above the rest (2^10 and more), early and late, and a common mean in the bulk."""
    def rows(b, t, g):
        x = 0.3 * torch.randn((t, D), generator=g) + 0.5
        x[3 if b == 0 else t - 2] *= 6
        return x
    c = Case(32, [4, 4], [1500, 1500], seed=13, rows=rows)
    c.q_lat.copy_((c.q_lat.float() * 0.4 + 0.3).bfloat16())
    check(c)


def test_strided_queries():
    c = Case(20, [7, 3], [90, 201], seed=14)
    want, _, _ = run(c)
    both = torch.cat([c.q_lat, c.q_rope], -1)           # [total, H, 576]
    c.q_lat, c.q_rope = both[..., :DL], both[..., DL:]
    assert torch.equal(run(c)[0], want)
    hm = both.transpose(0, 1).contiguous().transpose(0, 1)  # heads outermost in memory
    c.q_lat, c.q_rope = hm[..., :DL], hm[..., DL:]
    assert torch.equal(run(c)[0], want)
    one = c.q_lat[:1].expand(c.q_lat.shape[0], -1, -1)  # a stride of 0
    c.q_lat = one
    got = run(c)[0]
    c.q_lat = one.contiguous()
    assert torch.equal(run(c)[0], got)


def test_bad_table_entries_and_lengths_are_reported_and_read_as_empty():
    c = Case(16, [3, 4], [300, 200], seed=15)
    keep = [torch.ones(300, dtype=torch.bool), torch.ones(200, dtype=torch.bool)]
    c.table[0, 1] = -1
    c.table[1, 0] = c.codes.shape[0] // PAGE
    keep[0][64:128] = False
    keep[1][:64] = False
    out, l, err = run(c)
    assert err == -5
    c.check(out, l, keep=keep)
    c = Case(16, [3], [300], seed=16)
    c.lens[0] = -4
    out, l, err = run(c)
    assert err == -5 and (out == 0).all() and torch.isneginf(l).all()


def test_bad_query_ranges_are_reported_and_leave_their_rows():
    c = Case(16, [3, 4, 2], [300, 200, 90], seed=17)
    c.start.copy_(torch.tensor([0, 3, 100, 9], dtype=torch.int32))
    out, l, err = run(c)
    assert err == -5
    ref, _, tol, _ = c.reference(0)  # the batch's other sequences decide where a row's keys are cut
    assert ((out[:3].double() - ref).abs() <= tol).all()
    assert (out[3:] == 7).all() and (l[3:] == 7).all()


def test_no_query_at_all():
    c = Case(16, [0, 0], [30, 40], seed=18, pad=2)
    out, l, err = run(c)
    assert err == 0 and (out == 7).all() and (l == 7).all()
    got = pkg.mla_absorb_chunk_fp8_batch(c.q_lat[:0], c.q_rope[:0], *c.args()[2:], SM_SCALE)
    assert got.shape == (0, 16, DL)


def test_same_bits_every_time_and_with_a_larger_table():
    c = Case(128, [4, 9, 1], [3000, 700, 5000], seed=19)
    want, want_l, _ = run(c)
    for _ in range(3):
        out, l, _ = run(c)
        assert torch.equal(out, want) and torch.equal(l, want_l)


def test_captured_and_replayed_on_other_streams():
    c = Case(128, [4, 2], [900, 333], seed=20)
    d = Case(16, [30, 1], [200, 1000], seed=21)
    want_c, want_d = run(c)[0], run(d)[0]
    outs, graphs, streams = [], [], []
    for k in (c, d):
        rows = k.q_lat.shape[0]
        ws = pkg.alloc_workspace(pkg.mla_absorb_chunk_fp8_batch_workspace_size(len(k.nq), k.H, rows, k.max_blocks))
        out = torch.zeros((rows, k.H, DL), dtype=torch.bfloat16, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pkg.mla_absorb_chunk_fp8_batch(*k.args(), SM_SCALE, out=out, workspace=ws)
        outs.append((out, ws))
        graphs.append(g)
        streams.append(s)
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], want_c) and torch.equal(outs[1][0], want_d)


def test_one_token_agrees_with_the_decode_call():
    """A chunk of one token is a decode step (whose query is f32): both within their tolerances."""
    c = Case(128, [1, 1, 1], [1000, 64, 2500], seed=22)
    out, l, _ = run(c)
    dec_l = torch.empty((3, 128), device="cuda")
    dec = pkg.mla_absorb_decode_fp8_batch(c.q_lat.float(), c.q_rope.float(), c.codes, c.scales, c.table, c.lens,
                                          SM_SCALE, lse=dec_l)
    # the decode call's stated 1e-2 of the largest output, and this one's bf16 steps
    assert (out.float() - dec).abs().max() <= 1.5e-2 * dec.abs().max()
    assert (l - dec_l).abs().max() <= 3e-3 * dec_l.abs().max()


@pytest.mark.parametrize("pieces", [[50, 50], [1, 98, 1], [33, 33, 34]])
def test_a_prompt_in_pieces_is_the_prompt_at_once(pieces):
    """The same rows whichever chunk they come in (each within the tolerance of the definition)."""
    c = Case(32, [100], [100], seed=23)
    at = 0
    for n in pieces:
        d = Case(32, [100], [100], seed=23)
        d.q_lat, d.q_rope = d.q_lat[at: at + n].contiguous(), d.q_rope[at: at + n].contiguous()
        d.nq, d.lens_list, d.slots = [n], [at + n], [d.slots[0][: at + n]]
        d.start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        d.lens = torch.tensor([at + n], dtype=torch.int32, device="cuda")
        check(d)
        at += n
    check(c)


@pytest.mark.parametrize("H,nq,lens,causal", [(128, [300, 170], [400, 1000], True), (128, [90, 200], [2000, 50], False),
                                              (64, [41] * 12, [60 * i + 41 for i in range(12)], True),
                                              (20, [700, 1, 300], [900, 5000, 333], True)])
def test_many_row_tiles_a_cluster(H, nq, lens, causal):
    """Every cluster goes through many row tiles, whole ones and parts that are joined."""
    check(Case(H, nq, lens, seed=sum(nq), pad=5), causal)


def test_a_workspace_of_any_content_shared_by_calls_in_a_row():
    c, d = Case(128, [6, 3], [900, 333], seed=24), Case(16, [90, 1], [200, 1000], seed=25)
    want = [run(k)[:2] for k in (c, d)]
    size = max(pkg.mla_absorb_chunk_fp8_batch_workspace_size(2, k.H, k.q_lat.shape[0], k.max_blocks) for k in (c, d))
    ws = pkg.alloc_workspace(size)
    ws.view(torch.uint8).fill_(0xFF)
    got = []
    for _ in range(3):
        for k in (c, d):
            out = torch.empty((k.q_lat.shape[0], k.H, DL), dtype=torch.bfloat16, device="cuda")
            lse = torch.empty(out.shape[:2], device="cuda")
            pkg.mla_absorb_chunk_fp8_batch(*k.args(), SM_SCALE, out=out, lse=lse, workspace=ws)
            got.append((out, lse))
    for i, (out, lse) in enumerate(got):
        n = sum((c, d)[i % 2].nq)
        assert torch.equal(out[:n], want[i % 2][0][:n]) and torch.equal(lse[:n], want[i % 2][1][:n])


def test_pages_far_up_a_large_pool():
    """Rows past 2^31 bytes of codes, and past 2^31 / 8 of scales."""
    c = Case(16, [30, 2], [500, 300], seed=26)
    want = run(c)[:2]
    far = 70000
    codes = torch.full((far * 64, 576), 0x7F, dtype=torch.uint8, device="cuda")
    scales = torch.full((far * 64, 2), float("nan"), device="cuda")
    table = c.table.clone()
    held = sorted(int(p) for p in c.table.flatten().tolist() if p >= 0)
    for i, p in enumerate(held):
        to = far - 1 - i * 37
        codes[to * 64: to * 64 + 64] = c.codes[p * 64: p * 64 + 64]
        scales[to * 64: to * 64 + 64] = c.scales[p * 64: p * 64 + 64]
        table[c.table == p] = to
    c.codes, c.scales, c.table = codes, scales, table
    out, l, err = run(c)
    assert err == 0 and torch.equal(out, want[0]) and torch.equal(l, want[1])


def test_thousands_of_sequences():
    """More sequences and row tiles than the plan holds in shared memory or in one pass."""
    lens = [1 + (29 * i) % 90 for i in range(4500)]
    c = Case(2, [1 + (i % 7 == 0) for i in range(4500)], [max(2, t) for t in lens], seed=27)
    out, l, err = run(c)
    assert err == 0
    few = list(range(0, 4500, 90)) + [4095, 4096, 4097, 4499]
    nq = list(c.nq)
    c.nq = [n if b in few else 0 for b, n in enumerate(nq)]
    c.check(out, l)
    assert torch.isfinite(out.float()).all() and torch.isfinite(l).all()


def test_on_a_stream_of_its_own_while_the_current_one_is_busy():
    """What the call allocates for itself is not memory that the current stream still reads."""
    c = Case(64, [40], [500], seed=28)
    want = run(c)[0]
    s = torch.cuda.Stream()
    for _ in range(3):
        held = torch.full(want.shape, 3.0, dtype=torch.bfloat16, device="cuda")
        kept = torch.empty_like(held)
        torch.cuda.synchronize()
        torch.cuda._sleep(20000000)  # 10 ms or so
        kept.copy_(held)
        del held
        out = pkg.mla_absorb_chunk_fp8_batch(*c.args(), SM_SCALE, stream=s)
        s.synchronize()
        assert torch.equal(out, want)
        torch.cuda.synchronize()
        assert (kept == 3.0).all()
