"""The pages of a cache: append, fork, free, compact and copy against a host model, alone, in long
random sequences, and together with the quantizer and the chunk attention."""
import numpy as np
import pytest
import torch

import fp8_mla_latent_gb300 as pkg
from chunk_helpers import D, DL, DR, SM_SCALE, quantized
from pages_ref import PAGE, Pool, n_pages

pytestmark = pytest.mark.gpu


class Dev:
    """A pool's state on the GPU, and the calls on it."""

    def __init__(self, p):
        self.table = torch.from_numpy(p.table.copy()).cuda()
        self.lens = torch.from_numpy(p.lens.copy()).cuda()
        self.refs = torch.from_numpy(p.refs.copy()).cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def state(self):
        return self.table, self.lens, self.refs

    def same(self, p, err=0):
        assert np.array_equal(self.table.cpu().numpy(), p.table)
        assert np.array_equal(self.lens.cpu().numpy(), p.lens)
        assert np.array_equal(self.refs.cpu().numpy(), p.refs)
        assert int(self.err[0]) == err
        self.err.zero_()

    def append(self, n_new, cap):
        q, s = pkg.kv8_pages_append(*self.state(), i32(n_new), cap=cap, err_word=self.err)
        return q.cpu().numpy(), s.cpu().numpy()

    def fork(self, src, dst, fork_len=None):
        m = torch.full((max(1, len(src)), 2), -9, dtype=torch.int32, device="cuda")
        m, n = pkg.kv8_pages_fork(*self.state(), i32(src), i32(dst), None if fork_len is None else i32(fork_len),
                                  moves=m, err_word=self.err)
        m, n = m.cpu().numpy(), int(n[0])
        assert (m[n:] == -9).all()
        return [tuple(map(int, r)) for r in m[:n]]

    def free(self, seq):
        pkg.kv8_pages_free(*self.state(), i32(seq), err_word=self.err)

    def compact(self):
        live = torch.full((1,), -9, dtype=torch.int32, device="cuda")
        m, n = pkg.kv8_pages_compact(*self.state(), n_live=live, err_word=self.err)
        return [tuple(map(int, r)) for r in m[: int(n[0])].cpu().numpy()], int(live[0])


def i32(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def filled(rng, B, max_blocks, n_blocks, lens):
    """A host pool whose sequences grew in turns, so that their pages interleave."""
    p = Pool(B, max_blocks, n_blocks)
    left = np.array(lens, np.int32)
    while left.any():
        step = np.minimum(left, rng.integers(0, 100, B)).astype(np.int32)
        assert p.append(step, int(step.sum()))[2] == 0
        left -= step
    return p


@pytest.mark.parametrize("B,max_blocks,n_blocks,top", [(1, 1, 1, 64), (1, 5, 40, 200), (7, 4, 60, 130),
                                                       (64, 9, 700, 500), (300, 40, 20000, 900),
                                                       (1100, 3, 40000, 150)])
def test_append(B, max_blocks, n_blocks, top):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, min(top, max_blocks * PAGE) + 1, B)
    p = filled(rng, B, max_blocks, n_blocks, lens)
    d = Dev(p)
    for turn in range(3):
        room = max_blocks * PAGE - p.lens
        n_new = np.minimum(room, rng.integers(0, 70, B)).astype(np.int32)
        n_new[rng.random(B) < 0.3] = 0
        cap = int(n_new.sum()) + 5 * turn
        q, s, err = p.append(n_new, cap)
        gq, gs = d.append(n_new, cap)
        assert np.array_equal(gq, q) and np.array_equal(gs, s)
        d.same(p, err)


def test_append_a_long_prompt():
    p = Pool(2, 2000, 4100)
    d = Dev(p)
    for n_new in ([100003, 1], [0, 65], [64, 0]):
        q, s, err = p.append(np.array(n_new), sum(n_new) + 1)
        gq, gs = d.append(n_new, sum(n_new) + 1)
        assert np.array_equal(gq, q) and np.array_equal(gs, s)
        d.same(p, err)


@pytest.mark.parametrize("n_new,cap,err", [([1, 65, 0], 65, 2),          # more tokens than slots
                                           ([1, 64 * 4 + 1, 0], 400, 2),  # a table row too short
                                           ([60, 200, 130], 400, 2),      # too few free pages
                                           ([1, -1, 1], 400, 1)])
def test_append_that_cannot_be_takes_nothing(n_new, cap, err):
    p = Pool(3, 4, 5)
    assert p.append([70, 0, 3], 73)[2] == 0
    d = Dev(p)
    before = p.copy()
    assert p.append(n_new, cap)[2] == err
    gq, gs = d.append(n_new, cap)
    assert (gq == 0).all() and (gs == -1).all()
    d.same(before, err)


def test_append_refuses_a_shared_page_and_bad_state():
    p = Pool(3, 4, 9)
    p.append([70, 0, 3], 73)
    for hurt in ("shared", "page", "length"):
        q = p.copy()
        if hurt == "shared":
            q.refs[q.table[0, 1]] = 2
        elif hurt == "page":
            q.table[0, 1] = 9
        else:
            q.lens[0] = -1
        d = Dev(q)
        gq, gs = d.append([1, 1, 1], 3)
        assert (gq == 0).all() and (gs == -1).all()
        d.same(q, 1)


@pytest.mark.parametrize("B,max_blocks,n_blocks,top,n", [(2, 1, 4, 64, 1), (6, 4, 60, 256, 3), (90, 30, 3000, 900, 40),
                                                         (500, 60, 30000, 3000, 250)])
def test_fork(B, max_blocks, n_blocks, top, n):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, top + 1, B)
    lens[B - n:] = 0
    p = filled(rng, B, max_blocks, n_blocks, lens)
    d = Dev(p)
    dst = list(map(int, B - n + rng.permutation(n)))
    src = list(map(int, rng.integers(0, B - n, n)))  # a source may be named often
    moves, err = p.fork(src, dst)
    assert d.fork(src, dst) == moves
    d.same(p, err)
    assert p.consistent()
    p.free(dst)
    d.free(dst)
    d.same(p)
    cut = [int(rng.integers(0, p.lens[a] + 1)) for a in src]
    moves, err = p.fork(src, dst, cut)
    assert d.fork(src, dst, cut) == moves
    d.same(p, err)
    assert p.consistent()


@pytest.mark.parametrize("src,dst,fork_len", [([0], [0], None), ([0, 1], [3, 3], None), ([0, 3], [3, 4], None),
                                              ([0], [1], None), ([5], [3], None), ([0], [-1], None),
                                              ([0], [3], [71]), ([0], [3], [-1])])
def test_fork_that_cannot_be_changes_nothing(src, dst, fork_len):
    p = Pool(5, 4, 12)
    p.append([70, 3, 64, 0, 0], 137)
    d = Dev(p)
    assert p.copy().fork(src, dst, fork_len) == ([], 1)
    assert d.fork(src, dst, fork_len) == []
    d.same(p, 1)


def test_fork_without_a_free_page():
    p = Pool(4, 4, 3)
    p.append([70, 3, 0, 0], 73)
    d = Dev(p)
    assert d.fork([0], [2]) == []
    d.same(p, 2)
    assert p.fork([0], [2], [64]) == ([], 0)  # whole pages need none
    assert d.fork([0], [2], [64]) == []
    d.same(p)


def test_free_refuses_bad_lists_and_reports_bad_counts():
    p = Pool(4, 4, 9)
    p.append([70, 3, 64, 1], 138)
    for seq in ([0, 0], [4], [-1], [1, 2, 9]):
        d = Dev(p)
        d.free(seq)
        d.same(p, 1)
    d = Dev(p)
    d.refs[int(p.table[2, 0])] = 0  # a held page whose count is gone
    d.free([2])
    assert int(d.err[0]) == 1 and (d.refs >= 0).all() and int(d.lens[2]) == 0
    d = Dev(p)
    d.table[0, 0] = 100
    d.free([0])
    assert int(d.err[0]) == 1 and int(d.refs[int(p.table[0, 1])]) == 0
    d = Dev(p)
    d.free([])
    d.same(p)


@pytest.mark.parametrize("B,max_blocks,n_blocks,top,gone", [(1, 1, 1, 64, 0), (1, 2, 7, 100, 1), (6, 4, 40, 256, 3),
                                                            (90, 30, 3000, 900, 45), (300, 70, 21000, 4000, 200),
                                                            (40, 9, 300000, 500, 20)])
def test_compact(B, max_blocks, n_blocks, top, gone):
    rng = np.random.default_rng(B + 1)
    p = filled(rng, B, max_blocks, n_blocks, rng.integers(0, top + 1, B))
    if n_blocks > 100000:  # pages far up in a large pool
        far = np.sort(rng.choice(n_blocks, int((p.refs > 0).sum()), replace=False)).astype(np.int32)
        at = {int(a): int(z) for a, z in zip(np.flatnonzero(p.refs > 0), far)}
        refs = np.zeros_like(p.refs)
        for b in range(B):
            for c in range(n_pages(int(p.lens[b]))):
                refs[at[int(p.table[b, c])]] += 1
                p.table[b, c] = at[int(p.table[b, c])]
        p.refs = refs
    p.free(list(map(int, rng.permutation(B)[:gone])))
    d = Dev(p)
    moves, live = p.compact()
    assert d.compact() == (moves, live)
    d.same(p)
    assert p.consistent() and (p.refs[:live] > 0).all() and (p.refs[live:] == 0).all()
    assert d.compact() == ([], live)  # nothing is left to move
    d.same(p)


def test_compact_reports_entries_that_hold_no_page():
    p = Pool(3, 4, 12)
    p.append([70, 3, 64], 137)
    p.free([0])
    for value in (-1, 12, 9):
        q = p.copy()
        q.table[1, 0] = value
        d = Dev(q)
        d.compact()
        assert int(d.err[0]) == 1 and int(d.table[1, 0]) == value


def pool_bytes(rng, layers, n_blocks, extra=0):
    slots = n_blocks * PAGE + extra
    codes = torch.from_numpy(rng.integers(0, 256, (layers, slots, D), dtype=np.uint8)).cuda()
    scales = torch.from_numpy(rng.random((layers, slots, 2), dtype=np.float32)).cuda()
    return codes, scales


def moved(codes, scales, pairs):
    c, s = codes.clone(), scales.clone()
    for a, d in pairs:
        c[:, d * PAGE: d * PAGE + PAGE] = codes[:, a * PAGE: a * PAGE + PAGE]
        s[:, d * PAGE: d * PAGE + PAGE] = scales[:, a * PAGE: a * PAGE + PAGE]
    return c, s


@pytest.mark.parametrize("layers,n_blocks,n", [(1, 2, 1), (1, 40, 7), (3, 40, 20), (2, 700, 350), (5, 33, 16)])
def test_copy(layers, n_blocks, n):
    rng = np.random.default_rng(n)
    codes, scales = pool_bytes(rng, layers, n_blocks)
    order = rng.permutation(n_blocks)
    pairs = [(int(a), int(d)) for a, d in zip(order[:n], order[n: 2 * n])]
    want = moved(codes, scales, pairs)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    m = torch.tensor(pairs, dtype=torch.int32, device="cuda")
    pkg.kv8_pages_copy(codes, scales, m, err_word=err)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1]) and int(err[0]) == 0


def test_copy_of_one_layer_with_a_source_for_many_and_a_count():
    rng = np.random.default_rng(3)
    codes, scales = pool_bytes(rng, 1, 20, extra=17)
    codes, scales = codes[0], scales[0]
    pairs = [(4, 7), (4, 9), (4, 4), (0, 3), (19, 2)]
    for count, real in ((5, 5), (2, 2), (0, 0), (-3, 0), (99, 5)):
        c, s = codes.clone(), scales.clone()
        want = moved(codes[None], scales[None], pairs[:real])
        m = torch.tensor(pairs, dtype=torch.int32, device="cuda")
        pkg.kv8_pages_copy(c, s, m, n_moves=i32([count]))
        assert torch.equal(c, want[0][0]) and torch.equal(s, want[1][0])
    pkg.kv8_pages_copy(codes, scales, torch.zeros((0, 2), dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("pairs,real", [([(1, 2), (3, 2), (4, 5)], [(4, 5)]),           # a destination twice
                                        ([(1, 2), (1, 2), (4, 5)], [(4, 5)]),
                                        ([(1, 2), (2, 3), (4, 5)], [(1, 2), (4, 5)]),   # a source that is overwritten
                                        ([(1, 2), (2, 1), (4, 5)], [(4, 5)]),
                                        ([(1, 8), (8, 2), (-1, 2), (4, 5)], [(4, 5)])])  # pages outside the pool
def test_copy_leaves_out_pairs_that_cannot_be(pairs, real):
    rng = np.random.default_rng(4)
    codes, scales = pool_bytes(rng, 2, 8)
    want = moved(codes, scales, real)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkg.kv8_pages_copy(codes, scales, torch.tensor(pairs, dtype=torch.int32, device="cuda"), err_word=err)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1]) and int(err[0]) == 1


@pytest.mark.parametrize("seed", range(4))
def test_a_long_life(seed):
    """Random steps; after each, the state is the host model's and every sequence still reads, page
    by page, the rows that were written to it."""
    rng = np.random.default_rng(seed)
    B, mb, nb = 12, 6, 40
    p = Pool(B, mb, nb)
    d = Dev(p)
    codes = torch.zeros((nb * PAGE, D), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((nb * PAGE, 2), device="cuda")
    said = [[] for _ in range(B)]  # the value of each token, carried in its scale
    stamp = 0
    for _ in range(60):
        what = rng.choice(["append", "append", "append", "fork", "free", "compact"])
        if what == "append":
            n_new = (rng.integers(0, 50, B) * (rng.random(B) < 0.4)).astype(np.int32)
            q, s, err = p.append(n_new, 600)
            gq, gs = d.append(n_new, 600)
            assert np.array_equal(gq, q) and np.array_equal(gs, s)
            d.same(p, err)
            for b in range(B):
                for i in range(q[b], q[b + 1]):
                    stamp += 1
                    said[b].append(float(stamp))
                    scales[int(s[i])] = float(stamp)
        elif what == "fork":
            empty = [b for b in range(B) if p.lens[b] == 0]
            held = [b for b in range(B) if p.lens[b] > 0]
            if not empty or not held:
                continue
            dst = empty[: int(rng.integers(1, len(empty) + 1))]
            src = [int(rng.choice(held)) for _ in dst]
            cut = [int(rng.integers(0, p.lens[a] + 1)) for a in src]
            moves, err = p.fork(src, dst, cut)
            assert d.fork(src, dst, cut) == moves
            d.same(p, err)
            if moves:
                pkg.kv8_pages_copy(codes, scales, torch.tensor(moves, dtype=torch.int32, device="cuda"), err_word=d.err)
            if not err:
                for a, z, t in zip(src, dst, cut):
                    said[z] = said[a][:t]
        elif what == "free":
            seq = [b for b in range(B) if rng.random() < 0.25]
            p.free(seq)
            d.free(seq)
            d.same(p)
            for b in seq:
                said[b] = []
        else:
            moves, live = p.compact()
            assert d.compact() == (moves, live)
            if moves:
                pkg.kv8_pages_copy(codes, scales, torch.tensor(moves, dtype=torch.int32, device="cuda"), err_word=d.err)
            d.same(p)
        assert p.consistent()
        w = scales.cpu().numpy()
        for b in range(B):
            got = [w[int(p.table[b, t // PAGE]) * PAGE + t % PAGE, 0] for t in range(int(p.lens[b]))]
            assert got == said[b]


def test_serving_on_one_cache():
    """A prompt in two chunks, two branches of it, one step of each, a compaction: the chunk
    attention over the paged, shared, moved pages is the definition over each branch's own rows."""
    from chunk_helpers import Case
    H, mb, nb = 16, 8, 30
    g = torch.Generator().manual_seed(1)
    state = (torch.full((4, mb), -1, dtype=torch.int32, device="cuda"),
             torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(nb, dtype=torch.int32, device="cuda"))
    codes = torch.zeros((nb * PAGE, D), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((nb * PAGE, 2), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    own = [torch.zeros((0, D)) for _ in range(4)]  # each sequence's rows

    def step(n_new):
        rows = [torch.randn((n, D), generator=g) for n in n_new]
        total = sum(n_new)
        q_start, slots = pkg.kv8_pages_append(*state, i32(n_new), cap=total + 3, err_word=err)
        pkg.kv8_quantize_rows(torch.cat(rows + [torch.zeros((3, D))]).cuda(), codes, scales, dst_slot=slots)
        q_lat = torch.randn((total + 3, H, DL), generator=g).bfloat16().cuda()
        q_rope = torch.randn((total + 3, H, DR), generator=g).bfloat16().cuda()
        out = pkg.mla_absorb_chunk_fp8_batch(q_lat, q_rope, codes, scales, state[0], state[1], q_start, SM_SCALE)
        for b in range(4):
            own[b] = torch.cat([own[b], rows[b]])
        # the same tokens in a plain case of their own
        ref = Case(H, n_new, [len(r) for r in own], seed=2, rows=lambda b, t, _: own[b])
        ref.q_lat, ref.q_rope = q_lat, q_rope
        ref.check(out[:total])

    step([100, 0, 0, 37])
    step([41, 0, 0, 0])
    moves, n_moves = pkg.kv8_pages_fork(*state, i32([0, 0]), i32([1, 2]), i32([141, 70]), err_word=err)
    pkg.kv8_pages_copy(codes, scales, moves, n_moves=n_moves, err_word=err)
    own[1], own[2] = own[0], own[0][:70]
    step([2, 3, 60, 1])
    pkg.kv8_pages_free(*state, i32([0]), err_word=err)
    own[0] = own[0][:0]
    moves, n_moves = pkg.kv8_pages_compact(*state, err_word=err)
    pkg.kv8_pages_copy(codes, scales, moves, n_moves=n_moves, err_word=err)
    step([5, 1, 1, 64])
    assert int(err[0]) == 0


def test_a_captured_step_replayed():
    """append, quantize, attention in one graph: every replay takes the state one token on."""
    H, mb, nb, B = 16, 4, 12, 3
    p = Pool(B, mb, nb)
    p.append([63, 10, 64], 137)
    d = Dev(p)
    rows = torch.randn((B, D), device="cuda")
    codes = torch.zeros((nb * PAGE, D), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((nb * PAGE, 2), device="cuda")
    n_new = i32([1, 1, 1])
    q_start = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    slots = torch.zeros(B, dtype=torch.int64, device="cuda")
    ql, qr = torch.randn((B, H, DL), device="cuda").bfloat16(), torch.randn((B, H, DR), device="cuda").bfloat16()
    out = torch.zeros((B, H, DL), dtype=torch.bfloat16, device="cuda")
    ws = pkg.alloc_workspace(pkg.mla_absorb_chunk_fp8_batch_workspace_size(B, H, B, mb))

    def step():
        pkg.kv8_pages_append(*d.state(), n_new, q_start=q_start, dst_slot=slots, err_word=d.err)
        pkg.kv8_quantize_rows(rows, codes, scales, dst_slot=slots)
        pkg.mla_absorb_chunk_fp8_batch(ql, qr, codes, scales, d.table, d.lens, q_start, SM_SCALE, out=out, workspace=ws)

    step()
    p.append([1, 1, 1], 3)
    d.same(p)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(5):
        g.replay()
        _, s, _ = p.append([1, 1, 1], 3)
        d.same(p)
        assert np.array_equal(slots.cpu().numpy(), s)
        lat = codes[int(s[0])].view(torch.float8_e4m3fn).float() * scales[int(s[0]), 0]
        assert torch.equal(quantized(rows)[0][0], codes[int(s[0])]) or (lat[:DL] - rows[0, :DL]).abs().max() < 0.5
    assert torch.isfinite(out).all()


def test_free_pages_far_up_a_large_pool():
    """Pages are found a pass of the pool after the other; too few of them change nothing."""
    rng = np.random.default_rng(77)
    p = Pool(40, 30, 50000)
    p.refs[:] = 1
    spots = np.concatenate([rng.choice(16000, 5, replace=False), 16384 + rng.choice(16000, 90, replace=False),
                            33000 + rng.choice(17000, 100, replace=False)])
    p.refs[spots] = 0
    d = Dev(p)
    n_new = np.zeros(40, np.int32)
    n_new[:20] = rng.integers(1, 500, 20)
    q, s, err = p.append(n_new, int(n_new.sum()))
    gq, gs = d.append(n_new, int(n_new.sum()))
    assert err == 0 and np.array_equal(gq, q) and np.array_equal(gs, s)
    d.same(p)
    src, dst = [int(i) for i in rng.integers(0, 20, 15)], list(range(20, 35))
    moves, err = p.fork(src, dst)
    assert err == 0 and d.fork(src, dst) == moves
    d.same(p)
    before = p.copy()
    n_new = np.full(40, 600, np.int32)
    n_new[:35] = 0
    while True:  # as many as are free, and then one page more
        need = sum((int(n) + 63) // 64 for n in n_new)
        if need > int((p.refs == 0).sum()):
            break
        n_new[35:] += 64
    assert n_new.max() <= 30 * PAGE
    q, s, err = p.append(n_new, int(n_new.sum()))
    gq, gs = d.append(n_new, int(n_new.sum()))
    assert err == 2 and (gq == 0).all() and (gs == -1).all()
    d.same(before, 2)


def test_copy_far_up_a_large_pool():
    """Pages past 2^31 bytes of codes."""
    n_blocks = 70000
    codes = torch.zeros((n_blocks * PAGE, D), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((n_blocks * PAGE, 2), device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    pairs = [(3, 69999), (69998, 4), (60001, 60003)]
    for a, _ in pairs:
        codes[a * PAGE: (a + 1) * PAGE].random_(0, 256, generator=g)
        scales[a * PAGE: (a + 1) * PAGE].normal_(generator=g)
    pkg.kv8_pages_copy(codes, scales, torch.tensor(pairs, dtype=torch.int32, device="cuda"))
    for a, b in pairs:
        for w in (codes, scales):
            assert torch.equal(w[a * PAGE: (a + 1) * PAGE], w[b * PAGE: (b + 1) * PAGE])
            w[a * PAGE: (a + 1) * PAGE] = 0
            w[b * PAGE: (b + 1) * PAGE] = 0
    assert not codes.any() and not scales.any()


def test_calls_with_nothing_to_do():
    p = Pool(3, 4, 9)
    p.append([70, 0, 3], 73)
    d = Dev(p)
    q, s = d.append([0, 0, 0], 0)
    assert (q == 0).all() and len(s) == 0
    q, s = d.append([0, 0, 0], 4)
    assert (q == 0).all() and (s == -1).all()
    assert d.fork([], []) == []
    d.free([])
    d.same(p)
    codes, scales = pool_bytes(np.random.default_rng(1), 1, 9)
    want = codes.clone()
    pkg.kv8_pages_copy(codes, scales, torch.zeros((0, 2), dtype=torch.int32, device="cuda"), err_word=d.err)
    pkg.kv8_pages_copy(codes, scales, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), n_moves=i32([0]),
                       err_word=d.err)
    assert torch.equal(codes, want)
    d.same(p)
    e = Dev(Pool(3, 4, 9))
    assert e.compact() == ([], 0)
    e.same(Pool(3, 4, 9))


def test_on_a_stream_of_its_own_while_the_current_one_is_busy():
    """What a call allocates for itself is not memory that the current stream still reads."""
    p = Pool(3, 40, 100)
    p.append([70, 0, 3], 73)
    s = torch.cuda.Stream()
    for cap in (5000, 70000):
        want = p.copy()
        moves, _ = want.fork([0], [1])
        q_want, s_want, _ = want.append([0, 5, 0], cap)
        d = Dev(p)
        src, dst, n_new = i32([0]), i32([1]), i32([0, 5, 0])
        held = [torch.full((n,), 3, dtype=t, device="cuda") for n, t in ((cap, torch.int64), (4, torch.int32),
                                                                         (2, torch.int32), (1, torch.int32))]
        torch.cuda.synchronize()
        torch.cuda._sleep(20000000)  # 10 ms or so
        kept = [h.clone() for h in held]
        del held
        m, n = pkg.kv8_pages_fork(*d.state(), src, dst, err_word=d.err, stream=s)
        q, slots = pkg.kv8_pages_append(*d.state(), n_new, cap=cap, err_word=d.err, stream=s)
        s.synchronize()
        torch.cuda.synchronize()
        assert [tuple(r) for r in m[: int(n[0])].tolist()] == moves
        assert np.array_equal(q.cpu().numpy(), q_want) and np.array_equal(slots.cpu().numpy(), s_want)
        assert all((k == 3).all() for k in kept)
        d.same(want)
