"""Cases for the operators over a paged fp8 latent cache that keeps growing: the
absorbed attention of a chunk of new tokens, and the copying, forking, appending,
freeing and compacting of the cache's pages.

``run`` computes a case in elementary torch operations, or, with ``own`` set, by
the library's calls.  Lengths follow from a case's sizes alone; the values, the
page order and the sequences that take part follow from the seed.
"""
import math
import random

import torch

own = False

DL, DR, D, PAGE = 512, 64, 576, 64
SM_SCALE = 1.0 / math.sqrt(192.0)
ROW_BYTES = D + 8


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a few tokens of a small model's single sequence: latency is all there is
        dict(name="chunk tiny", op="chunk", B=1, H=4, q=1, T=256, ragged=False, causal=True, lse=True, pad=0),
        # a batch of 32 served sequences, each checking four drafted tokens
        dict(name="chunk draft", op="chunk", B=32, H=128, q=4, T=16384, ragged=True, causal=True, lse=False, pad=0),
        # the first chunk of a prompt: nothing before it, half of the square masked
        dict(name="chunk prompt", op="chunk", B=1, H=128, q=4096, T=4096, ragged=False, causal=True, lse=False, pad=0),
        # a later chunk of two long prompts
        dict(name="chunk long", op="chunk", B=2, H=128, q=256, T=65536, ragged=False, causal=True, lse=True, pad=0),
        # a mixed batch of a 16-head shard: single tokens beside short chunks, a padded query array
        dict(name="chunk mixed", op="chunk", B=64, H=16, q=61, T=8192, ragged=True, causal=True, lse=True, pad=37),
        # every new token sees the whole sequence; a head count that no tile divides
        dict(name="chunk both ways", op="chunk", B=5, H=20, q=333, T=1999, ragged=True, causal=False, lse=False, pad=0),
        # a handful of pages of one layer
        dict(name="copy few", op="copy", L=1, n_blocks=256, n=5),
        # a prefix duplicated in every layer of a four-layer slice of the cache
        dict(name="copy many", op="copy", L=4, n_blocks=8192, n=3500),
        # one sequence branches twice and both branches append a token
        dict(name="branch few", op="branch", B=4, n=2, T=300, new=1, ragged=False),
        # sampling several continuations of 64 sequences
        dict(name="branch many", op="branch", B=64, n=192, T=4096, new=8, ragged=True),
        # a small pool after a few sequences left it
        dict(name="compact small", op="compact", L=1, B=6, T=900, keep=0.5),
        # half of a large pool's sequences have left
        dict(name="compact large", op="compact", L=2, B=256, T=2048, keep=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "copy", "branch", "compact"])
    if op == "copy":
        n_blocks = _log(rng, 16, 8192)
        return dict(op=op, L=rng.choice([1, 1, 2, 3, 4]), n_blocks=n_blocks, n=_log(rng, 1, n_blocks * 0.42))
    if op == "branch":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, n=_log(rng, 1, 3 * B + 1), T=_log(rng, 1, 4096), new=_log(rng, 1, 300),
                    ragged=rng.random() < 0.7)
    if op == "compact":
        return dict(op=op, L=rng.choice([1, 2]), B=_log(rng, 2, 256), T=_log(rng, 64, 2048),
                    keep=rng.choice([0.1, 0.3, 0.5, 0.8]))
    B, q, T = _log(rng, 1, 64), _log(rng, 1, 4096), _log(rng, 1, 131072)
    H = rng.choice([1, 3, 4, 16, 20, 32, 64, 128, 128, 128])
    causal = rng.random() < 0.8
    if causal and T < q:
        T += q - 1
    # no more than the largest listed case, in work and in the plain form's scores
    while B * q * H * T > 2 * 256 * 128 * 65536:
        if B > 1:
            B = max(1, B // 2)
        elif q > 64:
            q = q // 2 + 1
        else:
            T = max(q, T // 2)
    return dict(op="chunk", B=B, H=H, q=q, T=T, ragged=rng.random() < 0.6, causal=causal, lse=rng.random() < 0.5,
                pad=rng.choice([0, 0, 5, 130]))


def _lens(case):
    """Query counts and cache lengths of a chunk case's sequences, from its sizes alone."""
    B, q, T = case["B"], case["q"], case["T"]
    if not case["ragged"]:
        return [q] * B, [T] * B
    r = random.Random(f"{B} {q} {T}")
    nq = [1 + r.randrange(q) for _ in range(B)]
    lens = [max(n, 1 + r.randrange(T)) if case["causal"] else 1 + r.randrange(T) for n in nq]
    nq[0], lens[0] = q, max(T, q) if case["causal"] else T
    return nq, lens


def _branch_lens(case):
    r = random.Random(f"{case['B']} {case['T']}")
    return [1 + r.randrange(case["T"]) if case["ragged"] else case["T"] for _ in range(case["B"])]


def _pages(t):
    return (t + PAGE - 1) // PAGE


# ---------------------------------------------------------------- inputs

def _pool(gen, n_blocks, layers=None):
    """A cache of latent rows with channel gains and a few outlying rows, quantized."""
    codes, scales = [], []
    for _ in range(layers or 1):
        gain = torch.exp(0.5 * torch.randn(D, generator=gen, device="cuda"))
        x = torch.randn((n_blocks * PAGE, D), generator=gen, device="cuda") * gain
        x *= 1.0 + 1.5 * (torch.rand((n_blocks * PAGE, 1), generator=gen, device="cuda") < 0.01)
        s = torch.stack([x[:, :DL].abs().amax(1), x[:, DL:].abs().amax(1)], 1) / 448.0
        y = torch.cat([x[:, :DL] / s[:, :1], x[:, DL:] / s[:, 1:]], 1)
        codes.append(y.to(torch.float8_e4m3fn).view(torch.uint8))
        scales.append(s)
    if layers is None:
        return codes[0], scales[0]
    return torch.stack(codes), torch.stack(scales)


def _tables(gen, lens, max_blocks, n_blocks):
    """Pages of the sequences, from a random order of the pool; -1 elsewhere."""
    n = torch.tensor([_pages(t) for t in lens], device="cuda")
    col = torch.arange(max_blocks, device="cuda")
    held = col[None, :] < n[:, None]
    order = torch.randperm(n_blocks, generator=gen, device="cuda").int()
    table = torch.full((len(lens), max_blocks), -1, dtype=torch.int32, device="cuda")
    table[held] = order[: int(n.sum())]
    return table


def _refs(table, n_blocks):
    refs = torch.zeros(n_blocks, dtype=torch.int32, device="cuda")
    held = table[table >= 0].long()
    return refs.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "chunk":
        H = case["H"]
        nq, lens = _lens(case)
        mb = _pages(max(lens))
        n_blocks = sum(_pages(t) for t in lens) + 3
        codes, scales = _pool(gen, n_blocks)
        rows = sum(nq) + case["pad"]
        start = [0]
        for n in nq:
            start.append(start[-1] + n)
        return dict(op=op, case=case, codes=codes, scales=scales,
                    table=_tables(gen, lens, mb, n_blocks),
                    lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                    start=torch.tensor(start, dtype=torch.int32, device="cuda"),
                    q_lat=torch.randn((rows, H, DL), generator=gen, device="cuda").bfloat16(),
                    q_rope=torch.randn((rows, H, DR), generator=gen, device="cuda").bfloat16(),
                    out=torch.zeros((rows, H, DL), dtype=torch.bfloat16, device="cuda"),
                    lse=torch.zeros((rows, H), device="cuda") if case["lse"] else None)
    if op == "copy":
        L, nb, n = case["L"], case["n_blocks"], case["n"]
        codes, scales = _pool(gen, nb, L)
        order = torch.randperm(nb, generator=gen, device="cuda").int()
        moves = torch.stack([order[:n], order[n: 2 * n]], 1).contiguous()
        return dict(op=op, codes=codes, scales=scales, moves=moves)
    if op == "branch":
        B, n, T, new = case["B"], case["n"], case["T"], case["new"]
        lens = _branch_lens(case)
        mb = _pages(T + new)
        n_blocks = sum(_pages(t) for t in lens) + n * (_pages(new) + 2)
        codes, scales = _pool(gen, n_blocks)
        table = _tables(gen, lens + [0] * n, mb, n_blocks)
        order = torch.randint(B, (n,), generator=gen, device="cuda", dtype=torch.int32)
        n_new = torch.zeros(B + n, dtype=torch.int32, device="cuda")
        n_new[B:] = new
        return dict(op=op, codes=codes, scales=scales, table=table, refs=_refs(table, n_blocks),
                    lens=torch.tensor(lens + [0] * n, dtype=torch.int32, device="cuda"), src=order,
                    dst=torch.arange(B, B + n, dtype=torch.int32, device="cuda"), n_new=n_new,
                    moves=torch.full((n, 2), -1, dtype=torch.int32, device="cuda"),
                    n_moves=torch.zeros(1, dtype=torch.int32, device="cuda"),
                    start=torch.zeros(B + n + 1, dtype=torch.int32, device="cuda"),
                    slots=torch.full((n * new,), -1, dtype=torch.int64, device="cuda"))
    L, B, T = case["L"], case["B"], case["T"]
    lens = [T - (37 * b) % max(1, T // 2) for b in range(B)]
    n_blocks = sum(_pages(t) for t in lens) + 5
    codes, scales = _pool(gen, n_blocks, L)
    table = _tables(gen, lens, _pages(T), n_blocks)
    gone = torch.randperm(B, generator=gen, device="cuda")[max(1, round(B * case["keep"])):]
    table[gone] = -1
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    lens[gone] = 0
    refs = _refs(table, n_blocks)
    return dict(op=op, codes=codes, scales=scales, table=table.clone(), refs=refs.clone(), table0=table,
                refs0=refs, lens=lens,
                moves=torch.full((n_blocks // 2, 2), -1, dtype=torch.int32, device="cuda"),
                n_moves=torch.zeros(1, dtype=torch.int32, device="cuda"))


# ---------------------------------------------------------------- plain forms

def _chunk(s):
    """Padded to the longest sequence and the largest chunk, in 32 bits."""
    c, start, lens = s["case"], s["start"].long(), s["lens"].long()
    H, qm = c["H"], c["q"]
    rows = s["q_lat"].shape[0]
    t = torch.arange(s["table"].shape[1] * PAGE, device="cuda")
    slot = s["table"].long().clamp(min=0)[:, t // PAGE] * PAGE + t % PAGE
    valid = t[None, :] < lens[:, None]
    x = s["codes"][slot].view(torch.float8_e4m3fn).float()
    sc = s["scales"][slot]
    lat = (x[..., :DL] * sc[..., :1]).masked_fill(~valid[..., None], 0.0)
    rope = (x[..., DL:] * sc[..., 1:]).masked_fill(~valid[..., None], 0.0)
    i = torch.arange(qm, device="cuda")
    nq = start[1:] - start[:-1]
    at = (start[:-1, None] + i[None, :]).clamp(max=rows - 1)
    ql, qr = s["q_lat"][at].float().flatten(1, 2), s["q_rope"][at].float().flatten(1, 2)
    z = torch.baddbmm(ql @ lat.transpose(1, 2), qr, rope.transpose(1, 2)).mul_(SM_SCALE)
    see = lens[:, None].expand(-1, qm) - (nq[:, None] - 1 - i[None, :] if c["causal"] else 0)
    see = see.clamp(min=0).minimum(lens[:, None])
    z = z.unflatten(1, (qm, H)).masked_fill_((t >= see[..., None])[:, :, None, :], -math.inf)
    m = z.amax(-1, keepdim=True).clamp(min=-3e38)
    p = z.sub_(m).exp_()
    den = p.sum(-1, keepdim=True)
    o = (p.flatten(1, 2) @ lat).unflatten(1, (qm, H)) / den.clamp(min=1e-38)
    r = torch.arange(rows, device="cuda")
    b = (torch.searchsorted(start, r, right=True) - 1).clamp(max=lens.numel() - 1)
    mine = (r < start[-1])[:, None]
    k = (r - start[b]).clamp(max=qm - 1)
    s["out"].copy_(torch.where(mine[..., None], o[b, k].bfloat16(), s["out"]))
    if s["lse"] is not None:
        s["lse"].copy_(torch.where(mine, (m + den.log())[..., 0][b, k], s["lse"]))


def _copy(codes, scales, moves, n_moves=None):
    """Pages moves[:, 0] -> moves[:, 1] of every layer; a pair past n_moves copies a page to itself."""
    src, dst = moves[:, 0].long(), moves[:, 1].long()
    if n_moves is not None:
        real = torch.arange(moves.shape[0], device="cuda") < n_moves
        none = src[:1].clamp(min=0)
        src, dst = torch.where(real, src, none), torch.where(real, dst, none)
    c = codes.view(-1, codes.shape[-2] // PAGE, PAGE * D)
    w = scales.view(-1, scales.shape[-2] // PAGE, PAGE * 2)
    c[:, dst] = c[:, src]
    w[:, dst] = w[:, src]


def _free_pages(refs):
    """The free pages in order, and the others behind them."""
    return torch.argsort((refs != 0).to(torch.int8), stable=True)


def _free(s, seq):
    seq = seq.long()
    col = torch.arange(s["table"].shape[1], device="cuda")
    held = col[None, :] < ((s["lens"][seq] + PAGE - 1) // PAGE)[:, None]
    page = s["table"][seq].clamp(min=0).long()
    s["refs"].index_add_(0, page.flatten(), -held.flatten().int())
    s["table"][seq] = s["table"][seq].masked_fill(held, -1)
    s["lens"][seq] = 0


def _fork(s):
    src, dst = s["src"].long(), s["dst"].long()
    lens = s["lens"][src]
    have = (lens + PAGE - 1) // PAGE
    part = (lens % PAGE) != 0
    col = torch.arange(s["table"].shape[1], device="cuda")
    page = s["table"][src].long()
    last = (col[None, :] == (have - 1)[:, None]) & part[:, None]
    k = torch.cumsum(part, 0) - 1
    fresh = _free_pages(s["refs"])[k.clamp(min=0)]
    old = page.gather(1, (have - 1).clamp(min=0).long()[:, None])[:, 0]
    row = torch.where(last, fresh[:, None], page)
    held = col[None, :] < have[:, None]
    s["table"][dst] = torch.where(held, row, s["table"][dst].long()).int()
    s["refs"].index_add_(0, row.clamp(min=0).flatten(), held.flatten().int())
    s["lens"][dst] = lens
    s["n_moves"].copy_(part.sum()[None])
    at = torch.where(part, k, src.numel())
    moves = torch.cat([s["moves"], s["moves"][:1]])
    moves[at] = torch.stack([old, fresh], 1).int()
    s["moves"].copy_(moves[:-1])


def _append(s):
    lens, new = s["lens"].long(), s["n_new"].long()
    have, want = (lens + PAGE - 1) // PAGE, (lens + new + PAGE - 1) // PAGE
    need = want - have
    first = torch.cumsum(need, 0) - need
    col = torch.arange(s["table"].shape[1], device="cuda")
    take = (col[None, :] >= have[:, None]) & (col[None, :] < want[:, None])
    order = _free_pages(s["refs"])
    k = (first[:, None] + col[None, :] - have[:, None]).clamp(min=0, max=order.numel() - 1)
    page = order[k]
    s["table"].copy_(torch.where(take, page.int(), s["table"]))
    s["refs"].index_add_(0, page.flatten(), take.flatten().int())
    s["start"][1:] = torch.cumsum(new, 0).int()
    i = torch.arange(s["slots"].numel(), device="cuda")
    b = torch.searchsorted(s["start"].long(), i, right=True) - 1
    pos = lens[b] + i - s["start"][b]
    s["slots"].copy_(s["table"][b, pos // PAGE].long() * PAGE + pos % PAGE)
    s["lens"].copy_((lens + new).int())


def _compact(s):
    refs = s["refs"]
    idx = torch.arange(refs.numel(), device="cuda")
    live = refs > 0
    n_live = live.sum()
    hole, mover = ~live & (idx < n_live), live & (idx >= n_live)
    n = mover.sum()
    holes = torch.argsort((~hole).to(torch.int8), stable=True)
    movers = torch.argsort((~mover).to(torch.int8), stable=True)
    to = holes[(torch.cumsum(mover, 0) - 1).clamp(min=0)]
    remap = torch.where(mover, to, idx)
    held = torch.arange(s["table"].shape[1], device="cuda")[None, :] < ((s["lens"] + PAGE - 1) // PAGE)[:, None]
    s["table"].copy_(torch.where(held, remap[s["table"].clamp(min=0).long()].int(), s["table"]))
    back = torch.zeros_like(refs).index_add_(0, remap, refs)
    refs.copy_(back)
    k = torch.arange(s["moves"].shape[0], device="cuda")
    pair = torch.stack([movers[: k.numel()], holes[: k.numel()]], 1).int()
    s["moves"].copy_(torch.where((k < n)[:, None], pair, s["moves"]))
    s["n_moves"].copy_(n[None])


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "chunk":
        _chunk(s)
    elif op == "copy":
        _copy(s["codes"], s["scales"], s["moves"])
    elif op == "branch":
        _free(s, s["dst"])
        _fork(s)
        _copy(s["codes"], s["scales"], s["moves"], s["n_moves"])
        _append(s)
    else:
        s["table"].copy_(s["table0"])
        s["refs"].copy_(s["refs0"])
        _compact(s)
        _copy(s["codes"], s["scales"], s["moves"], s["n_moves"])
    return _outputs(s)


def _outputs(s):
    if s["op"] == "chunk":
        return {"out": s["out"], "lse": s["lse"]} if s["lse"] is not None else {"out": s["out"]}
    got = {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]}
    for k in ("table", "refs", "lens", "moves", "n_moves", "start", "slots"):
        if k in s and s["op"] != "copy":
            got[k] = s[k]
    return got


def _run_own(s):
    import fp8_mla_latent_gb300 as kv
    op = s["op"]
    if op == "chunk":
        kv.mla_absorb_chunk_fp8_batch(s["q_lat"], s["q_rope"], s["codes"], s["scales"], s["table"], s["lens"],
                                      s["start"], SM_SCALE, causal=s["case"]["causal"], out=s["out"], lse=s["lse"])
    elif op == "copy":
        kv.kv8_pages_copy(s["codes"], s["scales"], s["moves"])
    elif op == "branch":
        kv.kv8_pages_free(s["table"], s["lens"], s["refs"], s["dst"])
        kv.kv8_pages_fork(s["table"], s["lens"], s["refs"], s["src"], s["dst"], moves=s["moves"],
                          n_moves=s["n_moves"])
        kv.kv8_pages_copy(s["codes"], s["scales"], s["moves"], n_moves=s["n_moves"])
        kv.kv8_pages_append(s["table"], s["lens"], s["refs"], s["n_new"], q_start=s["start"], dst_slot=s["slots"])
    else:
        s["table"].copy_(s["table0"])
        s["refs"].copy_(s["refs0"])
        kv.kv8_pages_compact(s["table"], s["lens"], s["refs"], moves=s["moves"], n_moves=s["n_moves"])
        kv.kv8_pages_copy(s["codes"], s["scales"], s["moves"], n_moves=s["n_moves"])
    return _outputs(s)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    page = PAGE * ROW_BYTES
    if op == "chunk":
        nq, lens = _lens(case)
        H = case["H"]
        if case["causal"]:
            seen = sum(n * t - n * (n - 1) // 2 for n, t in zip(nq, lens))
        else:
            seen = sum(n * t for n, t in zip(nq, lens))
        rows = sum(nq) * H
        nbytes = ROW_BYTES * sum(lens) + rows * (2 * D + 2 * DL + (4 if case["lse"] else 0))
        nbytes += 4 * sum(_pages(t) for t in lens) + 8 * case["B"]
        return {"bytes": nbytes, "flops": 2 * (D + DL) * H * seen}
    if op == "copy":
        return {"bytes": 2 * page * case["n"] * case["L"] + 8 * case["n"], "flops": 0}
    if op == "branch":
        n, new = case["n"], case["new"]
        lens = _branch_lens(case)
        mean = sum(_pages(t) for t in lens) / len(lens)
        part = sum(t % PAGE != 0 for t in lens) / len(lens)
        # the copied pages; table entries and reference counts of the branches, freed and taken
        nbytes = 2 * page * part * n + n * mean * 4 * 8 + n * new * 8 + 4 * 4 * (case["B"] + n)
        return {"bytes": nbytes, "flops": 0}
    B, T = case["B"], case["T"]
    lens = [_pages(T - (37 * b) % max(1, T // 2)) for b in range(B)]
    nb = sum(lens) + 5
    live = max(1, round(B * case["keep"])) / B
    moved = nb * live * (1 - live)
    return {"bytes": 2 * page * moved * case["L"] + 4 * (4 * nb + 4 * B * _pages(T)), "flops": 0}


# ---------------------------------------------------------------- in 64 bits

def _e4m3_values():
    """The 256 values of the format, from its definition (the two NaN codes are not used)."""
    v = []
    for byte in range(256):
        e, f = (byte >> 3) & 15, byte & 7
        mag = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v.append(-mag if byte & 128 else mag)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def exact(case, seed):
    if case["op"] != "chunk":
        return None  # pages are moved, not computed
    s = prepare(case, seed)
    nq, lens = _lens(case)
    value = _e4m3_values()
    out, lse = s["out"].double(), None if s["lse"] is None else s["lse"].double()
    first = 0
    for b, (n, T) in enumerate(zip(nq, lens)):
        pages = s["table"][b, : _pages(T)].long()
        slot = (pages[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten()[:T]
        row = value[s["codes"][slot].long()]
        key = torch.cat([row[:, :DL] * s["scales"][slot, :1].double(), row[:, DL:] * s["scales"][slot, 1:].double()], 1)
        step = max(1, int(4e8 // (T * case["H"])))
        for i in range(0, n, step):
            j = min(n, i + step)
            q = torch.cat([s["q_lat"][first + i: first + j], s["q_rope"][first + i: first + j]], -1).double()
            z = (q.flatten(0, 1) @ key.T).unflatten(0, (j - i, case["H"])) * SM_SCALE
            if case["causal"]:
                last = T - n + torch.arange(i, j, device="cuda")
                z.masked_fill_(torch.arange(T, device="cuda")[None, None, :] > last[:, None, None], -math.inf)
            w = torch.logsumexp(z, -1)
            p = torch.exp(z - w[..., None])
            out[first + i: first + j] = (p.flatten(0, 1) @ key[:, :DL]).unflatten(0, (j - i, case["H"]))
            if lse is not None:
                lse[first + i: first + j] = w
        first += n
    return {"out": out, "lse": lse} if lse is not None else {"out": out}
