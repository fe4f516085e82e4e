"""Cases for the operators around a paged fp8 latent cache that a serving layer runs beside the chunk
attention: attention with a sliding window and first tokens that stay visible, attention of a batch
whose sequences share a long prefix, and the norm that opens the layer, with the residual's addition
and an output in 8 bits.

``run`` computes a case in elementary torch operations, or, with ``own`` set, by the library's calls.
Lengths follow from a case's sizes alone; the values and the page order follow from the seed.
"""
import math
import random

import torch

own = False

DL, DR, D, PAGE = 512, 64, 576, 64
SM_SCALE = 1.0 / math.sqrt(192.0)
ROW_BYTES = D + 8
EPS = 1e-6
BLOCK = 256  # query tokens that the plain window attention takes at a time
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token of a small model's single sequence behind a short window: latency is all there is
        dict(name="window tiny", op="window", B=1, H=4, q=1, T=700, W=128, S=4, ragged=False, lse=False, pad=0),
        # single tokens of 64 served sequences on a 16-head shard
        dict(name="window tokens, 16 heads", op="window", B=64, H=16, q=1, T=8192, W=4096, S=4, ragged=True, lse=True, pad=0),
        # single tokens of 32 served sequences with all heads on one device
        dict(name="window tokens", op="window", B=32, H=128, q=1, T=32768, W=2048, S=64, ragged=True, lse=False, pad=0),
        # short chunks beside single tokens; a head count that no tile divides, an odd window, padded rows
        dict(name="window mixed", op="window", B=24, H=20, q=61, T=6000, W=1111, S=70, ragged=True, lse=True, pad=37),
        # a later chunk of one long prompt
        dict(name="window prompt", op="window", B=1, H=128, q=4096, T=32768, W=2048, S=128, ragged=False, lse=False, pad=0),
        # a few continuations of one short prompt: latency
        dict(name="shared tiny", op="shared", G=1, B=3, H=4, q=1, P=500, own=40, lse=False, pad=0),
        # 64 conversations behind one long system prompt on a 16-head shard, a token each
        dict(name="shared tokens, 16 heads", op="shared", G=1, B=64, H=16, q=1, P=16384, own=700, lse=True, pad=0),
        # 32 samples of one long prompt with all heads on one device
        dict(name="shared tokens", op="shared", G=1, B=32, H=128, q=1, P=32768, own=500, lse=False, pad=0),
        # several prompts, each with some continuations that check drafted tokens; lengths that no page divides
        dict(name="shared groups", op="shared", G=5, B=29, H=20, q=4, P=5001, own=333, lse=True, pad=9),
        # the norm in front of a decode step of one sequence
        dict(name="norm token", op="norm", n=1, w=7168, type="bf16", group=0, add=True, normed=False),
        # an odd width, a scale per row, the normed rows kept in 16 bits as well
        dict(name="norm odd", op="norm", n=517, w=1501, type="f16", group=0, add=True, normed=True),
        # the norm in front of a prompt's chunk, a scale for every 128 channels
        dict(name="norm prompt", op="norm", n=16384, w=7168, type="bf16", group=128, add=True, normed=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "shared", "shared", "norm"])
    if op == "norm":
        n, w = _log(rng, 1, 16384), _log(rng, 16, 16384)
        w = w if rng.random() < 0.4 else max(16, w // 16 * 16)
        return dict(op=op, n=min(n, max(1, 16384 * 7168 // w)), w=w, type=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    group=rng.choice([0, 128]), add=rng.random() < 0.7, normed=rng.random() < 0.4)
    H = rng.choice([1, 3, 4, 16, 20, 32, 64, 128, 128, 128])
    if op == "window":
        B, q, T = _log(rng, 1, 64), rng.choice([1, _log(rng, 1, 4096)]), _log(rng, 1, 65536)
        W, S = _log(rng, 1, 8192), rng.choice([0, 1, 4, 64, _log(rng, 1, 512)])
        T = max(T, q)
        while B > 1 and B * T > 2 ** 20:
            B //= 2
        # no more than the largest listed case, in work and in the plain form's scores
        while B * q * H * min(T, W + S) > 4096 * 128 * 2176 or B * q * H * min(T, W + S + min(q, BLOCK)) > 2 ** 30:
            if B > 1:
                B = max(1, B // 2)
            elif q > 64:
                q = q // 2 + 1
            else:
                W = W // 2 + 1
        return dict(op=op, B=B, H=H, q=q, T=T, W=W, S=S, ragged=rng.random() < 0.6, lse=rng.random() < 0.5,
                    pad=rng.choice([0, 0, 5, 130]))
    G = rng.choice([1, 1, 1, 2, 3, _log(rng, 2, 12)])
    B = max(G, _log(rng, 1, 96))
    q, P, mine = rng.choice([1, 1, 1, 2, 4, _log(rng, 1, 16)]), _log(rng, 1, 65536), _log(rng, 1, 4096)
    while B > G and B * mine > 2 ** 18:
        B = max(G, B // 2)
    while B * q * H * (P + mine) > 96 * 128 * 33000:
        P = P // 2 + 1
    return dict(op=op, G=G, B=B, H=H, q=q, P=P, own=max(mine, q), lse=rng.random() < 0.5, pad=rng.choice([0, 0, 5, 130]))


def _lens(case):
    """Query counts and cache lengths of a case's sequences, from its sizes alone."""
    B, q = case["B"], case["q"]
    if case["op"] == "shared":
        r = random.Random(f"{B} {q} {case['own']}")
        nq = [1 + r.randrange(q) for _ in range(B)]
        mine = [max(n, 1 + r.randrange(case["own"])) for n in nq]
        nq[0], mine[0] = q, case["own"]
        return nq, [p + t for p, t in zip((_prefix(case)[g] for g in _member(case)), mine)]
    T = case["T"]
    if not case["ragged"]:
        return [q] * B, [T] * B
    r = random.Random(f"{B} {q} {T}")
    nq = [1 + r.randrange(q) for _ in range(B)]
    lens = [max(n, 1 + r.randrange(T)) for n in nq]
    nq[0], lens[0] = q, max(T, q)
    return nq, lens


def _sizes(case):
    """Sequences of every group."""
    G, B = case["G"], case["B"]
    cuts = sorted(random.Random(f"{G} {B}").sample(range(1, B), G - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [B])]


def _member(case):
    return [g for g, n in enumerate(_sizes(case)) for _ in range(n)]


def _prefix(case):
    """Shared tokens of every group: the first the longest, the others down to half of that."""
    r = random.Random(f"{case['G']} {case['P']}")
    return [case["P"]] + [case["P"] - r.randrange(case["P"] // 2 + 1) for _ in range(case["G"] - 1)]


def _pages(t):
    return (t + PAGE - 1) // PAGE


# ---------------------------------------------------------------- inputs

def _pool(gen, n_blocks):
    """A cache of latent rows with channel gains and a few outlying rows, quantized."""
    gain = torch.exp(0.5 * torch.randn(D, generator=gen, device="cuda"))
    x = torch.randn((n_blocks * PAGE, D), generator=gen, device="cuda") * gain
    x *= 1.0 + 1.5 * (torch.rand((n_blocks * PAGE, 1), generator=gen, device="cuda") < 0.01)
    s = torch.stack([x[:, :DL].abs().amax(1), x[:, DL:].abs().amax(1)], 1) / 448.0
    y = torch.cat([x[:, :DL] / s[:, :1], x[:, DL:] / s[:, 1:]], 1)
    return y.to(torch.float8_e4m3fn).view(torch.uint8), s


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "norm":
        n, w, t = case["n"], case["w"], TYPES[case["type"]]
        gain = torch.exp(0.5 * torch.randn(w, generator=gen, device="cuda"))
        rows = lambda by: (torch.randn((n, w), generator=gen, device="cuda") * by).to(t)  # noqa: E731
        # the layer's last product, and the stream that it is added to: some channels stand out there
        s = dict(op=op, case=case, x=rows(0.3), weight=1.0 + 0.1 * torch.randn(w, generator=gen, device="cuda"),
                 residual=rows(gain * (1.0 + 20.0 * (torch.rand(w, generator=gen, device="cuda") < 0.002))) if case["add"] else None,
                 codes=torch.zeros((n, w), dtype=torch.uint8, device="cuda"),
                 scales=torch.zeros((n, -(-w // (case["group"] or w))), device="cuda"))
        s["residual_out"] = torch.zeros_like(s["x"]) if case["add"] else None
        s["normed"] = torch.zeros_like(s["x"]) if case["normed"] else None
        return s
    B, H = case["B"], case["H"]
    nq, lens = _lens(case)
    if op == "window":
        shared, member = [0], [0] * B
    else:
        shared, member = _prefix(case), _member(case)
    # whole pages of a prefix are the group's, the others a sequence's own
    pages = [_pages(t) - shared[g] // PAGE for t, g in zip(lens, member)]
    n_blocks = sum(pages) + sum(p // PAGE for p in shared) + 3
    codes, scales = _pool(gen, n_blocks)
    order = torch.randperm(n_blocks, generator=gen, device="cuda").int()
    table = torch.full((B, max(_pages(t) for t in lens)), -1, dtype=torch.int32, device="cuda")
    at, common = 0, []
    for p in shared:
        common.append(order[at: at + p // PAGE])
        at += p // PAGE
    for b, g in enumerate(member):
        k = common[g].numel()
        table[b, :k] = common[g]
        table[b, k: k + pages[b]] = order[at: at + pages[b]]
        at += pages[b]
    rows = sum(nq) + case["pad"]
    start, first = [0], [0]
    for n in nq:
        start.append(start[-1] + n)
    s = dict(op=op, case=case, codes=codes, scales=scales, table=table, lens=_ints(lens), start=_ints(start),
             q_lat=torch.randn((rows, H, DL), generator=gen, device="cuda").bfloat16(),
             q_rope=torch.randn((rows, H, DR), generator=gen, device="cuda").bfloat16(),
             out=torch.zeros((rows, H, DL), dtype=torch.bfloat16, device="cuda"),
             lse=torch.zeros((rows, H), device="cuda") if case["lse"] else None)
    if op == "shared":
        for n in _sizes(case):
            first.append(first[-1] + n)
        s["group_start"], s["shared_len"] = _ints(first), _ints(shared)
    return s


# ---------------------------------------------------------------- plain forms

def _keys(s, table, t):
    """Latent and rope keys of the tokens t [n, m] of table rows [n, :], in 32 bits."""
    t = t.clamp(min=0, max=table.shape[1] * PAGE - 1)
    slot = table.long().clamp(min=0).gather(1, t // PAGE) * PAGE + t % PAGE
    x, sc = s["codes"][slot].view(torch.float8_e4m3fn).float(), s["scales"][slot]
    return x[..., :DL] * sc[..., :1], x[..., DL:] * sc[..., 1:]


def _parts(s, at, lat, rope, see):
    """The scores' maximum, the weights' sum and the weighted sum of keys of the queries of tokens at
    [n, k] over keys [n, m, :], see [n, k, m] of them."""
    H = s["case"]["H"]
    ql, qr = s["q_lat"][at].float().flatten(1, 2), s["q_rope"][at].float().flatten(1, 2)
    z = torch.baddbmm(ql @ lat.transpose(1, 2), qr, rope.transpose(1, 2)).mul_(SM_SCALE).unflatten(1, (at.shape[1], H))
    z.masked_fill_(~see[:, :, None, :], -math.inf)
    m = z.amax(-1, keepdim=True).clamp(min=-3e38)
    p = z.sub_(m).exp_()
    return m, p.sum(-1, keepdim=True), (p.flatten(1, 2) @ lat).unflatten(1, (at.shape[1], H))


def _rows_of(s):
    """Of every row of the queries: its sequence, its place there, and whether it is one's."""
    start = s["start"].long()
    r = torch.arange(s["q_lat"].shape[0], device="cuda")
    b = (torch.searchsorted(start, r, right=True) - 1).clamp(max=s["lens"].numel() - 1)
    return r, b, r - start[b], (r < start[-1])[:, None]


def _write(s, mine, m, den, o):
    s["out"].copy_(torch.where(mine[..., None], (o / den.clamp(min=1e-38)).bfloat16(), s["out"]))
    if s["lse"] is not None:
        s["lse"].copy_(torch.where(mine, (m + den.log())[..., 0], s["lse"]))


def _window(s):
    """Blocks of query tokens, each over the first tokens and the keys that its windows cover."""
    c, start, lens = s["case"], s["start"].long(), s["lens"].long()
    q, W = c["q"], c["W"]
    step = min(q, BLOCK)
    n_blk = -(-q // step)
    most = max(_lens(c)[1])
    sinks, span = min(c["S"], most), min(W + step - 1, most)
    i = torch.arange(n_blk * step, device="cuda").unflatten(0, (n_blk, step))
    pos = (lens - (start[1:] - start[:-1]))[:, None, None] + i            # [B, n_blk, step]
    lo = (pos[..., :1] - W + 1).clamp(min=sinks)
    near = lo + torch.arange(span, device="cuda")
    far = torch.arange(sinks, device="cuda").expand(*lo.shape[:2], sinks)
    t, pos = torch.cat([far, near], -1).flatten(0, 1), pos.flatten(0, 1)
    see = (t[:, None, :] <= pos[..., None]) & ((t[:, None, :] > pos[..., None] - W) | (t[:, None, :] < sinks))
    lat, rope = _keys(s, s["table"].repeat_interleave(n_blk, 0), t)
    at = (start[:-1, None, None] + i).clamp(max=s["q_lat"].shape[0] - 1).flatten(0, 1)
    m, den, o = _parts(s, at, lat, rope, see)
    r, b, k, mine = _rows_of(s)
    blk, k = b * n_blk + k.clamp(max=q - 1) // step, k.clamp(max=q - 1) % step
    _write(s, mine, m[blk, k], den[blk, k], o[blk, k])


def _shared(s):
    """The groups' tokens over the prefixes, every sequence's over the rest, and the two joined."""
    c, start, lens, first = s["case"], s["start"].long(), s["lens"].long(), s["group_start"].long()
    rows, nq = s["q_lat"].shape[0], start[1:] - start[:-1]
    P = (s["shared_len"].long() // PAGE) * PAGE
    r, b, k, mine = _rows_of(s)
    g = torch.searchsorted(first, b, right=True) - 1
    member = torch.searchsorted(first, torch.arange(lens.numel(), device="cuda"), right=True) - 1
    # the prefixes, a batch of groups padded to the largest
    lead = start[first[:-1]]
    most = int(c["q"]) * max(_sizes(c))
    at = (lead[:, None] + torch.arange(most, device="cuda")).clamp(max=rows - 1)
    t = torch.arange(max(_prefix(c)) // PAGE * PAGE, device="cuda").expand(c["G"], -1)
    lat, rope = _keys(s, s["table"][first[:-1]], t)
    m0, l0, o0 = _parts(s, at, lat, rope, (t < P[:, None])[:, None, :]) if t.shape[1] else (None, None, None)
    # the rest, a batch of sequences padded to the longest
    i = torch.arange(c["q"], device="cuda")
    t = P[member][:, None] + torch.arange(c["own"] + PAGE, device="cuda")
    lat, rope = _keys(s, s["table"], t)
    at = (start[:-1, None] + i).clamp(max=rows - 1)
    last = (lens - nq)[:, None] + i
    m1, l1, o1 = (x[b, k.clamp(max=c["q"] - 1)] for x in _parts(s, at, lat, rope, t[:, None, :] <= last[..., None]))
    if m0 is not None:
        j = (r - lead[g]).clamp(max=most - 1)
        m0, l0, o0 = m0[g, j], l0[g, j], o0[g, j]
        m = torch.maximum(m0, m1)
        f0, f1 = (m0 - m).exp(), (m1 - m).exp()
        m1, l1, o1 = m, l0 * f0 + l1 * f1, o0 * f0 + o1 * f1
    _write(s, mine, m1, l1, o1)


def _norm(s):
    c = s["case"]
    n, w, group = c["n"], c["w"], c["group"] or c["w"]
    x = s["x"].float()
    if c["add"]:
        x = x + s["residual"].float()
        s["residual_out"].copy_(x)
    y = x * (1.0 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()) * s["weight"]
    if c["normed"]:
        s["normed"].copy_(y)
    v = torch.nn.functional.pad(y, (0, -w % group)).unflatten(1, (-1, group))
    top = v.abs().amax(-1, keepdim=True)
    s["scales"].copy_(top[..., 0] / 448.0)
    v = (v * (448.0 / top)).clamp(-448.0, 448.0).flatten(1)[:, :w]
    s["codes"].copy_(v.to(torch.float8_e4m3fn).view(torch.uint8))


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "window":
        _window(s)
    elif s["op"] == "shared":
        _shared(s)
    else:
        _norm(s)
    return _outputs(s)


def _outputs(s):
    if s["op"] != "norm":
        return {"out": s["out"], "lse": s["lse"]} if s["lse"] is not None else {"out": s["out"]}
    got = {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]}
    return got | {k: s[k] for k in ("residual_out", "normed") if s[k] is not None}


def _run_own(s):
    import fp8_mla_latent_gb300 as kv
    c = s["case"]
    if s["op"] == "norm":
        kv.kv8_norm_quantize_rows(s["x"], s["weight"], EPS, residual=s["residual"], residual_out=s["residual_out"],
                                  normed=s["normed"], codes=s["codes"], scales=s["scales"], group=c["group"])
        return _outputs(s)
    args = (s["q_lat"], s["q_rope"], s["codes"], s["scales"], s["table"], s["lens"], s["start"])
    if s["op"] == "window":
        kv.mla_absorb_window_fp8_batch(*args, SM_SCALE, c["W"], c["S"], out=s["out"], lse=s["lse"])
    else:
        kv.mla_absorb_shared_fp8_batch(*args, SM_SCALE, s["group_start"], s["shared_len"], out=s["out"], lse=s["lse"])
    return _outputs(s)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "norm":
        n, w, b = case["n"], case["w"], torch.finfo(TYPES[case["type"]]).bits // 8
        moved = 1 + 2 * case["add"] + case["normed"]
        groups = -(-w // (case["group"] or w))
        return {"bytes": n * w * (b * moved + 1) + 4 * n * groups + 4 * w, "flops": 0}
    nq, lens = _lens(case)
    H = case["H"]
    if case["op"] == "window":
        W, S = case["W"], case["S"]
        seen = read = 0
        for n, T in zip(nq, lens):
            for p in range(T - n, T):
                seen += min(p + 1, W + min(S, max(0, p + 1 - W)))
            lo = max(0, T - n - W + 1)
            read += T - lo + min(S, lo)
    else:
        shared, member = _prefix(case), _member(case)
        seen = sum(n * T - n * (n - 1) // 2 for n, T in zip(nq, lens))
        whole = [p // PAGE * PAGE for p in shared]
        read = sum(T - whole[g] for T, g in zip(lens, member)) + sum(whole)
    rows = sum(nq) * H
    nbytes = ROW_BYTES * read + rows * (2 * D + 2 * DL + (4 if case["lse"] else 0)) + 4 * read // PAGE + 8 * case["B"]
    return {"bytes": nbytes, "flops": 2 * (D + DL) * H * seen}


# ---------------------------------------------------------------- in 64 bits

def _e4m3_values():
    """The 256 values of the format, from its definition (the two NaN codes are not used)."""
    v = []
    for byte in range(256):
        e, f = (byte >> 3) & 15, byte & 7
        mag = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v.append(-mag if byte & 128 else mag)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _exact_norm(case, s):
    t = s["x"].double()
    if case["add"]:
        t = t + s["residual"].double()
    y = t / torch.sqrt((t * t).sum(1, keepdim=True) / case["w"] + EPS) * s["weight"].double()
    codes, scales = torch.empty_like(y), s["scales"].double()
    group = case["group"] or case["w"]
    for k in range(scales.shape[1]):
        part = y[:, k * group: (k + 1) * group]
        scales[:, k] = part.abs().amax(1) / 448.0
        codes[:, k * group: (k + 1) * group] = part / scales[:, k: k + 1]
    got = {"codes": codes, "scales": scales}
    if case["add"]:
        got["residual_out"] = t
    if case["normed"]:
        got["normed"] = y
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    nq, lens = _lens(case)
    value = _e4m3_values()
    out, lse = s["out"].double(), None if s["lse"] is None else s["lse"].double()
    first = 0
    for b, (n, T) in enumerate(zip(nq, lens)):
        i = 0
        while i < n:
            j = min(n, i + 64)
            p = T - n + torch.arange(i, j, device="cuda")
            t = torch.arange(T, device="cuda")
            if case["op"] == "window":  # what some row of the block sees
                t = t[(t < case["S"]) | (t > T - n + i - case["W"])]
            t = t[t <= T - n + j - 1]
            slot = s["table"][b].long()[t // PAGE] * PAGE + t % PAGE
            row, sc = value[s["codes"][slot].long()], s["scales"][slot].double()
            key = torch.cat([row[:, :DL] * sc[:, :1], row[:, DL:] * sc[:, 1:]], 1)
            q = torch.cat([s["q_lat"][first + i: first + j], s["q_rope"][first + i: first + j]], -1).double()
            z = (q.flatten(0, 1) @ key.T).unflatten(0, (j - i, case["H"])) * SM_SCALE
            hide = t[None, :] > p[:, None]
            if case["op"] == "window":
                hide |= (t[None, :] <= p[:, None] - case["W"]) & (t[None, :] >= case["S"])
            z.masked_fill_(hide[:, None, :], -math.inf)
            x = torch.logsumexp(z, -1)
            out[first + i: first + j] = (torch.exp(z - x[..., None]).flatten(0, 1) @ key[:, :DL]).unflatten(0, (j - i, case["H"]))
            if lse is not None:
                lse[first + i: first + j] = x
            i = j
        first += n
    return {"out": out, "lse": lse} if lse is not None else {"out": out}
