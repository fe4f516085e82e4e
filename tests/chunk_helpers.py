"""Chunk attention cases and their definition in 64 bits, shared by the tests."""
import math

import numpy as np
import torch

DL, DR, D, PAGE = 512, 64, 576, 64
SM_SCALE = 1.0 / math.sqrt(192.0)


def e4m3_values(device):
    """The 256 values of the format from its definition (the two NaN codes give NaN)."""
    v = []
    for byte in range(256):
        e, f = (byte >> 3) & 15, byte & 7
        mag = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        if byte & 127 == 127:
            mag = math.nan
        v.append(-mag if byte & 128 else mag)
    return torch.tensor(v, dtype=torch.float64, device=device)


def quantized(x):
    """Codes and scales of rows x [n, 576], as the cache holds them."""
    s = torch.stack([x[:, :DL].abs().amax(1), x[:, DL:].abs().amax(1)], 1) / 448.0
    y = torch.cat([x[:, :DL] / s[:, :1].clamp(min=1e-38), x[:, DL:] / s[:, 1:].clamp(min=1e-38)], 1)
    return y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


class Case:
    """B sequences with nq[b] queries over lens[b] cached tokens, in pages of a random order;
    every byte of the pool that no sequence holds is a NaN code under a NaN scale."""

    def __init__(self, H, nq, lens, seed=0, device="cuda", pad=0, gains=0.5, rows=None, spare=3):
        g = torch.Generator().manual_seed(seed)
        self.H, self.nq, self.lens_list, self.device = H, list(nq), list(lens), device
        B = len(nq)
        pages = [(t + PAGE - 1) // PAGE for t in lens]
        self.max_blocks = max(max(pages), 1) + 1
        n_blocks = sum(pages) + spare
        order = torch.randperm(n_blocks, generator=g).int()
        table = torch.full((B, self.max_blocks), -1, dtype=torch.int32)
        codes = torch.full((n_blocks * PAGE, D), 0x7F, dtype=torch.uint8)
        scales = torch.full((n_blocks * PAGE, 2), math.nan)
        gain = torch.exp(gains * torch.randn(D, generator=g))
        at = 0
        self.slots = []
        for b, t in enumerate(lens):
            table[b, : pages[b]] = order[at: at + pages[b]]
            at += pages[b]
            i = torch.arange(t)
            slot = table[b].long()[i // PAGE] * PAGE + i % PAGE
            self.slots.append(slot)
            x = rows(b, t, g) if rows is not None else torch.randn((t, D), generator=g) * gain
            if t:
                codes[slot], scales[slot] = quantized(x)
        total = sum(nq) + pad
        self.q_lat = torch.randn((total, H, DL), generator=g).bfloat16().to(device)
        self.q_rope = torch.randn((total, H, DR), generator=g).bfloat16().to(device)
        self.codes, self.scales, self.table = codes.to(device), scales.to(device), table.to(device)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=device)
        self.start = torch.tensor(np.concatenate([[0], np.cumsum(nq)]), dtype=torch.int32, device=device)

    def limits(self, b, causal):
        n, T = self.nq[b], self.lens_list[b]
        lim = torch.arange(T - n + 1, T + 1) if causal else torch.full((n,), T)
        return lim.clamp(min=0).to(self.device)

    def reference(self, b, causal=True, sm_scale=SM_SCALE, keep=None):
        """(out, lse, tol_out, tol_lse) of sequence b in float64 (keep: which keys have a page).

        The tolerances follow the arithmetic that the call states.  A weight g_t = p_t sLc_t is
        held to 2^-9 (two e4m3 terms) plus 3 2^-11 (half a step of f16 is eps / 2 = 2^-11: of the
        value, of the factor between its page's reference and the row's, and of their product, which
        is what is split; (1 + 2^-9)(1 + 2^-11)^3 - 1 < 2^-9 + 3 2^-11 + 2^-17), or to 2^-17 of the
        row's largest where the second term runs out of bits; p_t moves by the score's error, the
        query's (2^-17 of its row's largest value) and the f32 sums' (2^-19 of the sum of
        magnitudes); out is rounded to bf16: half a step, torch.finfo(torch.bfloat16).eps / 2 = 2^-8 of
        the value (a step is 2^-7 of the binade's first value)."""
        n, T, H = self.nq[b], self.lens_list[b], self.H
        dev = self.device
        first = int(self.start[b])
        q = torch.cat([self.q_lat[first: first + n], self.q_rope[first: first + n]], -1).double()
        slot = self.slots[b].to(dev)
        row = e4m3_values(dev)[self.codes[slot].long()]
        s = self.scales[slot].double()
        key = torch.cat([row[:, :DL] * s[:, :1], row[:, DL:] * s[:, 1:]], 1)
        see = torch.arange(T, device=dev)[None, :] < self.limits(b, causal)[:, None]
        if keep is not None:
            see = see & keep.to(dev)[None, :]
        see = see[:, None, :].expand(n, H, T)
        key = torch.where(see.any(0).any(0)[:, None], key, 0.0)  # what nobody sees
        z = (torch.einsum("nhd,td->nht", q, key) * sm_scale).masked_fill(~see, -math.inf)
        some = see.any(-1)
        lse = torch.logsumexp(z, -1) if T else torch.full((n, H), -math.inf, dtype=torch.float64, device=dev)
        p = torch.exp(z - torch.where(some, lse, 0.0)[..., None])
        out = torch.einsum("nht,td->nhd", p, key[:, :DL])
        mag = torch.einsum("nhd,td->nht", q.abs(), key.abs())
        ez = sm_scale * (2.0 ** -17 * q.abs().amax(-1)[..., None] * key.abs().sum(-1) + 2.0 ** -19 * mag)
        ez = torch.where(see, ez, 0.0).amax(-1) if T else torch.zeros((n, H), dtype=torch.float64, device=dev)
        gmax = (p * s[:, 0]).amax(-1) if T else torch.zeros((n, H), dtype=torch.float64, device=dev)
        each = torch.maximum((2.0 ** -9 + 3 * 2.0 ** -11 + 2.0 ** -17 + 2 * ez[..., None]) * p,
                             2.0 ** -17 * gmax[..., None] / s[:, 0].clamp(min=1e-300))
        each = torch.where(see, each, 0.0)
        tol = torch.einsum("nht,td->nhd", each, key[:, :DL].abs()) + 2.0 ** -8 * out.abs() + 1e-30
        return out, lse, tol, ez + 2e-5 * torch.where(some, lse, 0.0).abs().clamp(min=1.0)

    def args(self):
        return (self.q_lat, self.q_rope, self.codes, self.scales, self.table, self.lens, self.start)

    def check(self, out, lse=None, causal=True, sm_scale=SM_SCALE, keep=None):
        """Compare with the reference, sequence by sequence; the worst error over tolerance."""
        worst = 0.0
        for b, n in enumerate(self.nq):
            if n == 0:
                continue
            first = int(self.start[b])
            ref, ref_l, tol, tol_l = self.reference(b, causal, sm_scale, None if keep is None else keep[b])
            got = out[first: first + n].double()
            assert torch.isfinite(got).all(), f"sequence {b}: non-finite output"
            r = float(((got - ref).abs() / tol).amax())
            assert r <= 1.0, f"sequence {b}: error {r:.3g} of the tolerance"
            worst = max(worst, r)
            empty = torch.isneginf(ref_l)
            assert (got[empty] == 0).all(), f"sequence {b}: a row that sees nothing is not 0"
            if lse is not None:
                gl = lse[first: first + n].double()
                assert torch.equal(torch.isneginf(gl), empty), f"sequence {b}: lse of empty rows"
                rl = ((gl - ref_l).abs() / tol_l)[~empty]
                assert rl.numel() == 0 or float(rl.amax()) <= 1.0, \
                    f"sequence {b}: lse error {float(rl.amax()):.3g} of the tolerance"
        return worst
