"""Cases of window and shared-prefix attention and their definition in 64 bits, shared by the tests."""
import math

import torch

from chunk_helpers import DL, PAGE, SM_SCALE, Case, e4m3_values


class MaskCase(Case):
    """A chunk case whose rows see what sees() says."""

    def sees(self, b, causal=True):
        """[n, T]: the keys that the sequence's new tokens see."""
        return torch.arange(self.lens_list[b], device=self.device)[None, :] < self.limits(b, causal)[:, None]

    def reference(self, b, causal=True, sm_scale=SM_SCALE, keep=None):
        """As Case.reference, with its tolerances (derived there): the arithmetic of a row is the same
        whatever it sees.  Parts of a row joined by weights 2^(m - M) add an error of 2^-21 of the value
        (ex2's, and two f32 roundings), within the 2^-17 that the sum there is rounded up by."""
        n, T, H = self.nq[b], self.lens_list[b], self.H
        dev, first = self.device, int(self.start[b])
        see = self.sees(b, causal)
        if keep is not None:
            see = see & keep.to(dev)[None, :]
        q = torch.cat([self.q_lat[first: first + n], self.q_rope[first: first + n]], -1).double()
        out = torch.zeros((n, H, DL), dtype=torch.float64, device=dev)
        lse = torch.full((n, H), -math.inf, dtype=torch.float64, device=dev)
        tol, tol_l = torch.full_like(out, 1e-30), torch.full_like(lse, 2e-5)
        t = see.any(0).nonzero()[:, 0]
        if t.numel() == 0:
            return out, lse, tol, tol_l
        see = see[:, None, t]
        slot = self.slots[b].to(dev)[t]
        row, s = e4m3_values(dev)[self.codes[slot].long()], self.scales[slot].double()
        key = torch.cat([row[:, :DL] * s[:, :1], row[:, DL:] * s[:, 1:]], 1)
        z = (torch.einsum("nhd,td->nht", q, key) * sm_scale).masked_fill(~see, -math.inf)
        lse = torch.logsumexp(z, -1)
        some = see.any(-1).expand(n, H)
        p = torch.exp(z - torch.where(some, lse, 0.0)[..., None])
        out = torch.einsum("nht,td->nhd", p, key[:, :DL])
        mag = torch.einsum("nhd,td->nht", q.abs(), key.abs())
        ez = sm_scale * (2.0 ** -17 * q.abs().amax(-1)[..., None] * key.abs().sum(-1) + 2.0 ** -19 * mag)
        ez = torch.where(see, ez, 0.0).amax(-1)
        gmax = (p * s[:, 0]).amax(-1)
        each = torch.maximum((2.0 ** -9 + 3 * 2.0 ** -11 + 2.0 ** -17 + 2 * ez[..., None]) * p,
                             2.0 ** -17 * gmax[..., None] / s[:, 0].clamp(min=1e-300))
        tol = torch.einsum("nht,td->nhd", torch.where(see, each, 0.0), key[:, :DL].abs()) + 2.0 ** -8 * out.abs() + 1e-30
        return out, lse, tol, ez + 2e-5 * torch.where(some, lse, 0.0).abs().clamp(min=1.0)


class WindowCase(MaskCase):
    def __init__(self, H, nq, lens, window, sinks, **kw):
        self.window, self.sinks = window, sinks
        super().__init__(H, nq, lens, **kw)

    def sees(self, b, causal=True):
        n, T = self.nq[b], self.lens_list[b]
        t, p = torch.arange(T, device=self.device)[None, :], torch.arange(T - n, T, device=self.device)[:, None]
        return (t <= p) & ((t > p - self.window) | (t < self.sinks))


class SharedCase(MaskCase):
    """Groups of `sizes` consecutive sequences (the rest in no group) whose first shared[g] tokens are the
    same, the whole pages of them by the first member's table entries."""

    def __init__(self, H, nq, lens, sizes, shared, **kw):
        super().__init__(H, nq, lens, **kw)
        first, edge = 0, [0]
        table, codes, scales = self.table.cpu(), self.codes.cpu(), self.scales.cpu()
        for size, P in zip(sizes, shared):
            members = range(first, first + size)
            lead = max(members, key=lambda b: lens[b], default=0)
            for b in members:
                if b == lead:
                    continue
                m = min(max(P, 0), lens[b], lens[lead])
                k = m // PAGE
                table[b, :k] = table[lead, :k]
                i = torch.arange(lens[b])
                self.slots[b] = table[b].long()[i // PAGE] * PAGE + i % PAGE
                part = slice(k * PAGE, m)
                codes[self.slots[b][part]] = codes[self.slots[lead][part]]
                scales[self.slots[b][part]] = scales[self.slots[lead][part]]
            first += size
            edge.append(first)
        d = self.device
        self.table, self.codes, self.scales = table.to(d), codes.to(d), scales.to(d)
        self.group_start = torch.tensor(edge, dtype=torch.int32, device=d)
        self.shared_len = torch.tensor(shared, dtype=torch.int32, device=d)
