"""Chunk attention over keys of very different weight: a bulk under a few keys far above it, in one
cluster's range of key tiles, against the definition in 64 bits for a few of the rows."""
import math

import pytest
import torch

import fp8_mla_latent_gb300 as pkg
from chunk_helpers import D, DL, DR, SM_SCALE, Case, e4m3_values

pytestmark = pytest.mark.gpu

TILE = 128


def run(c, causal=True, **kw):
    rows = c.q_lat.shape[0]
    ws = pkg.alloc_workspace(pkg.mla_absorb_chunk_fp8_batch_workspace_size(len(c.nq), c.H, rows, c.max_blocks))
    lse = torch.empty((rows, c.H), device="cuda")
    out = pkg.mla_absorb_chunk_fp8_batch(*c.args(), SM_SCALE, causal=causal, lse=lse, workspace=ws, **kw)
    assert pkg.kv8_workspace_error(ws) == 0
    return out, lse


def some_rows(c, tokens, heads, peaks):
    """The definition (out, its tolerance) of rows (token, head) of the one sequence of `c`, no mask.

    A weight g_t = p_t sLc_t is held to 2^-9 + 3 2^-11 + 2^-17 of itself, and p_t moves by twice the
    score's error (as chunk_helpers.Case.reference derives both).  In the tiles that hold a peak,
    and there alone, it may also be off by 2^-17 of the largest weight, or lost: never by more than
    itself, since rounding to the nearest step gives 0 or a step of at most twice the value.  Each
    other page's reference is its own, so nothing here grows with the number of keys.  out is
    rounded to bf16, by half a step: 2^-8 of the value."""
    slot = c.slots[0].cuda()
    row, s = e4m3_values("cuda")[c.codes[slot].long()], c.scales[slot].double()
    key = torch.cat([row[:, :DL] * s[:, :1], row[:, DL:] * s[:, 1:]], 1)
    q = torch.cat([c.q_lat, c.q_rope], -1)[tokens][:, heads].flatten(0, 1).double()
    z = q @ key.T * SM_SCALE
    p = torch.softmax(z, -1)
    out = p @ key[:, :DL]
    ez = SM_SCALE * (2.0 ** -17 * q.abs().amax(-1)[:, None] * key.abs().sum(-1) + 2.0 ** -19 * (q.abs() @ key.abs().T))
    near = torch.zeros(key.shape[0], dtype=torch.bool, device="cuda")
    for t in peaks:
        near[t // TILE * TILE: (t // TILE + 1) * TILE] = True
    top = (p * s[:, 0]).amax(-1, keepdim=True)
    lost = torch.minimum(p, 2.0 ** -17 * top / s[:, 0].clamp(min=1e-300)) * near
    each = (2.0 ** -9 + 3 * 2.0 ** -11 + 2.0 ** -17 + 2 * ez.amax(-1, keepdim=True)) * p + lost
    return out, each @ key[:, :DL].abs() + 2.0 ** -8 * out.abs() + 1e-30


def check_some(c, peaks, skip=0):
    out, _ = run(c, causal=False)
    tokens, heads = [0, 35, c.nq[0] - 1], [0, 1, 77, c.H - 1]
    ref, tol = some_rows(c, tokens, heads, peaks)
    got = out[tokens][:, heads].flatten(0, 1).double()
    worst = float(((got - ref).abs() / tol)[:, skip:].amax())
    assert worst <= 1.0, f"error {worst:.3g} of the tolerance"


@pytest.mark.parametrize("peaks", [(10, 266, 522, 778), (74, 330, 586, 842), (10, 202, 266, 458, 522, 30000, 50001),
                                   tuple(5 + 385 * i for i in range(12))])
def test_a_bulk_under_several_far_higher_keys(peaks):
    """Keys 17 to 20 binades above 65536 others whose values have a mean, as attention sinks are: a
    reference that comes down after each of them goes on coming down.  36 row tiles: every cluster
    has all keys of one."""
    def rows(b, t, g):
        x = torch.cat([0.5 + 0.3 * torch.randn((t, DL), generator=g), 0.05 * torch.randn((t, DR), generator=g)], 1)
        for k in peaks:
            x[k, :DL] = 0.1 * torch.randn(DL, generator=g)
            x[k, DL:] = 2.55
        return x
    c = Case(128, [72], [65536], seed=31, rows=rows)
    c.q_lat *= 0.02
    c.q_rope.copy_((1.0 + 0.15 * torch.arange(128, device="cuda") / 127)[None, :, None].expand_as(c.q_rope))
    check_some(c, peaks)


def test_a_bulk_under_rows_of_far_larger_scale():
    """The same by the rows' scales: rows 18 binades larger, in one channel alone."""
    peaks = (10, 266, 522, 778)

    def rows(b, t, g):
        x = torch.cat([0.5 + 0.1 * torch.randn((t, DL), generator=g), 0.1 * torch.randn((t, DR), generator=g)], 1)
        for k in peaks:
            x[k] = 0
            x[k, 0] = 2.0 ** 18
        return x
    c = Case(128, [72], [8192], seed=32, rows=rows)
    c.q_lat *= 0.1
    c.q_lat[..., 0] = 0
    check_some(c, peaks, skip=1)


@pytest.mark.parametrize("H,nq,T", [(128, 40, 3000), (16, 300, 9000), (128, 4, 30000)])
def test_same_bits_in_many_runs_with_other_work_between(H, nq, T):
    """Buffers that pass between the SMs of a cluster are overwritten only behind their reads: a
    value that came too early would show as another result now and then."""
    c = Case(H, [nq, 1], [T, 77], seed=33)
    want, want_l = run(c)
    ws = pkg.alloc_workspace(pkg.mla_absorb_chunk_fp8_batch_workspace_size(2, H, nq + 1, c.max_blocks))
    out, lse = torch.empty_like(want), torch.empty_like(want_l)
    noise, side = torch.randn((4096, 4096), device="cuda"), torch.cuda.Stream()
    for i in range(40):
        if i % 2:
            with torch.cuda.stream(side):
                noise.mul_(1.0001)
        out.fill_(float("nan"))
        pkg.mla_absorb_chunk_fp8_batch(*c.args(), SM_SCALE, out=out, lse=lse, workspace=ws)
        assert torch.equal(out, want) and torch.equal(lse, want_l)
    torch.cuda.synchronize()


@pytest.mark.parametrize("times", [64, 256, 512])
@pytest.mark.parametrize("part", ["rope", "latent"])
def test_queries_with_an_outlying_channel(part, times):
    """One channel of the query far above the others, which the two terms of its row's scale then
    hold to 2^-17 of it.  out and lse keep the call's stated bounds: a score is off by
    sm_scale (2^-17 max |q| sum |key| + 2^-19 sum |q key|) at most, lse by the largest of these and
    2e-5 of its size or of 1 (Case.reference has both, and what follows for out).  (2e-5 alone does
    not hold: at 64, 256 and 512 times lse was off by 2.8e-5, 7.1e-5 and 1.2e-4.)"""
    c = Case(16, [9, 40], [300, 1000], seed=34 + times)
    (c.q_rope if part == "rope" else c.q_lat)[..., 17] *= times
    out, lse = run(c)
    c.check(out, lse)


def test_a_negative_latent_scale_counts_as_none():
    """No call writes one: the row scale is a largest magnitude."""
    c = Case(16, [9, 3], [300, 200], seed=35)
    for b in (0, 1):
        slot = c.slots[b][::7].cuda()
        c.scales[slot, 0] = -c.scales[slot, 0]
    out, lse = run(c)
    c.scales[:, 0] = torch.where(c.scales[:, 0] < 0, 0.0, c.scales[:, 0])
    want, want_l = run(c)
    assert torch.equal(out, want) and torch.equal(lse, want_l)
    c.check(want, want_l)


@pytest.mark.parametrize("H,nq,lens", [(128, [4, 9, 1], [3000, 700, 5000]), (16, [1, 0, 3], [90, 5, 400])])
def test_same_bits_with_a_wider_table(H, nq, lens):
    """Columns that no sequence holds change the workspace and the launch, not the result."""
    c = Case(H, nq, lens, seed=36)
    want, want_l = run(c)
    for wide in (c.max_blocks + 1, 300, 5000):
        table = torch.full((len(nq), wide), -1, dtype=torch.int32, device="cuda")
        table[:, : c.max_blocks] = c.table
        d = Case(H, nq, lens, seed=36)
        d.table, d.max_blocks = table, wide
        out, lse = run(d)
        assert torch.equal(out, want) and torch.equal(lse, want_l)


@pytest.mark.parametrize("binades", [6.0, 9.0, 9.9, 10.1, 13.0, 30.0, 47.0, 60.0])
def test_a_weight_is_held_to_its_tiles_largest(binades):
    """A bulk of weights that vary little, under a key `binades` above them in every other tile of the
    first half: a weight is off by its own relative error, or by what the header allows beside it,
    the smaller of 2^-17 of the row's largest and 2^-7 of its tile's largest (while that is over
    2^-50 of the row's)."""
    def rows(b, t, g):
        x = torch.cat([0.5 + 0.3 * torch.randn((t, DL), generator=g), 0.02 * torch.randn((t, DR), generator=g)], 1)
        x[: t // 2: 2 * TILE] = torch.cat([0.1 * torch.randn(DL, generator=g), torch.full((DR,), binades / 16.99 * 2.55)])
        return x
    c = Case(128, [72], [8192], seed=37, rows=rows)
    c.q_lat *= 0.02
    c.q_rope.fill_(1.0)
    out, _ = run(c, causal=False)
    tokens, heads = [0, 35, 71], [0, 1, 77, 127]
    slot = c.slots[0].cuda()
    row, s = e4m3_values("cuda")[c.codes[slot].long()], c.scales[slot].double()
    key = torch.cat([row[:, :DL] * s[:, :1], row[:, DL:] * s[:, 1:]], 1)
    q = torch.cat([c.q_lat, c.q_rope], -1)[tokens][:, heads].flatten(0, 1).double()
    p = torch.softmax(q @ key.T * SM_SCALE, -1)
    ez = SM_SCALE * (2.0 ** -17 * q.abs().amax(-1)[:, None] * key.abs().sum(-1) + 2.0 ** -19 * (q.abs() @ key.abs().T))
    weight = p * s[:, 0]
    top, tile = weight.amax(-1, keepdim=True), weight.unflatten(1, (-1, TILE)).amax(-1).repeat_interleave(TILE, 1)
    other = torch.where(tile >= 2.0 ** -50 * top, torch.minimum(2.0 ** -17 * top, 2.0 ** -7 * tile), 2.0 ** -17 * top)
    each = torch.maximum((2.0 ** -9 + 3 * 2.0 ** -11 + 2.0 ** -17 + 2 * ez.amax(-1, keepdim=True)) * p, other / s[:, 0])
    ref = p @ key[:, :DL]
    tol = each @ key[:, :DL].abs() + 2.0 ** -8 * ref.abs() + 1e-30
    got = out[tokens][:, heads].flatten(0, 1).double()
    assert float(((got - ref).abs() / tol).amax()) <= 1.0
