"""The norm with the residual's addition and an output in 8 bits, against its definition in 64 bits."""
import math

import pytest
import torch

import fp8_mla_latent_gb300 as pkg
from chunk_helpers import e4m3_values

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
EPS = 1e-6


def inputs(n, w, dtype, seed=0, add=True):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((n, w), generator=g) * 0.5).to(dtype).cuda()
    r = (torch.randn((n, w), generator=g) * torch.exp(torch.randn(w, generator=g))).to(dtype).cuda() if add else None
    return x, r, (1 + 0.2 * torch.randn(w, generator=g)).cuda()


def check(x, r, weight, codes, scales, group, t_out=None, normed=None, eps=EPS):
    """Every output within its roundings of the definition.  In f32 (u = 2^-24), t is off by u of itself.
    The sum of w squares is off by (w / n + 12) u of itself at most, for n threads that add up w / n squares
    each and ten steps between them, plus the squares' and t's 3 u; a thread holds at most 32 (and 64 in a
    warp's row), so 80 u; 1 / sqrt halves that, and what comes before it (1 / width, its product, eps: 3 u),
    and adds 4 u (two units in the last place); two products 2 u: y is off by e = 48 u.  A
    scale adds u; what is rounded to a code is off by 2 e + 3 u <= 100 u.  A rounding is half a step of its type."""
    u = 2.0 ** -24
    n, w = x.shape
    t = x.double() + (0 if r is None else r.double())
    y = t / torch.sqrt((t * t).mean(1, keepdim=True) + eps) * weight.double()
    if t_out is not None:
        half = torch.finfo(x.dtype).eps / 2
        assert ((t_out.double() - t).abs() <= (half + u) * t.abs() + 2.0 ** -25).all()
    if normed is not None:
        half = torch.finfo(x.dtype).eps / 2 if x.dtype != torch.float32 else 0
        assert ((normed.double() - y).abs() <= (half + 48 * u) * y.abs() + 2.0 ** -25).all()
    g = group or w
    pad = -w % g
    v = torch.nn.functional.pad(y, (0, pad)).unflatten(1, (-1, g))
    s = v.abs().amax(-1) / 448
    assert ((scales.double() - s).abs() <= 49 * u * s).all()
    q = (v / s.clamp(min=1e-300)[..., None]).flatten(1)[:, :w]
    got = e4m3_values("cuda")[codes.long()]
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    assert ((got - q).abs() <= step / 2 + 100 * u * q.abs()).all()
    assert (torch.signbit(got) == torch.signbit(q))[q != 0].all()


def call(x, r, weight, group=0, **kw):
    return pkg.kv8_norm_quantize_rows(x, weight, EPS, residual=r, group=group, **kw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("w", [1, 2, 7, 8, 31, 33, 64, 127, 128, 255, 256, 257, 511, 512, 520, 576, 1000, 1024, 1501, 2048,
                               4096, 7168, 8191, 8200, 16384, 16392, 32768])
def test_widths(w, dtype):
    for n, group, add in ((1, 0, True), (5, 128, True), (3, 32, False)):
        x, r, weight = inputs(n, w, dtype, seed=w, add=add)
        t, y = torch.empty_like(x), torch.empty_like(x)
        codes, scales = call(x, r, weight, group, residual_out=t if add else None, normed=y)
        check(x, r, weight, codes, scales, group, t if add else None, y)


@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("n,w", [(1, 100), (3, 257), (40, 640), (333, 1501), (400, 2056), (200, 7168)])
def test_groups_and_rows(n, w, group):
    x, r, weight = inputs(n, w, torch.bfloat16, seed=n)
    t = torch.empty_like(x)
    codes, scales = call(x, r, weight, group, residual_out=t)
    assert scales.shape == (n, -(-w // group) if group else 1)
    check(x, r, weight, codes, scales, group, t)


def test_many_rows():
    x, r, weight = inputs(20000, 72, torch.bfloat16)
    codes, scales = call(x, r, weight)
    check(x, r, weight, codes, scales, 0)


@pytest.mark.parametrize("w", [40, 512, 2000, 2001])
@pytest.mark.parametrize("dtype", TYPES)
def test_strided_rows_and_what_lies_between_them(w, dtype):
    """Rows of wider arrays, at 16-byte boundaries and at others; what lies between them stays as it is."""
    for off, gap in ((0, 64), (8, 40), (3, 13)):
        big = [torch.full((6, w + gap), 5.0, dtype=dtype, device="cuda") for _ in range(4)]
        codes = torch.full((6, w + gap), 99, dtype=torch.uint8, device="cuda")
        x, r, weight = inputs(6, w, dtype, seed=w + gap)
        part = [b[:, off: off + w] for b in big]
        part[0].copy_(x)
        part[1].copy_(r)
        got = call(part[0], part[1], weight, 64, residual_out=part[2], normed=part[3], codes=codes[:, off: off + w])
        check(x, r, weight, *got, 64, part[2], part[3])
        for b, v in [(b, 5.0) for b in big] + [(codes, 99)]:
            assert (b[:, :off] == v).all() and (b[:, off + w:] == v).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,w", [(153, 513), (400, 519), (1300, 1501), (700, 2047), (330, 7169), (200, 8191), (170, 8193),
                                 (160, 16383)])
def test_many_rows_of_odd_widths(n, w, dtype):
    """Rows behind one another, each at a place of its own; in parts of wider arrays at equal and at different
    places; and over the rows that are read.  Nothing but the rows is written."""
    for add in (True, False):
        x, r, weight = inputs(n, w, dtype, seed=w, add=add)
        t, y = (torch.empty_like(x) if add else None), torch.empty_like(x)
        want = call(x, r, weight, residual_out=t, normed=y)
        check(x, r, weight, *want, 0, t, y)
        for offs, gap, group in (((3, 3, 3, 3, 3), 11, 0), ((8, 8, 8, 8, 8), 32 + -w % 8, 128), ((1, 2, 3, 4, 5), 11, 64)):
            big = [torch.full((n, w + gap), 5.0, dtype=dtype, device="cuda") for _ in range(4)]
            codes = torch.full((n, w + gap), 99, dtype=torch.uint8, device="cuda")
            part = [b[:, o: o + w] for b, o in zip(big + [codes], offs)]
            part[0].copy_(x)
            if add:
                part[1].copy_(r)
            got = call(part[0], part[1] if add else None, weight, group, residual_out=part[2] if add else None,
                       normed=part[3], codes=part[4])
            check(x, r, weight, *got, group, part[2] if add else None, part[3])
            for b, o, v in zip(big + [codes], offs, (5.0, 5.0, 5.0, 5.0, 99)):
                assert (b[:, :o] == v).all() and (b[:, o + w:] == v).all()
        if add:
            x2, r2 = x.clone(), r.clone()
            got = call(x2, r2, weight, residual_out=r2, normed=x2)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert torch.equal(r2, t) and torch.equal(x2, y)


def test_nan_and_infinities_in_odd_rows_stay_in_them():
    x, r, weight = inputs(1000, 1501, torch.float16)
    clean = call(x, r, weight)
    x[7, 0], x[8, 1500], x[300, 750], r[999, 1500] = math.nan, math.inf, math.nan, math.nan
    got = call(x, r, weight)
    hit = torch.zeros(1000, dtype=torch.bool, device="cuda")
    hit[[7, 8, 300, 999]] = True
    assert (got[0][hit] & 0x7F == 0).all() and (got[1][hit] == 0).all()
    assert torch.equal(got[0][~hit], clean[0][~hit]) and torch.equal(got[1][~hit], clean[1][~hit])


def test_one_row_for_all():
    """A residual (or input) that is one row, read again for every row."""
    x, r, weight = inputs(9, 264, torch.bfloat16)
    one = r[:1].expand(9, 264)
    a, b = call(x, one, weight), call(x, one.contiguous(), weight)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("w", [1024, 1501])
def test_one_row_for_many_and_weights_at_an_odd_address(w):
    x, r, weight = inputs(400, w, torch.bfloat16)
    one = r[:1].expand(400, w)
    check(x, one, weight, *call(x, one, weight), 0)
    check(one, x, weight, *call(one, x, weight), 0)
    odd = torch.empty(w + 1, device="cuda")[1:].copy_(weight)
    t, y = torch.empty_like(x), torch.empty_like(x)
    check(x, r, weight, *call(x, r, odd, 128, residual_out=t, normed=y), 128, t, y)


@pytest.mark.parametrize("w", [64, 1000, 1001, 7168])
def test_in_place(w):
    x, r, weight = inputs(20, w, torch.bfloat16)
    t, y = torch.empty_like(x), torch.empty_like(x)
    want = call(x, r, weight, 128, residual_out=t, normed=y)
    x2, r2 = x.clone(), r.clone()
    got = call(x2, r2, weight, 128, residual_out=r2, normed=x2)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(r2, t) and torch.equal(x2, y)


def test_the_same_bits_each_time_and_beside_other_rows():
    """A row's outputs do not depend on its neighbours, at the same number of rows."""
    x, r, weight = inputs(64, 1536, torch.bfloat16)
    a = call(x, r, weight, 128)
    b = call(x, r, weight, 128)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x[1:], r[1:] = 3.0, -1.0
    c = call(x, r, weight, 128)
    assert torch.equal(a[0][0], c[0][0]) and torch.equal(a[1][0], c[1][0])


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("w", [256, 261, 3000])
def test_zeros_nan_and_infinities(w, group):
    x, r, weight = inputs(6, w, torch.float32)
    x[0], r[0] = 0.0, 0.0
    x[1, 5] = math.nan
    x[2, 7] = math.inf
    x[3], r[3] = 1e30, 1e30           # the sum of squares is over the range
    weight[3] = -0.0
    weight[200] = math.nan
    y = torch.empty_like(x)
    codes, scales = call(x, r, weight, group, normed=y)
    assert (codes[0, :3] == 0).all() and (scales[0] == 0).all()
    for k in (1, 2, 3):
        assert (codes[k] & 0x7F == 0).all() and (scales[k] == 0).all(), k
    assert torch.isnan(y[1]).all() and torch.isnan(y[2, 7])
    for k in (4, 5):                  # one column is NaN: code 0, not in the scale
        assert codes[k, 200] == 0 and torch.isfinite(scales[k]).all() and (scales[k] > 0).all()
        assert codes[k, 3] in (0, 0x80) and torch.isnan(y[k, 200])


def test_subnormal_maximum():
    """448 / amax is not finite: signed zeros, and the scale as computed."""
    x = torch.tensor([[1.0, -1.0, 0.0, 2.0] * 16], device="cuda")
    weight = torch.full((64,), 1e-39, device="cuda")
    codes, scales = call(x, None, weight)
    assert codes.flatten().tolist() == [0, 0x80, 0, 0] * 16
    assert 0 < float(scales) < 1e-41


@pytest.mark.parametrize("n", [3, 400])
def test_eps_of_zero(n):
    """A row of zeros has no norm: NaN in the normed row, codes and scale 0."""
    x, r, weight = inputs(n, 1024, torch.bfloat16)
    x[1] = r[1] = 0
    y = torch.empty_like(x)
    codes, scales = pkg.kv8_norm_quantize_rows(x, weight, 0.0, residual=r, normed=y)
    assert torch.isnan(y[1]).all() and (codes[1] == 0).all() and scales[1] == 0
    keep = torch.arange(n, device="cuda") != 1
    check(x[keep], r[keep], weight, codes[keep], scales[keep], 0, None, y[keep], eps=0.0)


@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("n,w,dtype", [(400, 7168, torch.bfloat16), (400, 8192, torch.float32), (200, 16384, torch.float16),
                                       (300, 520, torch.float32), (300, 16376, torch.bfloat16), (160, 1000, torch.float16)])
def test_many_rows_of_every_group_and_type(n, w, dtype, group):
    for add in (True, False):
        x, r, weight = inputs(n, w, dtype, seed=w + group, add=add)
        t, y = torch.empty_like(x), torch.empty_like(x)
        codes, scales = call(x, r, weight, group, residual_out=t if add else None, normed=y)
        check(x, r, weight, codes, scales, group, t if add else None, y)


@pytest.mark.parametrize("group", [0, 128])
def test_zeros_nan_and_infinities_among_many_rows(group):
    x, r, weight = inputs(400, 1024, torch.float32)
    x[0], r[0] = 0.0, 0.0
    x[1, 5] = math.nan
    x[2, 7] = math.inf
    x[3], r[3] = 1e30, 1e30
    x[4, 100] = 3e18                   # its square is in range, and the others far below it
    y = torch.empty_like(x)
    codes, scales = call(x, r, weight, group, normed=y)
    for k in (0, 1, 2, 3):
        assert (codes[k] & 0x7F == 0).all() and (scales[k] == 0).all(), k
    assert torch.isnan(y[1]).all() and torch.isnan(y[2, 7])
    check(x[4:], r[4:], weight, codes[4:], scales[4:], group, None, y[4:])
    weight[200], weight[300] = math.nan, math.inf
    codes, scales = call(x, r, weight, group, normed=y)
    assert (codes[4:, 200] == 0).all() and torch.isnan(y[4:, 200]).all()
    # an infinite y: its scale is infinite, and what it scales is 0
    assert torch.isinf(scales[5:, 300 // 128 if group else 0]).all()
    assert (codes[5:, 300] & 0x7F == 0).all()


def test_nothing_to_do():
    x, r, weight = inputs(0, 64, torch.bfloat16)
    codes, scales = call(x, r, weight)
    assert codes.shape == (0, 64) and scales.shape == (0, 1)


def test_captured():
    x, r, weight = inputs(7, 2048, torch.bfloat16)
    want = call(x, r, weight, 128)
    codes, scales = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(x, r, weight, 128, codes=codes, scales=scales)
    codes.zero_()
    g.replay()
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
