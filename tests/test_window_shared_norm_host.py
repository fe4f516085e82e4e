"""Window attention, attention over shared prefixes and the quantizing norm, on the host: the C calls'
refusals and the binding's, workspace sizes, and what orders one kernel's accesses before another's."""
import ctypes
import os
import re
import types

import pytest
import torch

import fp8_mla_latent_gb300 as pkg
from fp8_mla_latent_gb300 import _lib

EINVAL, EALIGN, EUNSUPPORTED, EWORKSPACE = -1, -2, -3, -6
G = 1 << 20  # an aligned address that no refused call reads


class Call:
    """A C call with good arguments; each check changes some of them."""

    def __init__(self, name, **args):
        self.fn, self.args = getattr(pkg.lib(), name), args

    def __call__(self, **kw):
        a = dict(self.args, **kw)
        assert set(a) == set(self.args)
        return self.fn(*[ctypes.c_void_p(v) if k.startswith("p_") and v is not None else v for k, v in a.items()])


CHUNK = dict(p_ql=G, ql_t=512 * 16, ql_h=512, p_qr=G, qr_t=64 * 16, qr_h=64, p_codes=G, p_scales=G, p_table=G, p_lens=G,
             p_start=G, total=8, B=2, H=16, mb=4, bs=64, nb=8)
TAIL = dict(sm=0.1, p_out=G, p_lse=G, p_ws=G, ws=1 << 40, p_stream=None)
CALLS = [("mla_absorb_window_fp8_batch", dict(window=100, sinks=4), (100, 4)),
         ("mla_absorb_shared_fp8_batch", dict(p_groups=G, p_shared=G, groups=1, share=0, causal=1), (1,))]


@pytest.mark.parametrize("name,own,size", CALLS)
def test_attention_refuses_bad_arguments(name, own, size):
    f = Call(name, **CHUNK, **own, **TAIL)
    for k in ("p_ql", "p_qr", "p_codes", "p_scales", "p_table", "p_lens", "p_start", "p_out"):
        assert f(**{k: None}) == EINVAL, k
    for k in ("p_ql", "p_qr", "p_codes", "p_scales", "p_out"):
        assert f(**{k: G + 8}) == EALIGN, k
    for k in ("p_table", "p_lens", "p_start", "p_lse"):
        assert f(**{k: G + 2}) == EALIGN, k
    for k in ("ql_t", "ql_h", "qr_t", "qr_h"):
        assert f(**{k: 68}) == EALIGN and f(**{k: -64}) == EINVAL, k
    for kw in (dict(B=-1), dict(H=0), dict(H=1025), dict(mb=0), dict(mb=1 << 25), dict(nb=0), dict(total=-1),
               dict(total=(1 << 31) // 16), dict(total=1 << 62), dict(sm=0.0), dict(sm=-1.0), dict(sm=float("nan")),
               dict(sm=float("inf"))):
        assert f(**kw) == EINVAL, kw
    assert f(bs=128) == EUNSUPPORTED
    need = getattr(pkg.lib(), name + "_workspace_size")(2, 16, 8, 4, *size)
    assert need > 0 and f(ws=need - 1) == EWORKSPACE and f(p_ws=None) == EWORKSPACE
    assert f(p_ws=G + 128) == EALIGN
    assert f(B=0) == 0 and f(total=0) == 0  # nothing to do


def test_window_and_groups_are_refused():
    f = Call(CALLS[0][0], **CHUNK, **CALLS[0][1], **TAIL)
    for kw in (dict(window=0), dict(window=-5), dict(sinks=-1)):
        assert f(**kw) == EINVAL, kw
    f = Call(CALLS[1][0], **CHUNK, **CALLS[1][1], **TAIL)
    for kw in (dict(groups=-1), dict(p_groups=None), dict(p_shared=None), dict(share=2), dict(share=-1)):
        assert f(**kw) == EINVAL, kw
    assert f(p_groups=G + 2) == EALIGN and f(p_shared=G + 1) == EALIGN


@pytest.mark.parametrize("name,own,size", CALLS)
def test_workspace_sizes(name, own, size):
    f = getattr(pkg.lib(), name + "_workspace_size")
    assert f(1, 1, 1, 1, *size) >= 256
    for bad in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 1025, 1, 1), (1, 1, -1, 1), (1, 1, 1, 0), (1, 128, 1 << 24, 1)):
        assert f(*bad, *size) == -1
    with pytest.raises(ValueError):
        getattr(pkg, name + "_workspace_size")(1, 0, 1, 1, *size)
    # every kind of call: few rows a sequence and many, few sequences and many, short tables and long
    for B in (1, 3, 64, 5000):
        for H in (1, 16, 20, 64, 128, 1024):
            for q in (B, 3 * B, 40 * B):
                for mb in (1, 9, 512, 1 << 24):
                    assert 256 <= f(B, H, q, mb, *size) < 1 << 37, (B, H, q, mb)
    if len(size) == 2:
        assert f(1, 1, 1, 1, 0, 0) == -1 and f(1, 1, 1, 1, 1, -1) == -1
        assert f(4, 16, 4, 1 << 20, 2 ** 31 - 1, 2 ** 31 - 1) > 0
    else:
        assert f(1, 1, 1, 1, -1) == -1 and f(1, 1, 1, 1, 0) > 0


def norm_call():
    return Call("kv8_norm_quantize_rows", p_x=G, xs=100, p_r=G, rs=100, p_ro=G, ros=100, p_w=G, eps=1e-6, n=3, w=100, t=0, g=0,
                p_y=G, ys=100, p_c=G, cs=100, p_s=G, p_stream=None)


def test_norm_refuses_bad_arguments():
    f = norm_call()
    for k in ("p_x", "p_w", "p_c", "p_s", "p_r"):  # (residual_out without residual)
        assert f(**{k: None}) == EINVAL, k
    for kw in (dict(n=-1), dict(w=0), dict(t=-1), dict(t=3), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(xs=-1), dict(rs=-1), dict(ros=99), dict(ys=99), dict(cs=99)):
        assert f(**kw) == EINVAL, kw
    for kw in (dict(g=1), dict(g=16), dict(g=100), dict(g=512), dict(g=-32), dict(n=1 << 31)):
        assert f(**kw) == EUNSUPPORTED, kw
    assert f(w=32769, xs=32769, rs=32769, ros=32769, ys=32769, cs=32769) == EUNSUPPORTED
    for k in ("p_x", "p_r", "p_ro", "p_y"):
        assert f(**{k: G + 1}) == EALIGN and f(**{k: G + 2}, t=2) == EALIGN, k
    for k in ("p_w", "p_s"):
        assert f(**{k: G + 2}) == EALIGN, k
    assert f(n=0) == 0
    # results over the rows that are read, or over one another
    apart = dict(p_x=G, p_r=2 * G, p_ro=3 * G, p_y=4 * G, p_c=5 * G, p_s=6 * G, p_w=7 * G)
    for kw in (dict(p_ro=G, xs=101), dict(p_ro=2 * G, ros=101), dict(p_y=G, ys=101), dict(p_y=2 * G, rs=104), dict(p_y=3 * G)):
        assert f(**{**apart, **kw}) == EINVAL, kw


# ------------------------------------------------------------------ the binding

STREAM = types.SimpleNamespace(cuda_stream=0)


class Reached(Exception):
    pass


class NoLibrary:
    def __getattr__(self, name):
        if name.endswith("_workspace_size"):
            return lambda *a: 1 << 16

        def call(*a):
            raise Reached(name)
        return call


@pytest.fixture
def host_as_device(monkeypatch):
    monkeypatch.setattr(_lib, "_is_device", lambda t: True)
    monkeypatch.setattr(_lib, "lib", lambda: NoLibrary())


def z(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype)


def variants(fn, good, bad):
    """The good arguments reach the library; each change in `bad` is refused by name."""
    with pytest.raises(Reached):
        fn(**good, stream=STREAM)
    for name, change in bad:
        with pytest.raises((ValueError, TypeError), match=name):
            fn(**{**good, **change}, stream=STREAM)


BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def attention():
    return dict(q_lat=z(6, 4, 512, dtype=BF), q_rope=z(6, 4, 64, dtype=BF), kv_codes=z(256, 576, dtype=U8),
                kv_scales=z(256, 2, dtype=F32), block_table=z(2, 2), seq_lens=z(2), q_start=z(3), sm_scale=0.1)


COMMON = [("q_lat", dict(q_lat=z(6, 4, 512, dtype=F32))), ("q_lat", dict(q_lat=z(6, 4, 576, dtype=BF))), ("q_lat", dict(q_lat=None)),
          ("q_rope", dict(q_rope=z(6, 5, 64, dtype=BF))), ("kv_codes", dict(kv_codes=z(256, 512, dtype=U8))),
          ("kv_codes", dict(kv_scales=z(255, 2, dtype=F32))), ("block_table", dict(block_table=z(2, 2, dtype=torch.int64))),
          ("seq_lens", dict(seq_lens=z(3))), ("q_start", dict(q_start=z(2))), ("out", dict(out=z(5, 4, 512, dtype=BF))),
          ("lse", dict(lse=z(6, 5, dtype=F32))), ("workspace", dict(workspace=z(100, 4)[:, :2]))]


def test_binding_window(host_as_device):
    variants(pkg.mla_absorb_window_fp8_batch, dict(attention(), window=5, n_sink=2), COMMON + [
        ("window", dict(window=0)), ("window", dict(window=2 ** 31)), ("n_sink", dict(n_sink=-1)),
        ("n_sink", dict(n_sink=2 ** 31))])


def test_binding_shared(host_as_device):
    variants(pkg.mla_absorb_shared_fp8_batch, dict(attention(), group_start=z(2), shared_len=z(1)), COMMON + [
        ("group_start", dict(group_start=z(3))), ("group_start", dict(group_start=z(2, dtype=torch.int64))),
        ("shared_len", dict(shared_len=z(1, dtype=torch.int64))), ("group_start", dict(group_start=None)),
        ("shared_len", dict(shared_len=z(2, 1)[:, 0].expand(2)[::2].reshape(1, 1)))])


def test_binding_norm(host_as_device):
    good = dict(x=z(3, 100, dtype=BF), norm_weight=z(100, dtype=F32), eps=1e-6, residual=z(3, 100, dtype=BF))
    variants(pkg.kv8_norm_quantize_rows, good, [
        ("x", dict(x=z(3, 100, dtype=torch.float64))), ("x", dict(x=z(100, dtype=BF))), ("x", dict(x=z(3, 0, dtype=BF))),
        ("x", dict(x=z(100, 3, dtype=BF).t())), ("residual", dict(residual=z(3, 100, dtype=F32))),
        ("residual", dict(residual=z(3, 99, dtype=BF))), ("residual_out", dict(residual_out=z(2, 100, dtype=BF))),
        ("residual_out", dict(residual=None, residual_out=z(3, 100, dtype=BF))), ("normed", dict(normed=z(3, 100, dtype=F32))),
        ("codes", dict(codes=z(3, 100, dtype=torch.int8))), ("codes", dict(codes=z(3, 101, dtype=U8))),
        ("norm_weight", dict(norm_weight=z(99, dtype=F32))), ("norm_weight", dict(norm_weight=z(100, dtype=BF))),
        ("group", dict(group=16)), ("group", dict(group=-1)), ("scales", dict(scales=z(3, 2, dtype=F32))),
        ("scales", dict(group=64, scales=z(3, 1, dtype=F32)))])
    wide = z(3, 140, dtype=BF)
    with pytest.raises(Reached):  # rows of a wider array, and one row for all
        pkg.kv8_norm_quantize_rows(wide[:, 7:107], good["norm_weight"], 0.0, residual=wide[:1, :100].expand(3, 100), stream=STREAM)


# ------------------------------------------------------------------ order

CSRC = os.path.join(os.path.dirname(os.path.abspath(pkg.__file__)), "csrc")


def source(name):
    """The file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(text, kernel):
    at = text.index(kernel + "(const ChunkArgs")
    return text[at: text.index("\n}", at)]


def test_the_join_reads_nothing_before_its_wait():
    b = body(source("chunk_work.cuh"), "parts_join_kernel")
    before = b[b.index("{"): b.index("grid_dependency_wait()")]
    assert "ps." not in before and "a." not in before and "return" not in before


def test_few_rows_beside_a_prefix_begin_behind_the_plans_and_end_behind_the_prefix():
    """Its kernel runs while the prefixes' does: it reads the plan behind the word that one sets (once, no
    loop), which is everywhere before that one lets it come, and waits for that one before it ends."""
    b = body(source("rows.cu"), "rows_kernel")
    first = b.index("ps.plan")
    assert 0 < b.index("load_acquire(ready)") < first and b.count("load_acquire(") == 1
    assert "grid_dependency_wait()" in b[b.index("MODE != kShared"):]
    early = b[b.index("if (!__syncthreads_and("): b.index("grid_dependents_launch();\n  }")]
    assert "grid_dependency_wait();\n      return;" in early, "a CTA without work waits as well"
    assert b.rstrip().endswith("if constexpr (MODE == kShared) grid_dependency_wait();")
    c = body(source("chunk.cu"), "chunk_kernel")
    part = c[c.index("store_release(&ws.plan->ready"): c.index("grid_dependents_launch()")]
    assert c.index("grid_dependency_wait()") < c.index("store_release(")
    assert re.search(r"__threadfence\(\);\s*}\s*__syncthreads\(\);", part)
