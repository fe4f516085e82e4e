"""The chunk attention's and the pages' refusals, on the host: the C calls' own checks, and the
binding's.  The host model of the pages is pinned here as well."""
import ctypes
import types

import numpy as np
import pytest
import torch

import fp8_mla_latent_gb300 as pkg
from fp8_mla_latent_gb300 import _lib
from pages_ref import Pool

EINVAL, EALIGN, EUNSUPPORTED, EWORKSPACE = -1, -2, -3, -6
G = 1 << 20  # an aligned address that no refused call reads
MAX_SEQS, MAX_BLOCKS = 16384, 524288


def P(x):
    return None if x is None else ctypes.c_void_p(x)


class Call:
    """A C call with good arguments; each check changes some of them."""

    def __init__(self, name, **args):
        self.fn, self.args = getattr(pkg.lib(), name), args

    def __call__(self, **kw):
        a = dict(self.args, **kw)
        assert set(a) == set(self.args)
        return self.fn(*[P(v) if k.startswith("p_") else v for k, v in a.items()])


def chunk():
    return Call("mla_absorb_chunk_fp8_batch", p_ql=G, ql_t=512 * 16, ql_h=512, p_qr=G, qr_t=64 * 16, qr_h=64,
                p_codes=G, p_scales=G, p_table=G, p_lens=G, p_start=G, total=8, B=2, H=16, mb=4, bs=64, nb=8,
                causal=1, sm=0.1, p_out=G, p_lse=G, p_ws=G, ws=1 << 40, p_stream=None)


def test_chunk_refuses_bad_arguments():
    f = chunk()
    for k in ("p_ql", "p_qr", "p_codes", "p_scales", "p_table", "p_lens", "p_start", "p_out"):
        assert f(**{k: None}) == EINVAL, k
    for k in ("p_ql", "p_qr", "p_codes", "p_scales", "p_out"):
        assert f(**{k: G + 8}) == EALIGN, k
    for k in ("p_table", "p_lens", "p_start", "p_lse"):
        assert f(**{k: G + 2}) == EALIGN, k
    for k in ("ql_t", "ql_h", "qr_t", "qr_h"):
        assert f(**{k: 68}) == EALIGN and f(**{k: -64}) == EINVAL, k
    for kw in (dict(B=-1), dict(H=0), dict(H=1025), dict(mb=0), dict(mb=1 << 25), dict(nb=0), dict(total=-1),
               dict(total=(1 << 31) // 16), dict(sm=0.0), dict(sm=-1.0), dict(sm=float("nan")),
               dict(sm=float("inf"))):
        assert f(**kw) == EINVAL, kw
    assert f(bs=128) == EUNSUPPORTED
    need = pkg.lib().mla_absorb_chunk_fp8_batch_workspace_size(2, 16, 8, 4)
    assert need > 0
    assert f(ws=need - 1) == EWORKSPACE and f(p_ws=None) == EWORKSPACE
    assert f(p_ws=G + 128) == EALIGN
    assert f(B=0) == 0 and f(total=0) == 0  # nothing to do


def test_chunk_workspace_size():
    f = pkg.lib().mla_absorb_chunk_fp8_batch_workspace_size
    assert f(1, 1, 1, 1) >= 256
    for bad in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 1025, 1, 1), (1, 1, -1, 1), (1, 1, 1, 0), (1, 128, 1 << 24, 1)):
        assert f(*bad) == -1
    with pytest.raises(ValueError):
        pkg.mla_absorb_chunk_fp8_batch_workspace_size(1, 0, 1, 1)
    # more tokens of the same table never need less
    sizes = [f(4, 128, n, 64) for n in (1, 2, 5, 64, 1000, 16000)]
    assert sizes == sorted(sizes)


TABLE = dict(p_table=G, p_lens=G, p_refs=G, B=4, mb=8, nb=64)
TAIL = dict(p_err=G, p_stream=None)


def pages_calls():
    return [Call("kv8_pages_append", **TABLE, p_new=G, p_start=G, p_slot=G, cap=4, **TAIL),
            Call("kv8_pages_fork", **TABLE, p_src=G, p_dst=G, p_len=None, n=2, p_moves=G, p_n=G, **TAIL),
            Call("kv8_pages_free", **TABLE, p_seq=G, n=2, **TAIL),
            Call("kv8_pages_compact", **TABLE, p_moves=G, p_n=G, p_live=None, **TAIL)]


def test_pages_refuse_bad_tables():
    for f in pages_calls():
        for k in ("p_table", "p_lens", "p_refs"):
            assert f(**{k: None}) == EINVAL and f(**{k: G + 2}) == EALIGN
        assert f(p_err=G + 1) == EALIGN
        assert f(B=0) == EINVAL and f(mb=0) == EINVAL and f(mb=1 << 25) == EINVAL and f(nb=0) == EINVAL
        assert f(B=MAX_SEQS + 1) == EUNSUPPORTED and f(nb=MAX_BLOCKS + 1) == EUNSUPPORTED


def test_pages_refuse_bad_lists():
    append, fork, free, compact = pages_calls()
    for k in ("p_new", "p_start", "p_slot"):
        assert append(**{k: None}) == EINVAL
        assert append(**{k: G + 4 if k == "p_slot" else G + 2}) == EALIGN
    assert append(cap=-1) == EINVAL and append(cap=1 << 31) == EINVAL
    for k in ("p_src", "p_dst", "p_moves", "p_n"):
        assert fork(**{k: None}) == EINVAL and fork(**{k: G + 1}) == EALIGN
    assert fork(p_len=G + 2) == EALIGN
    assert fork(n=-1) == EINVAL and fork(n=MAX_SEQS + 1) == EUNSUPPORTED
    assert free(p_seq=None) == EINVAL and free(p_seq=G + 2) == EALIGN
    assert free(n=-1) == EINVAL and free(n=MAX_SEQS + 1) == EUNSUPPORTED and free(n=0, p_seq=None) == 0
    assert compact(p_moves=None) == EINVAL and compact(p_n=None) == EINVAL
    assert compact(p_moves=G + 2) == EALIGN and compact(p_n=G + 2) == EALIGN and compact(p_live=G + 2) == EALIGN


def test_copy_refuses_bad_arguments():
    f = Call("kv8_pages_copy", p_codes=G, p_scales=G, layers=2, slots=640, p_moves=G, p_n=G, n=5, **TAIL)
    for k in ("p_codes", "p_scales", "p_moves"):
        assert f(**{k: None}) == EINVAL
    assert f(p_codes=G + 8) == EALIGN and f(p_scales=G + 8) == EALIGN
    assert f(p_moves=G + 2) == EALIGN and f(p_n=G + 2) == EALIGN and f(p_err=G + 2) == EALIGN
    assert f(layers=0) == EINVAL and f(slots=63) == EINVAL and f(slots=641) == EINVAL
    assert f(n=-1) == EINVAL and f(n=1 << 31) == EINVAL
    assert f(slots=(MAX_BLOCKS + 1) * 64) == EUNSUPPORTED
    assert f(n=0, p_moves=None, p_codes=None) == 0


# ------------------------------------------------------------------ the binding

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


STREAM = types.SimpleNamespace(cuda_stream=0)


def z(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype)


def variants(fn, good, bad):
    """The good arguments reach the library; each change in `bad` is refused by name."""
    with pytest.raises(Reached):
        fn(**good, stream=STREAM)
    for name, change in bad:
        with pytest.raises((ValueError, TypeError), match=name):
            fn(**{**good, **change}, stream=STREAM)


def test_binding_chunk(host_as_device):
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    good = dict(q_lat=z(6, 4, 512, dtype=bf), q_rope=z(6, 4, 64, dtype=bf), kv_codes=z(256, 576, dtype=u8),
                kv_scales=z(256, 2, dtype=f32), block_table=z(2, 2), seq_lens=z(2), q_start=z(3), sm_scale=0.1)
    variants(pkg.mla_absorb_chunk_fp8_batch, good, [
        ("q_lat", dict(q_lat=z(6, 4, 512, dtype=f32))), ("q_lat", dict(q_lat=z(6, 4, 576, dtype=bf))),
        ("q_lat", dict(q_lat=z(6, 512, 4, dtype=bf).transpose(1, 2))), ("q_lat", dict(q_lat=None)),
        ("q_rope", dict(q_rope=z(6, 5, 64, dtype=bf))), ("q_rope", dict(q_rope=z(6, 4, 63, dtype=bf))),
        ("kv_codes", dict(kv_codes=z(256, 512, dtype=u8))), ("kv_codes", dict(kv_scales=z(255, 2, dtype=f32))),
        ("block_table", dict(block_table=z(2, 2, dtype=torch.int64))), ("seq_lens", dict(seq_lens=z(3))),
        ("q_start", dict(q_start=z(2))), ("out", dict(out=z(6, 4, 512, dtype=f32))),
        ("out", dict(out=z(5, 4, 512, dtype=bf))), ("lse", dict(lse=z(6, 5, dtype=f32))),
        ("workspace", dict(workspace=z(100, 4)[:, :2]))])
    # views of a wider array, and a size-1 dimension of any stride, are taken
    both = z(6, 4, 576, dtype=bf)
    with pytest.raises(Reached):
        pkg.mla_absorb_chunk_fp8_batch(**{**good, "q_lat": both[..., :512], "q_rope": both[..., 512:]}, stream=STREAM)
    assert _lib._strides(z(6, 1, 512, dtype=bf).as_strided((6, 1, 512), (512, 7, 1))) == (512, 0)


def test_binding_pages(host_as_device):
    table = dict(block_table=z(3, 4), seq_lens=z(3), page_refs=z(20))
    common = [("block_table", dict(block_table=z(3, 4, dtype=torch.int64))), ("seq_lens", dict(seq_lens=z(4))),
              ("page_refs", dict(page_refs=z(20, dtype=torch.int64))), ("err_word", dict(err_word=z(0))),
              ("err_word", dict(err_word=z(1, dtype=torch.int64))), ("block_table", dict(block_table=z(4, 3).t()))]
    variants(pkg.kv8_pages_append, dict(**table, n_new=z(3), cap=5), common + [
        ("n_new", dict(n_new=z(2))), ("q_start", dict(q_start=z(3))), ("dst_slot", dict(dst_slot=z(5))),
        ("dst_slot", dict(cap=None))])
    variants(pkg.kv8_pages_fork, dict(**table, src_seq=z(2), dst_seq=z(2)), common + [
        ("dst_seq", dict(dst_seq=z(3))), ("fork_len", dict(fork_len=z(1))), ("moves", dict(moves=z(1, 2))),
        ("moves", dict(moves=z(2, 3))), ("n_moves", dict(n_moves=z(0)))])
    variants(pkg.kv8_pages_free, dict(**table, seq=z(2)), common + [("seq", dict(seq=z(2, dtype=torch.int64)))])
    variants(pkg.kv8_pages_compact, table, common + [
        ("moves", dict(moves=z(9, 2))), ("n_live", dict(n_live=z(0))), ("n_moves", dict(n_moves=z(0)))])
    u8, f32 = torch.uint8, torch.float32
    variants(pkg.kv8_pages_copy, dict(kv_codes=z(128, 576, dtype=u8), kv_scales=z(128, 2, dtype=f32), moves=z(2, 2)), [
        ("kv_codes", dict(kv_codes=z(128, 575, dtype=u8))), ("kv_codes", dict(kv_scales=z(64, 2, dtype=f32))),
        ("kv_codes", dict(kv_codes=z(0, 128, 576, dtype=u8), kv_scales=z(0, 128, 2, dtype=f32))),
        ("kv_codes", dict(kv_codes=z(2, 128, 576, dtype=u8), kv_scales=z(1, 128, 2, dtype=f32))),
        ("moves", dict(moves=z(2, 3))), ("n_moves", dict(n_moves=z(0))), ("err_word", dict(err_word=z(0)))])
    with pytest.raises(Reached):
        pkg.kv8_pages_copy(z(2, 128, 576, dtype=u8), z(2, 128, 2, dtype=f32), z(2, 2), stream=STREAM)


# ------------------------------------------------------------------ the host model

def test_host_model_of_the_pages():
    p = Pool(4, 4, 10)
    q, s, err = p.append([65, 0, 3, 0], 70)
    assert err == 0 and list(q) == [0, 65, 65, 68, 68] and p.consistent()
    assert s[0] == 0 and s[63] == 63 and s[64] == 64 and s[65] == 128 and s[68] == -1
    moves, err = p.fork([0, 0], [1, 3], [65, 64])
    assert err == 0 and moves == [(1, 3)] and list(p.refs[:4]) == [3, 1, 1, 1] and p.consistent()
    assert p.append([0, 1, 0, 0], 1)[1][0] == 3 * 64 + 1
    assert p.free([0]) == 0 and list(p.refs[:4]) == [2, 0, 1, 1] and p.consistent()
    assert p.compact() == ([(3, 1)], 3) and p.consistent()
    assert list(p.table[1, :2]) == [0, 1]
    assert p.append([0, 0, 0, 1000], 2000)[2] == 2 and p.fork([1], [1])[1] == 1 and p.free([1, 1]) == 1
    before = p.copy()
    assert p.append([64 * 4, 64 * 4, 0, 0], 512)[2] == 2
    assert np.array_equal(before.refs, p.refs) and np.array_equal(before.table, p.table)
