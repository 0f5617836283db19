"""Refusals of the paged latent cache's entry points (no GPU needed): bad
arguments return synchronously, before any CUDA call, with the status the
header documents."""
import ctypes
import os

import pytest
import torch

import gated_delta_rule_88_b200 as kda
from gated_delta_rule_88_b200 import build as kbuild

FAKE = 0x10000  # a 16-byte aligned fake device address; never dereferenced
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


def attn(lib, *, q=FAKE, cache=FAKE, table=FAKE, lens=FAKE, cu=None, out=FAKE, lse=None, T=4, H=2, dk=576, dv=512, N=2,
         pages=8, psize=64, mp=4, ps=0, scale=1.0, flags=0, dtype=1):
    return lib.kda_latent_attn(P(q), P(cache), P(table), P(lens), P(cu), P(out), P(lse), T, H, dk, dv, N, pages, psize,
                               mp, ps, scale, flags, dtype, None)


def append(lib, *, kv=FAKE, cache=FAKE, table=FAKE, lens=FAKE, cu=None, q_pe=FAKE, q=FAKE, freqs=FAKE, T=4, H=2,
           dk=576, rot=64, N=2, pages=8, psize=64, mp=4, ps=0, kvs=0, ts=0, hs=0, flags=0, scale=1.0, dtype=1):
    return lib.kda_latent_append(P(kv), P(cache), P(table), P(lens), P(cu), P(q_pe), P(q), P(freqs), T, H, dk, rot, N,
                                 pages, psize, mp, ps, kvs, ts, hs, flags, scale, dtype, None)


def rope(lib, *, x=FAKE, pos=FAKE, freqs=FAKE, out=FAKE, T=4, H=2, d=128, rot=64, offset=64, xs=0, os=0, flags=0,
         scale=1.0, dtype=1):
    return lib.kda_rope(P(x), P(pos), P(freqs), P(out), T, H, d, rot, offset, xs, os, flags, scale, dtype, None)


def copy(lib, *, pool=FAKE, src=FAKE, dst=FAKE, count=2, planes=1, pages=4, nbytes=64):
    return lib.kda_pages_copy(P(pool), P(src), P(dst), count, planes, pages, nbytes, None)


def compact(lib, *, pool=FAKE, pages=FAKE, new=FAKE, count=2, planes=1, n=4, nbytes=64):
    return lib.kda_pages_compact(P(pool), P(pages), P(new), count, planes, n, nbytes, None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw", [
    dict(q=0), dict(cache=0), dict(table=0), dict(lens=0), dict(out=0), dict(T=-1), dict(H=0), dict(dk=0), dict(N=0),
    dict(pages=0), dict(mp=0), dict(T=5), dict(N=65536, T=65536), dict(H=65536), dict(dtype=2), dict(flags=1),
    dict(flags=16), dict(scale=NAN), dict(scale=INF), dict(scale=3e38), dict(q=FAKE + 8), dict(cache=FAKE + 8), dict(out=FAKE + 4),
    dict(lse=FAKE + 2), dict(table=FAKE + 1), dict(lens=FAKE + 2), dict(cu=FAKE + 2), dict(ps=64 * 576 - 8),
    dict(ps=64 * 576 + 4), dict(ps=-8), dict(mp=1 << 26), dict(T=1 << 30, H=4, N=1)])
def test_attn_bad_arguments_rejected(lib, kw):
    assert attn(lib, **kw) == 1
    assert b"kda_latent_attn" in lib.kda_last_error_message()


@pytest.mark.parametrize("kw", [dict(dtype=0), dict(psize=8), dict(psize=48), dict(psize=256), dict(dv=128, dk=192),
                                dict(dk=544), dict(dk=640), dict(dv=500, dk=500), dict(dk=448)])
def test_attn_unsupported_rejected(lib, kw):
    assert attn(lib, **kw) == 2


def test_attn_no_tokens_is_a_no_op(lib):
    assert attn(lib, T=0) == 0
    assert attn(lib, T=0, cu=FAKE) == 0


@pytest.mark.parametrize("kw", [
    dict(kv=0), dict(cache=0), dict(table=0), dict(lens=0), dict(q=0), dict(q_pe=0), dict(T=-1), dict(H=0), dict(dk=0),
    dict(N=0), dict(T=5), dict(rot=24), dict(rot=-16), dict(rot=592), dict(rot=0), dict(rot=1040, dk=2048),
    dict(dk=580), dict(kvs=568), dict(kvs=580), dict(ts=100), dict(hs=60), dict(hs=72 + 4), dict(ts=32), dict(hs=32),
    dict(flags=32), dict(flags=1), dict(scale=INF), dict(scale=NAN), dict(dtype=-1), dict(kv=FAKE + 2),
    dict(cache=FAKE + 8), dict(q_pe=FAKE + 4), dict(q=FAKE + 8), dict(freqs=FAKE + 2), dict(ps=8), dict(ps=4),
    dict(H=65536)])
def test_append_bad_arguments_rejected(lib, kw):
    assert append(lib, **kw) == 1
    assert b"kda_latent_append" in lib.kda_last_error_message()


def test_append_unsupported_and_empty(lib):
    assert append(lib, psize=24) == 2
    assert append(lib, T=0) == 0
    assert append(lib, T=0, q=0, q_pe=0, freqs=0, rot=0) == 0


@pytest.mark.parametrize("kw", [
    dict(x=0), dict(pos=0), dict(freqs=0), dict(out=0), dict(T=-1), dict(H=0), dict(d=0), dict(T=1 << 31), dict(rot=0),
    dict(rot=24), dict(rot=144, d=128), dict(offset=72), dict(offset=-8), dict(offset=4), dict(d=100, offset=0),
    dict(rot=1040, d=2048, offset=0), dict(xs=128), dict(os=128), dict(xs=260), dict(os=-256), dict(flags=8),
    dict(flags=64), dict(scale=NAN), dict(dtype=3), dict(x=FAKE + 8), dict(out=FAKE + 2), dict(pos=FAKE + 2),
    dict(freqs=FAKE + 1), dict(xs=512), dict(H=1 << 24, d=128),
    dict(d=65544, offset=0)])
def test_rope_bad_arguments_rejected(lib, kw):
    assert rope(lib, **kw) == 1
    assert b"kda_rope" in lib.kda_last_error_message()


def test_rope_no_tokens_is_a_no_op(lib):
    assert rope(lib, T=0) == 0


@pytest.mark.parametrize("kw", [dict(pool=0), dict(src=0), dict(dst=0), dict(count=-1), dict(count=4097), dict(planes=0),
                                dict(planes=65536), dict(pages=0), dict(nbytes=0), dict(nbytes=24), dict(nbytes=-16),
                                dict(pool=FAKE + 8), dict(src=FAKE + 2), dict(dst=FAKE + 1), dict(nbytes=1 << 35)])
def test_copy_bad_arguments_rejected(lib, kw):
    assert copy(lib, **kw) == 1
    assert b"kda_pages_copy" in lib.kda_last_error_message()


@pytest.mark.parametrize("kw", [dict(pool=0), dict(pages=0), dict(new=0), dict(count=-1), dict(count=(1 << 31) + 1),
                                dict(planes=0), dict(n=0), dict(n=524289), dict(nbytes=0), dict(nbytes=8),
                                dict(pool=FAKE + 4), dict(pages=FAKE + 2), dict(new=FAKE + 3)])
def test_compact_bad_arguments_rejected(lib, kw):
    assert compact(lib, **kw) == 1
    assert b"kda_pages_compact" in lib.kda_last_error_message()


def test_nothing_to_move_is_a_no_op(lib):
    assert copy(lib, count=0, src=0, dst=0) == 0
    assert compact(lib, count=0, pages=0, new=0) == 0


def test_bindings_refuse_cpu_tensors():
    x = torch.zeros(2, 4, 576, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: kda.kda_latent_attn(x, x, i.view(1, 2), i[:1]),
                 lambda: kda.kda_latent_append(x[:, 0], x, i.view(1, 2), i[:1]),
                 lambda: kda.kda_rope(x, i, torch.ones(8)),
                 lambda: kda.kda_pages_copy(x, i, i),
                 lambda: kda.kda_pages_compact(x, i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_shares_the_process_cxx_runtime():
    # a statically linked second copy of it crashes when it formats a message
    with open(os.path.join(os.path.dirname(kda.library_path), "_paged.so"), "rb") as f:
        image = f.read()
    assert b"\0libstdc++.so.6\0" in image


def test_latent_attn_selftest_refuses(lib):
    args = [P(FAKE), P(FAKE), P(FAKE), P(FAKE), None, P(FAKE), None, 4, 2, 576, 512, 2, 8, 64, 4, 0, 1.0, 0, 1, None]
    assert lib.kda_selftest_latent_attn(P(0), *args[1:]) == 1
    assert b"kda_selftest_latent_attn" in lib.kda_last_error_message()
    args[9] = 512
    assert lib.kda_selftest_latent_attn(*args) == 2
