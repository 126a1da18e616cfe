"""Host-side checks of the 4-bit pages, the sampler and the page stack that need no
GPU: refusals of the C ABI before any launch (made-up addresses, in a child process
without a device), and of the binding."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from paged_kv_gqa_append_gb300 import build as B

B.build()  # no-op when libpkv.so is up to date
import paged_kv_gqa_append_gb300 as pkv  # noqa: E402
from oracle import int4_kv as O4  # noqa: E402


def test_block_bytes_agree():
    assert pkv.I4_BLOCK_BYTES == O4.BLOCK_BYTES
    pool = pkv.new_int4_pool(3, "cpu")
    assert pool.shape == (3, 8, 1152) and pool.dtype == torch.uint8 and not pool.any()
    ids, count = pkv.new_free_pages(4, "cpu")
    assert ids.tolist() == [3, 2, 1, 0] and count.tolist() == [4]


def test_cpu_tensors_are_refused():
    bf, i32 = torch.bfloat16, torch.int32
    k, pos = torch.zeros(2, 8, 64, dtype=bf), torch.zeros(2, dtype=i32)
    pool, q, bt = pkv.new_int4_pool(3, "cpu"), torch.zeros(2, 32, 64, dtype=bf), torch.zeros(2, 1, dtype=i32)
    x, one = torch.zeros(2, 8), torch.zeros(1, dtype=i32)
    for call in (lambda: pkv.kv_append_rope_int4(k, k, torch.arange(3, dtype=i32), pos, bt, pool), lambda: pkv.kv_read_int4(pool, pos),
                 lambda: pkv.paged_gqa_decode_int4(q, pool, bt, pos, q, 1.0), lambda: pkv.sample_logits(x, x),
                 lambda: pkv.grow_block_tables(pos, None, bt[None], pos, one),
                 lambda: pkv.release_pages(pos, pos > 0, bt[None], pos, one)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_host_side_validation_returns_before_launch():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", "import tests.test_more_ops_abi_cpu as t; t._checks()"], cwd=B.ROOT, env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr


def _checks():
    assert not torch.cuda.is_available()
    L, f, odd, none = pkv.lib, ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10002), None

    def caller(fn, defaults):
        return lambda **kw: fn(*(defaults | kw).values(), none)
    ap = caller(L.kv_append_rope_int4, dict(k=f, ks=512, v=f, vs=512, cu=f, lens=f, T=2, bt=f, S=1, row=4, mb=4, pool=f, pages=8,
                                            cos=f, sin=f, mp=64, q=f, qs=2048, qo=f, err=none))
    assert ap(T=0, k=none) == 0
    for bad in (dict(T=-1), dict(S=0), dict(row=3), dict(mb=0), dict(pages=0), dict(cos=none), dict(q=none),
                dict(cos=none, sin=none), dict(mp=0), dict(k=none), dict(cu=none), dict(lens=none), dict(bt=none),
                dict(pool=none), dict(ks=0), dict(vs=8), dict(qs=0)):
        assert ap(**bad) == 1, bad
    for bad in (dict(k=odd), dict(v=odd), dict(q=odd), dict(qo=odd), dict(pool=odd), dict(cos=odd), dict(cu=odd), dict(ks=513),
                dict(qs=2052), dict(err=odd)):
        assert ap(**bad) == 2, bad
    assert ap(mb=(1 << 26) + 1, row=(1 << 26) + 1) == 3 and ap(T=(1 << 29) + 1) == 3

    rd = caller(L.kv_read_int4, dict(pool=f, pages=8, ids=f, n=3, out=f, err=none))
    assert rd(n=0, pool=none) == 0
    assert [rd(n=-1), rd(pages=0), rd(ids=none), rd(out=none), rd(pool=none)] == [1] * 5
    assert [rd(pool=odd), rd(out=odd), rd(ids=odd), rd(err=odd)] == [2] * 4

    dc = caller(L.paged_gqa_decode_int4, dict(q=f, pool=f, pages=8, bt=f, row=4, mb=4, lens=f, S=2, ml=0, out=f, scale=0.125,
                                              ws=f, wsb=1 << 30, err=none))
    assert dc(S=0, q=none) == 0
    for bad in (dict(S=-1), dict(pages=0), dict(row=3), dict(mb=0), dict(ml=-1), dict(scale=float("nan")), dict(q=none),
                dict(pool=none), dict(bt=none), dict(lens=none), dict(out=none), dict(ws=none)):
        assert dc(**bad) == 1, bad
    for bad in (dict(q=odd), dict(pool=odd), dict(out=odd), dict(ws=odd), dict(bt=odd), dict(lens=odd), dict(err=odd)):
        assert dc(**bad) == 2, bad
    assert dc(S=4097) == 3 and dc(S=4096, mb=1 << 18, row=1 << 18) == 3
    assert L.paged_gqa_decode_int4_workspace_bytes(4097) == 0 and L.paged_gqa_decode_int4_workspace_bytes(-1) == 0

    sm = caller(L.pkv_sample_logits, dict(x=f, dtype=0, rows=2, vocab=100, stride=100, e=f, es=100, t=f, k=f, p=f, m=f, ids=f,
                                          lp=f))
    assert sm(rows=0, x=none) == 0
    for bad in (dict(rows=-1), dict(vocab=0), dict(stride=99), dict(es=99), dict(dtype=3), dict(dtype=-1), dict(x=none),
                dict(ids=none), dict(e=none, t=none)):
        assert sm(**bad) == 1, bad
    for bad in (dict(x=odd), dict(e=odd), dict(t=odd), dict(k=odd), dict(p=odd), dict(m=odd), dict(ids=odd), dict(lp=odd),
                dict(dtype=1, x=ctypes.c_void_p(0x10001))):
        assert sm(**bad) == 2, bad
    assert sm(vocab=(1 << 30) + 1, stride=1 << 31, es=1 << 31) == 3 and sm(rows=(1 << 27) + 1) == 3

    gr = caller(L.pkv_grow_block_tables, dict(lens=f, new=f, S=2, bt=f, layers=2, ls=8, row=4, mb=4, free=f, pages=8, count=f, lo=f,
                                              co=f, cu=f, pos=f, seq=f, slots=f, T=5, err=none))
    for bad in (dict(S=-1), dict(layers=0), dict(ls=7), dict(row=3), dict(mb=0), dict(pages=0), dict(T=-1), dict(lens=none),
                dict(bt=none), dict(free=none), dict(count=none), dict(lo=none), dict(co=none), dict(cu=none)):
        assert gr(**bad) == 1, bad
    for bad in (dict(lens=odd), dict(new=odd), dict(bt=odd), dict(free=odd), dict(count=odd), dict(lo=odd), dict(co=odd),
                dict(cu=odd), dict(pos=odd), dict(seq=odd), dict(slots=odd), dict(err=odd)):
        assert gr(**bad) == 2, bad
    assert gr(S=4097, ls=1 << 20) == 3 and gr(pages=1 << 27) == 3 and gr(T=(1 << 30) + 1) == 3
    assert gr(layers=1 << 20, mb=1 << 11, row=1 << 11, ls=1 << 20) == 3

    re = caller(L.pkv_release_pages, dict(lens=f, done=f, S=2, bt=f, layers=2, ls=8, row=4, mb=4, free=f, pages=8, count=f, lo=f,
                                          co=f, err=none))
    for bad in (dict(S=-1), dict(layers=0), dict(ls=7), dict(row=3), dict(mb=0), dict(pages=0), dict(lens=none), dict(done=none),
                dict(bt=none), dict(free=none), dict(count=none), dict(lo=none), dict(co=none)):
        assert re(**bad) == 1, bad
    for bad in (dict(lens=odd), dict(bt=odd), dict(free=odd), dict(count=odd), dict(lo=odd), dict(co=odd), dict(err=odd)):
        assert re(**bad) == 2, bad
    assert re(S=4097, ls=1 << 20) == 3 and re(pages=1 << 27) == 3
