"""Host-side checks of the normalised rotary append, the block-scaled pages and
the logits processing that need no GPU: refusals of the C ABI before any
launch (made-up addresses, in a child process without a device), the scaled
rotary frequencies and tables against the oracle, and the binding's checks."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from paged_kv_gqa_append_gb300 import build as B

B.build()  # no-op when libpkv.so is up to date
import paged_kv_gqa_append_gb300 as pkv  # noqa: E402
from oracle import norm_rope as ON, rope as OR  # noqa: E402


@pytest.mark.parametrize("scaling", [None, "linear", "ntk", "yarn"])
@pytest.mark.parametrize("dim", [4, 22, 32, 64])
def test_scaled_frequencies(scaling, dim):
    for theta, factor, orig in ((10000.0, 4.0, 4096), (500000.0, 32.0, 8192), (10000.0, 1.0, 2048)):
        got, mul = pkv.pkv_rope_inv_freq_scaled(dim, theta, scaling, factor, orig)
        want, wmul = ON.inv_freq(dim // 2, theta, scaling, factor, orig)
        assert np.allclose(got, want, rtol=1e-14, atol=0) and mul == pytest.approx(wmul, rel=1e-15)


def test_scaled_tables_without_scaling_are_the_plain_ones():
    f, mul = pkv.pkv_rope_inv_freq_scaled(64, 500000.0)
    cos, sin = pkv.rope_tables_scaled_device("cpu", 300, f, mul)
    c, s = OR.table(OR.inv_freq_plain(500000.0), 300)
    assert np.array_equal(cos.numpy().view(np.uint32), c.view(np.uint32))
    assert np.array_equal(sin.numpy().view(np.uint32), s.view(np.uint32))
    cos2, _ = pkv.rope_tables_scaled_device("cpu", 300, f[:5], 1.5)
    assert np.array_equal(cos2.numpy(), (np.cos(np.arange(300.0)[:, None] * f[:5]) * 1.5).astype(np.float32))


@pytest.mark.parametrize("kw", [dict(rotary_dim=0), dict(rotary_dim=66), dict(rotary_dim=7), dict(scaling="other")])
def test_frequency_refusals_of_the_binding(kw):
    with pytest.raises(ValueError):
        pkv.pkv_rope_inv_freq_scaled(**kw)


@pytest.mark.parametrize("kw", [dict(theta=1.0), dict(theta=float("inf")), dict(scaling="linear", factor=0.5),
                                dict(scaling="yarn", factor=2.0, original_max_pos=0),
                                dict(scaling="yarn", factor=2.0, beta_fast=1.0, beta_slow=1.0),
                                dict(scaling="ntk", factor=2.0, rotary_dim=2),
                                dict(scaling="ntk", factor=float("nan"))])
def test_frequency_refusals_of_the_library(kw):
    with pytest.raises(pkv.PkvError):
        pkv.pkv_rope_inv_freq_scaled(**kw)


def test_cpu_tensors_are_refused():
    bf = torch.bfloat16
    k, pos = torch.zeros(2, 8, 64, dtype=bf), torch.zeros(2, dtype=torch.int32)
    tab = torch.zeros(4, 32)
    pool, sc = pkv.new_bs8_pool(3, "cpu")
    e4, _ = pkv.new_bs8_pool(3, "cpu", torch.float8_e4m3fn)
    assert pool.dtype == torch.int8 and e4.dtype == torch.float8_e4m3fn and sc.shape == (3, 2, 8)
    q, bt = torch.zeros(2, 32, 64, dtype=bf), torch.zeros(2, 1, dtype=torch.int32)
    for call in (lambda: pkv.qk_norm_rope(q, k, pos, tab, tab, q, k),
                 lambda: pkv.kv_append_norm_rope(k, k, pos, bt, torch.zeros(3, 2, 8, 16, 64, dtype=bf), tab, tab),
                 lambda: pkv.kv_append_rope_bs8(k, k, torch.arange(3, dtype=torch.int32), pos, bt, pool, sc),
                 lambda: pkv.kv_read_bs8(pool, sc, pos), lambda: pkv.process_logits(torch.zeros(2, 8)),
                 lambda: pkv.paged_gqa_decode_bs8(q, pool, sc, bt, pos, q, 1.0)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_host_side_validation_returns_before_launch():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", "import tests.test_ops_abi_cpu as t; t._checks()"], cwd=B.ROOT, env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr


def _checks():
    assert not torch.cuda.is_available()
    L, f, odd, none = pkv.lib, ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10002), None

    def nr(**kw):
        a = dict(q=f, qs=2048, k=f, ks=512, v=f, vs=512, qw=f, kw=f, wf=0, eps=1e-6, cos=f, sin=f, mp=64, pairs=32,
                 inter=0, pos=f, seq=none, T=2, bt=f, S=1, row=4, mb=4, pool=f, pages=8, qo=f, ko=none, err=none)
        a |= kw
        return L.kv_append_norm_rope(*a.values(), none)
    assert nr(T=0, q=none, k=none, v=none, qw=none, kw=none, qo=none) == 0
    for bad in (dict(T=-1), dict(mp=0), dict(pairs=0), dict(pairs=33), dict(inter=2), dict(wf=2), dict(k=none), dict(v=none),
                dict(pos=none), dict(cos=none), dict(bt=none), dict(S=0), dict(row=3), dict(pages=0), dict(qo=none),
                dict(q=none), dict(q=none, qo=none), dict(pool=none), dict(eps=-1.0), dict(eps=float("nan")),
                dict(qs=2040), dict(ks=504), dict(vs=0), dict(qw=none, eps=float("inf"))):
        assert nr(**bad) == 1, bad
    for bad in (dict(q=odd), dict(k=odd), dict(v=odd), dict(pool=odd), dict(qo=odd), dict(ko=odd), dict(cos=odd),
                dict(pos=odd), dict(bt=odd), dict(qs=2052), dict(ks=516), dict(vs=516), dict(err=odd), dict(wf=1, kw=odd),
                dict(kw=ctypes.c_void_p(0x10001))):
        assert nr(**bad) == 2, bad
    assert nr(T=(1 << 30) + 1) == 3

    def ap(**kw):
        a = dict(k=f, ks=512, v=f, vs=512, cu=f, lens=f, T=2, bt=f, S=1, row=4, mb=4, pool=f, sc=f, pages=8, code=0, cos=f,
                 sin=f, mp=64, q=f, qs=2048, qo=f, err=none)
        a |= kw
        return L.kv_append_rope_bs8(*a.values(), none)
    assert ap(T=0, k=none) == 0
    for bad in (dict(T=-1), dict(S=0), dict(row=3), dict(mb=0), dict(pages=0), dict(code=2), dict(cos=none), dict(q=none),
                dict(cos=none, sin=none), dict(mp=0), dict(k=none), dict(cu=none), dict(lens=none), dict(bt=none),
                dict(pool=none), dict(sc=none), dict(ks=0), dict(vs=8), dict(qs=0)):
        assert ap(**bad) == 1, bad
    for bad in (dict(k=odd), dict(v=odd), dict(q=odd), dict(qo=odd), dict(pool=odd), dict(cos=odd), dict(cu=odd),
                dict(sc=odd), dict(ks=513), dict(qs=2052), dict(err=odd)):
        assert ap(**bad) == 2, bad
    assert ap(mb=(1 << 26) + 1, row=(1 << 26) + 1) == 3 and ap(T=(1 << 29) + 1) == 3

    def rd(**kw):
        a = dict(pool=f, sc=f, pages=8, code=1, ids=f, n=3, out=f, err=none)
        a |= kw
        return L.kv_read_bs8(*a.values(), none)
    assert rd(n=0, pool=none) == 0
    assert [rd(n=-1), rd(pages=0), rd(code=3), rd(ids=none), rd(out=none)] == [1] * 5
    assert [rd(pool=odd), rd(out=odd), rd(ids=odd), rd(sc=odd)] == [2] * 4

    def dc(**kw):
        a = dict(q=f, pool=f, sc=f, pages=8, code=0, bt=f, row=4, mb=4, lens=f, S=2, ml=0, out=f, scale=0.125, ws=f,
                 wsb=1 << 30, err=none)
        a |= kw
        return L.paged_gqa_decode_bs8(*a.values(), none)
    assert dc(S=0, q=none) == 0
    for bad in (dict(S=-1), dict(pages=0), dict(code=-1), dict(row=3), dict(mb=0), dict(ml=-1), dict(scale=float("nan")),
                dict(q=none), dict(pool=none), dict(sc=none), dict(bt=none), dict(lens=none), dict(out=none), dict(ws=none)):
        assert dc(**bad) == 1, bad
    for bad in (dict(q=odd), dict(pool=odd), dict(sc=odd), dict(out=odd), dict(ws=odd), dict(bt=odd), dict(lens=odd)):
        assert dc(**bad) == 2, bad
    assert dc(S=4097) == 3
    assert L.paged_gqa_decode_bs8_workspace_bytes(4097) == 0

    def lg(**kw):
        a = dict(x=f, dtype=0, rows=2, vocab=100, stride=100, out=none, os=0, ids=f, h=f, hs=8, hl=f, pl=f, rep=f, pres=f,
                 freq=f, bi=f, bv=f, B=3, mask=f, ms=4)
        a |= kw
        return L.pkv_process_logits(*a.values(), none)
    assert lg(rows=0, x=none) == 0
    for bad in (dict(rows=-1), dict(vocab=0), dict(stride=99), dict(dtype=3), dict(B=-1), dict(ids=none), dict(x=none),
                dict(out=f, os=99), dict(h=none), dict(hl=none), dict(hs=0), dict(bi=none), dict(bv=none), dict(ms=3),
                dict(out=f, os=101), dict(out=f, os=100, dtype=1)):
        assert lg(**bad) == 1, bad
    for bad in (dict(x=odd), dict(ids=odd), dict(h=odd), dict(bv=odd), dict(mask=odd), dict(dtype=1, x=ctypes.c_void_p(0x10001)),
                dict(out=odd, os=100)):
        assert lg(**bad) == 2, bad
    assert lg(vocab=(1 << 30) + 1, stride=1 << 31, ms=1 << 30) == 3
    assert lg(B=(1 << 30) + 1) == 3 and lg(hs=(1 << 30) + 1) == 3
