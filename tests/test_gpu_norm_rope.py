"""kv_append_norm_rope and qk_norm_rope against the FP64 oracle.

Tolerance of a bf16 result: half a step, 2^-8 of the value; plus the fp32
arithmetic in front of it.  The norm's sum of 64 squares, root, reciprocal and
two products are within 2^-18 of each y (a tree and a chain of at most 12
roundings, each 2^-24, on the sum, halved by the root; a few more behind it),
and the rotation adds two products and a sum, each within 2^-24 of |a| + |b|:
together below 2^-17 (|a| + |b|) f with f the tables' factor.
"""
import numpy as np
import pytest
import torch

from oracle import bf16 as OB, norm_rope as ON, rope as OR
from tests._util import bits, to_dev_bf16, to_dev_i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib(cuda_device):
    from paged_kv_gqa_append_gb300 import build
    build.build()
    import paged_kv_gqa_append_gb300 as m
    return m


def rows(seed, *shape, scale=1.0):
    g = np.random.default_rng(seed)
    return OB.from_f32_rne((scale * g.standard_normal(shape)).astype(np.float32))


def tables(lib, dev, pairs, max_pos, scaling=None, factor=1.0, orig=64):
    f, mul = lib.pkv_rope_inv_freq_scaled(2 * pairs, 10000.0, scaling, factor, orig)
    cos, sin = lib.rope_tables_scaled_device(dev, max_pos, f, mul)
    return cos, sin, mul


def want(x_bits, w, cos, sin, pos, inter, eps):
    y = ON.norm(OB.to_f64(x_bits), w, eps)
    c, s = cos[pos][:, None], sin[pos][:, None]
    f = np.sqrt((c[..., :1].astype(np.float64) ** 2 + s[..., :1].astype(np.float64) ** 2)).max()
    z = ON.rotate(y, c, s, inter)
    return z, 2.0 ** -8 * np.abs(z) + 2.0 ** -17 * max(f, 1.0) * ON.pair_sizes(y, c.shape[-1], inter) + 1e-38


def close(got, ref, tol, what):
    got = OB.to_f64(bits(got))
    assert np.isfinite(got).all(), what
    err = np.abs(got - ref) - tol
    assert (err <= 0).all(), f"{what}: {err.max():.3e} over at {np.unravel_index(err.argmax(), err.shape)}"


@pytest.mark.parametrize("T", [1, 3, 16, 77])
@pytest.mark.parametrize("pairs,inter", [(32, False), (32, True), (16, False), (8, False), (24, False), (1, False),
                                         (11, False), (4, True), (7, True), (31, False), (31, True)])
def test_qk_norm_rope_layouts(lib, cuda_device, T, pairs, inter):
    dev = cuda_device
    cos, sin, _ = tables(lib, dev, pairs, 300, "yarn", 4.0)
    pos = np.random.default_rng(T).integers(0, 300, T).astype(np.int32)
    q, k = rows(1, T, 32, 64, scale=3.0), rows(2, T, 8, 64)
    g = np.random.default_rng(5)
    qw, kw = OB.from_f32_rne(g.uniform(0.5, 2, 64).astype(np.float32)), OB.from_f32_rne(g.standard_normal(64).astype(np.float32))
    qo = torch.full((T, 32, 64), 7.0, dtype=torch.bfloat16, device=dev)
    ko = torch.full((T, 8, 64), 7.0, dtype=torch.bfloat16, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    for norm in (True, False):
        lib.qk_norm_rope(to_dev_bf16(q, dev), to_dev_bf16(k, dev), to_dev_i32(pos, dev), cos, sin, qo, ko,
                         q_weight=to_dev_bf16(qw, dev) if norm else None,
                         k_weight=to_dev_bf16(kw, dev) if norm else None, eps=1e-5, interleaved=inter, d_err=err)
        assert lib.pkv_read_device_error(err) == 0
        ch, sh = cos.cpu().numpy(), sin.cpu().numpy()
        close(qo, *want(q, OB.to_f64(qw) if norm else None, ch, sh, pos, inter, 1e-5), "q")
        close(ko, *want(k, OB.to_f64(kw) if norm else None, ch, sh, pos, inter, 1e-5), "k")


def test_float_weights_one_side_only_and_k_alone(lib, cuda_device):
    dev, T = cuda_device, 9
    cos, sin, _ = tables(lib, dev, 16, 64)
    ch, sh = cos.cpu().numpy(), sin.cpu().numpy()
    pos = np.arange(T, dtype=np.int32)
    q, k = rows(3, T, 32, 64), rows(4, T, 8, 64, scale=1e-3)
    kw = np.random.default_rng(6).standard_normal(64).astype(np.float32)
    qo, ko = torch.empty(T, 32, 64, dtype=torch.bfloat16, device=dev), torch.empty(T, 8, 64, dtype=torch.bfloat16, device=dev)
    args = (to_dev_i32(pos, dev), cos, sin)
    lib.qk_norm_rope(to_dev_bf16(q, dev), to_dev_bf16(k, dev), *args, qo, ko, k_weight=torch.from_numpy(kw).to(dev))
    close(qo, *want(q, None, ch, sh, pos, False, 1e-6), "q without a norm")
    close(ko, *want(k, kw, ch, sh, pos, False, 1e-6), "k")
    only = torch.empty_like(ko)
    lib.qk_norm_rope(None, to_dev_bf16(k, dev), *args, None, only, k_weight=torch.from_numpy(kw).to(dev))
    assert torch.equal(only.view(torch.int16), ko.view(torch.int16))


@pytest.mark.parametrize("fused", [False, True])
def test_append_into_pages(lib, cuda_device, fused):
    """One sequence's prompt in any token order and two decode tokens, from a
    fused projection's rows; only the tokens' slots change."""
    dev, T = cuda_device, 41
    cos, sin, _ = tables(lib, dev, 24, 64)
    ch, sh = cos.cpu().numpy(), sin.cpu().numpy()
    g = np.random.default_rng(8)
    pos = np.concatenate([g.permutation(39), [5, 63]]).astype(np.int32)
    seq = np.concatenate([np.zeros(39), [1, 2]]).astype(np.int32)
    bt = np.full((3, 7), -1, np.int32)
    bt[0, :3], bt[1, 0], bt[2, 3] = [5, 1, 3], 0, 8
    qkv = rows(9, T, 48, 64)
    q, k, v = qkv[:, :32], qkv[:, 32:40], qkv[:, 40:]
    kw = OB.from_f32_rne(g.standard_normal(64).astype(np.float32))
    d = to_dev_bf16(qkv, dev)
    parts = [d[:, :32], d[:, 32:40], d[:, 40:]] if fused else [to_dev_bf16(x, dev) for x in (q, k, v)]
    pool = torch.full((10, 2, 8, 16, 64), 3.5, dtype=torch.bfloat16, device=dev)
    qo, ko = (torch.empty(T, n, 64, dtype=torch.bfloat16, device=dev) for n in (32, 8))
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    lib.kv_append_norm_rope(parts[1], parts[2], to_dev_i32(pos, dev), to_dev_i32(bt, dev), pool, cos, sin,
                            token_seq=to_dev_i32(seq, dev), q_in=parts[0], q_out=qo, k_out=ko,
                            k_weight=to_dev_bf16(kw, dev), d_err=err, max_blocks=5)
    assert lib.pkv_read_device_error(err) == 0
    close(qo, *want(q, None, ch, sh, pos, False, 1e-6), "q")
    close(ko, *want(k, OB.to_f64(kw), ch, sh, pos, False, 1e-6), "k")
    expect = np.full((10, 2, 8, 16, 64), OB.from_f32_rne(np.float32(3.5)), np.uint16)
    for t in range(T):
        page, slot = bt[seq[t], pos[t] // 16], pos[t] % 16
        expect[page, 0, :, slot] = bits(ko)[t]
        expect[page, 1, :, slot] = v[t]
    assert np.array_equal(bits(pool), expect)


def test_without_weights_it_is_kv_append_rope_bit_for_bit(lib, cuda_device):
    dev, T = cuda_device, 130
    cos, sin = lib.rope_tables_device(dev, 256)
    k, v, q = rows(10, T, 8, 64), rows(11, T, 8, 64), rows(12, T, 32, 64)
    bt = np.random.default_rng(1).permutation(9).astype(np.int32)[None]
    pos, seq = np.arange(T, dtype=np.int32), np.zeros(T, np.int32)
    got = []
    for call in (lib.kv_append_rope, lib.kv_append_norm_rope):
        pool = torch.zeros((9, 2, 8, 16, 64), dtype=torch.bfloat16, device=dev)
        qd = to_dev_bf16(q, dev)
        call(to_dev_bf16(k, dev), to_dev_bf16(v, dev), to_dev_i32(pos, dev), to_dev_i32(bt, dev), pool, cos, sin,
             token_seq=to_dev_i32(seq, dev), q_in=qd, q_out=qd)     # in place
        got += [pool.view(torch.int16), qd.view(torch.int16)]
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])


def test_bad_tokens_are_skipped(lib, cuda_device):
    dev = cuda_device
    cos, sin, _ = tables(lib, dev, 32, 48)
    pos = np.array([0, -1, 48, 16, 32, 17, 2], np.int32)
    seq = np.array([0, 0, 0, 0, 0, 1, -1], np.int32)
    bt = np.array([[2, 9, -1]], np.int32)                 # page 9 is outside the pool
    k = to_dev_bf16(rows(13, 7, 8, 64), dev)
    q = to_dev_bf16(rows(14, 7, 32, 64), dev)
    pool = torch.zeros((4, 2, 8, 16, 64), dtype=torch.bfloat16, device=dev)
    qo, ko = torch.full_like(q, 9.0), torch.full_like(k, 9.0)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    lib.kv_append_norm_rope(k, k, to_dev_i32(pos, dev), to_dev_i32(bt, dev), pool, cos, sin,
                            token_seq=to_dev_i32(seq, dev), q_in=q, q_out=qo, k_out=ko, d_err=err)
    assert lib.pkv_read_device_error(err) == lib.ERR_DEVICE_INDEX
    assert (qo[1:] == 0).all() and (ko[1:] == 0).all() and torch.equal(qo[0], q[0])   # position 0 turns nothing
    assert torch.equal(pool[2, 0, :, 0], k[0]) and int((pool != 0).sum()) == 2 * int((k[0] != 0).sum())
    # without an append only the positions matter
    lib.qk_norm_rope(q, k, to_dev_i32(pos, dev), cos, sin, qo, ko, d_err=err)
    assert lib.pkv_read_device_error(err) == lib.ERR_DEVICE_INDEX
    assert (qo[1:3] == 0).all() and (qo[3:].float().abs().sum((1, 2)) > 0).all()


def test_many_tokens_equal_few(lib, cuda_device):
    """The form for many tokens (one warp per token) gives the bits of the one for few, in every layout, and
    reaches pages behind 4 GiB of the pool."""
    dev, T = cuda_device, 5000
    g = torch.Generator(dev).manual_seed(0)
    qkv = torch.randn(T, 48, 64, generator=g, device=dev).bfloat16()
    w = torch.randn(64, generator=g, device=dev)
    pool = torch.zeros((140000, 2, 8, 16, 64), dtype=torch.bfloat16, device=dev)     # 4.6 GB
    bt = torch.arange(140000 - 313, 140000, dtype=torch.int32, device=dev)[None]
    pos, seq = torch.arange(T, dtype=torch.int32, device=dev), torch.zeros(T, dtype=torch.int32, device=dev)
    for pairs, inter in ((32, False), (20, False), (9, False), (32, True), (13, True)):
        cos, sin, _ = tables(lib, dev, pairs, T)
        got = []
        for step in (T, 500):
            pool[-313:] = 0
            qo, ko = torch.zeros(T, 32, 64, dtype=torch.bfloat16, device=dev), torch.zeros(T, 8, 64, dtype=torch.bfloat16, device=dev)
            for t in range(0, T, step):
                x = qkv[t:t + step]
                lib.kv_append_norm_rope(x[:, 32:40], x[:, 40:], pos[t:t + step], bt, pool, cos, sin, token_seq=seq[t:t + step],
                                        q_in=x[:, :32], q_out=qo[t:t + step], k_out=ko[t:t + step], q_weight=w, k_weight=w,
                                        interleaved=inter)
            got.append((qo, ko, pool[-313:].clone()))
        for a, b in zip(*got):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        k = got[0][2].transpose(2, 3).reshape(313, 2, 16, 8, 64).transpose(0, 1).reshape(2, -1, 8, 64)[:, :T]
        assert torch.equal(k[0], got[0][1]) and torch.equal(k[1], qkv[:, 40:])
    assert not pool[:-313].any()


def test_zero_rows_and_no_tokens(lib, cuda_device):
    dev = cuda_device
    cos, sin, _ = tables(lib, dev, 32, 16)
    k = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device=dev)
    ko = torch.full_like(k, 1.0)
    w = torch.ones(64, device=dev)
    lib.qk_norm_rope(None, k, torch.arange(2, dtype=torch.int32, device=dev), cos, sin, None, ko, k_weight=w)
    assert (ko == 0).all()
    empty = torch.empty(0, 8, 64, dtype=torch.bfloat16, device=dev)
    lib.qk_norm_rope(None, empty, torch.empty(0, dtype=torch.int32, device=dev), cos, sin, None, empty)


def test_refusals(lib, cuda_device):
    dev = cuda_device
    cos, sin, _ = tables(lib, dev, 32, 16)
    k = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device=dev)
    pos = torch.zeros(2, dtype=torch.int32, device=dev)
    w = torch.ones(64, device=dev)

    def call(**kw):
        a = dict(q=None, k=k, positions=pos, rope_cos=cos, rope_sin=sin, q_out=None, k_out=torch.empty_like(k)) | kw
        lib.qk_norm_rope(**a)
    call()
    with pytest.raises(ValueError):
        call(k=k.cpu())
    with pytest.raises(ValueError):
        call(k_out=None)
    with pytest.raises(ValueError):
        call(q_weight=w)
    with pytest.raises(TypeError):
        call(k_weight=w.double())
    with pytest.raises(ValueError):
        call(k=torch.zeros(2, 64, 8, dtype=torch.bfloat16, device=dev).transpose(1, 2))
    with pytest.raises(ValueError):
        call(positions=pos[:1])
    with pytest.raises(ValueError):
        call(rope_cos=torch.zeros(16, 33, device=dev), rope_sin=torch.zeros(16, 33, device=dev))
    with pytest.raises(lib.PkvError):
        call(k_weight=w, eps=float("nan"))
    with pytest.raises(lib.PkvError):      # rows 513 elements apart are not 16-byte aligned
        call(k=torch.zeros(2 * 513, dtype=torch.bfloat16, device=dev).as_strided((2, 8, 64), (513, 64, 1)))
    with pytest.raises(lib.PkvError):      # one row twice
        call(k=k[:1].expand(2, 8, 64))
