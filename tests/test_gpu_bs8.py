"""Block-scaled 8-bit pages: kv_append_rope_bs8, kv_read_bs8 and
paged_gqa_decode_bs8 against the FP64 oracle.

Codes, scales and rotated q are compared bit for bit.  A decode output may be
off by its own rounding, 2^-8 of the value; by the rounding of the
probabilities to fp16, 2^-11 of sum p |v| / sum p =: A (the sum over p is not
rounded); and by fp32 arithmetic: a score is a sum of 64 exact products, off by
at most 2^-17 of scale sum |q| |k| =: R with its two scalings (64 + 3 steps of
2^-24), an exponential by 2^-21 more, each in numerator and denominator, so
2 (2^-17 R + 2^-21) A; the accumulation adds (n / 16 + 24) 2^-23 A.  A
probability enters the product as fp16 of 2^14 times it, whose least step is
2^-24: below 2^-28 of the largest the rounding is half that step, 2^-39 of the
largest probability, so n 2^-39 max |v| more (the sum is at least that one).
"""
import numpy as np
import pytest
import torch

from oracle import bf16 as OB, bs8_kv as O8, rope as OR
from tests._util import bits, to_dev_bf16, to_dev_i32

pytestmark = pytest.mark.gpu
KINDS = ["int8", "e4m3"]
TYPES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def lib(cuda_device):
    from paged_kv_gqa_append_gb300 import build
    build.build()
    import paged_kv_gqa_append_gb300 as m
    return m


@pytest.fixture(scope="module")
def tables(lib, cuda_device):
    cos_d, sin_d = lib.rope_tables_device(cuda_device, 600)
    cos_o, sin_o = OR.table(OR.inv_freq_llama3(), 600)
    return cos_d, sin_d, cos_o, sin_o


def rows(seed, *shape, scale=1.0):
    g = np.random.default_rng(seed)
    return OB.from_f32_rne((scale * g.standard_normal(shape)).astype(np.float32))


def random_pages(seed, pages, kind):
    g = np.random.default_rng(seed)
    codes = g.integers(0, 256, (pages, 2, 8, 16, 64)).astype(np.uint8)
    if kind == "int8":
        codes[codes == 0x80] = 0x81
    else:
        codes[(codes & 0x7F) == 0x7F] = 0x7E
    scales = np.exp(g.normal(-4 if kind == "int8" else -5, 0.7, (pages, 2, 8))).astype(np.float32)
    return codes, scales


def to_pool(codes, scales, kind, dev):
    return torch.from_numpy(codes.view(np.int8)).to(dev).view(TYPES[kind]), torch.from_numpy(scales).to(dev)


def pool_bytes(pool):
    return pool.view(torch.int8).cpu().numpy().view(np.uint8)


def tables_for(seed, lens, pages, width=None):
    g = np.random.default_rng(seed)
    need = [max(0, -(-int(n) // 16)) for n in lens]
    perm = g.permutation(pages).astype(np.int32)
    bt = np.full((len(lens), width or max(1, max(need))), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        bt[s, :n] = perm[at:at + n]
        at += n
    assert at <= pages
    return bt


# ------------------------------------------------------------------ append --

def append(lib, dev, kind, codes, scales, k, v, cu, lens, bt, rope=None, q=None, T=None):
    pool, sc = to_pool(codes, scales, kind, dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    kw = {}
    if rope is not None:
        kw = dict(rope_cos=rope[0], rope_sin=rope[1])
    if q is not None:
        kw |= dict(q_in=to_dev_bf16(q, dev), q_out=torch.zeros(q.shape, dtype=torch.bfloat16, device=dev))
    lib.kv_append_rope_bs8(to_dev_bf16(k, dev), to_dev_bf16(v, dev), to_dev_i32(cu, dev), to_dev_i32(lens, dev),
                           to_dev_i32(bt, dev), pool, sc, d_err=err, **kw)
    return pool, sc, kw.get("q_out"), lib.pkv_read_device_error(err)


def check_append(lib, dev, kind, codes, scales, k, v, cu, lens, bt, rope=None, q=None):
    cos, sin = (rope[2], rope[3]) if rope is not None else (None, None)
    want = O8.append(codes, scales, k, v, cu, lens, bt, kind, cos, sin, q)
    pool, sc, qo, code = append(lib, dev, kind, codes, scales, k, v, cu, lens, bt, rope, q)
    assert (code != 0) == want[3]
    assert np.array_equal(sc.cpu().numpy().view(np.uint32), want[1].view(np.uint32))
    assert np.array_equal(pool_bytes(pool), want[0])
    if q is not None:
        assert np.array_equal(bits(qo), want[2])
    return want


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new,held", [([1], [0]), ([1], [15]), ([1], [16]), ([17], [0]), ([40], [7]), ([3], [13]),
                                      ([1] * 33, list(range(33))), ([0, 5, 0, 0, 200, 1, 0], [9, 0, 3, 0, 31, 16, 2]),
                                      ([16, 16, 48], [0, 16, 8]), ([300], [250])])
def test_append_codes_scales_and_q(lib, cuda_device, tables, kind, new, held):
    lens = [n + h for n, h in zip(new, held)]
    T, pages = sum(new), sum(-(-n // 16) for n in lens) + 3
    cu = np.concatenate([[0], np.cumsum(new)])
    bt = tables_for(1, lens, pages)
    codes, scales = random_pages(2, pages, kind)
    k, v, q = rows(3, T, 8, 64), rows(4, T, 8, 64, scale=0.3), rows(5, T, 32, 64)
    check_append(lib, cuda_device, kind, codes, scales, k, v, cu, lens, bt, tables, q)
    check_append(lib, cuda_device, kind, codes, scales, k, v, cu, lens, bt)                 # K as it is
    check_append(lib, cuda_device, kind, codes, scales, k, v, cu, lens, bt, tables)


@pytest.mark.parametrize("kind", KINDS)
def test_append_token_by_token_with_growing_rows(lib, cuda_device, kind):
    """20 one-token calls on one pool, rows from tiny to large and back: the
    codes held are written again each time the scale grows."""
    dev = cuda_device
    codes, scales = random_pages(6, 4, kind)
    scales[:] = 1e30                                   # left by a former owner: slot 0 sets it anew
    bt = np.array([[2, 0]], np.int32)
    pool, sc = to_pool(codes, scales, kind, dev)
    for t in range(20):
        k = rows(20 + t, 1, 8, 64, scale=2.0 ** (t % 11 - 6))
        v = rows(60 + t, 1, 8, 64, scale=3.0 ** (7 - t % 9))
        if t == 3:
            v[:] = 0
        codes, scales, _, err = O8.append(codes, scales, k, v, [0, 1], [t + 1], bt, kind)
        lib.kv_append_rope_bs8(to_dev_bf16(k, dev), to_dev_bf16(v, dev), to_dev_i32([0, 1], dev),
                               to_dev_i32([t + 1], dev), to_dev_i32(bt, dev), pool, sc)
        assert not err
    assert np.array_equal(pool_bytes(pool), codes)
    assert np.array_equal(sc.cpu().numpy().view(np.uint32), scales.view(np.uint32))


@pytest.mark.parametrize("kind", KINDS)
def test_append_zero_and_extreme_rows(lib, cuda_device, kind):
    k = rows(7, 5, 8, 64)
    k[0] = 0
    k[1] = OB.from_f32_rne(np.float32(3e38))
    k[2, :, ::3] = 1                                    # the least subnormal
    k[2, :, 1::3] = 0
    k[2, :, 2::3] = 0x8001
    k[3] = OB.from_f32_rne(np.float32(-1e-38))
    v = rows(8, 5, 8, 64, scale=1e-20)
    codes, scales = random_pages(9, 7, kind)
    for t in range(5):                                  # each on a page of its own
        check_append(lib, cuda_device, kind, codes, scales, k[t:t + 1], v[t:t + 1], [0, 1], [1], np.array([[t]], np.int32))
    check_append(lib, cuda_device, kind, codes, scales, k, v, [0, 5], [5], np.array([[6]], np.int32))


@pytest.mark.parametrize("kind", KINDS)
def test_append_values_where_a_code_changes(lib, cuda_device, kind):
    """Quotients at and beside the middle between two codes, the tie itself among
    them, under scales of many significands and exponents."""
    pages = 24
    g = np.random.default_rng(71)
    amax = np.ldexp(1 + g.integers(0, 128, (pages, 2, 8)) / 128, g.integers(-90, 90, (pages, 2, 8))).astype(np.float32)
    top = np.float32(127 if kind == "int8" else 448)
    scale = (amax / top).astype(np.float64)
    if kind == "int8":
        middle = np.arange(127) + 0.5
    else:
        middle = (16 + np.arange(16)) / 16 * 2.0 ** np.arange(-10, 9)[:, None]
        middle = middle[(middle < 448)].ravel()
    at = g.choice(middle, (pages, 2, 8, 16, 64)) * scale[..., None, None]
    x = ((at.astype(np.float32).view(np.uint32) >> 16).astype(np.int64) + g.integers(-1, 3, at.shape)).astype(np.uint16)
    x |= (g.integers(0, 2, x.shape) << 15).astype(np.uint16)
    big = np.abs(OB.to_f64(x)) > amax[..., None, None]
    x[big] = 0
    x[:, :, :, 5, 7] = amax.view(np.uint32) >> 16                       # the block's largest, exactly
    rows_of = x.transpose(1, 0, 3, 2, 4).reshape(2, pages * 16, 8, 64)
    bt = g.permutation(pages).astype(np.int32)[None]
    codes, scales = np.zeros((pages, 2, 8, 16, 64), np.uint8), np.zeros((pages, 2, 8), np.float32)
    n = pages * 16
    check_append(lib, cuda_device, kind, codes, scales, rows_of[0], rows_of[1], [0, n], [n], bt)


@pytest.mark.parametrize("kind", KINDS)
def test_append_zeros_of_both_signs(lib, cuda_device, tables, kind):
    k, v, q = rows(73, 40, 8, 64), rows(74, 40, 8, 64), rows(75, 40, 32, 64)
    for x in (k, v, q):
        x[:, :, ::3] = 0x8000
        x[::7] = 0
        x[1::7] = 0x8000
    codes, scales = random_pages(76, 8, kind)
    bt = np.array([[3, 0, 5], [1, 7, 2]], np.int32)
    for rope in (None, tables):
        check_append(lib, cuda_device, kind, codes, scales, k, v, [0, 23, 40], [30, 17], bt, rope, None if rope is None else q)


@pytest.mark.parametrize("kind", KINDS)
def test_append_bad_sequences_are_skipped(lib, cuda_device, tables, kind):
    codes, scales = random_pages(10, 6, kind)
    k, v, q = rows(11, 60, 8, 64), rows(12, 60, 8, 64), rows(13, 60, 32, 64)
    bt = np.array([[0, 1], [2, 99], [-1, 3], [4, 5], [4, 5]], np.int32)
    #         fine; second page outside; first page missing; too long; fewer tokens than new ones
    want = check_append(lib, cuda_device, kind, codes, scales, k, v, [0, 20, 40, 50, 52, 55], [20, 20, 30, 33, 2], bt, tables, q)
    assert want[3]
    # rows behind the last sequence are left as they were; a range beyond the rows is refused
    pool, sc, qo, code = append(lib, cuda_device, kind, codes, scales, k, v, [0, 4], [4], bt, tables, q)
    assert code == 0 and (qo[4:] == 0).all() and (qo[:4] != 0).any()
    pool, sc, qo, code = append(lib, cuda_device, kind, codes, scales, k, v, [0, 61], [61], bt, tables, q)
    assert code == lib.ERR_DEVICE_INDEX and np.array_equal(pool_bytes(pool), codes)
    # longer than the tables of rotations
    pool, sc, qo, code = append(lib, cuda_device, kind, codes, scales, k, v, [0, 1], [601], np.zeros((1, 64), np.int32), tables, q)
    assert code == lib.ERR_DEVICE_INDEX and np.array_equal(pool_bytes(pool), codes)
    for n in (2 ** 31 - 1, -1, -2 ** 31):
        pool, sc, qo, code = append(lib, cuda_device, kind, codes, scales, k, v, [0, 1], [n], bt)
        assert code == lib.ERR_DEVICE_INDEX and np.array_equal(pool_bytes(pool), codes)


def test_append_many_sequences_and_strided_rows(lib, cuda_device, tables):
    """1500 sequences (the search takes more than one round), rows of a fused projection."""
    dev, S = cuda_device, 1500
    g = np.random.default_rng(14)
    new = g.integers(0, 3, S)
    held = g.integers(0, 32, S)
    lens = new + held
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1])
    pages = int(sum(-(-n // 16) for n in lens)) + 1
    bt = tables_for(15, lens, pages, 5)
    codes, scales = random_pages(16, pages, "int8")
    qkv = rows(17, T, 48, 64)
    want = O8.append(codes, scales, qkv[:, 32:40], qkv[:, 40:], cu, lens, bt, "int8", tables[2], tables[3], qkv[:, :32])
    d = to_dev_bf16(qkv, dev)
    pool, sc = to_pool(codes, scales, "int8", dev)
    qo = torch.zeros(T, 32, 64, dtype=torch.bfloat16, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    lib.kv_append_rope_bs8(d[:, 32:40], d[:, 40:], to_dev_i32(cu, dev), to_dev_i32(lens, dev), to_dev_i32(bt, dev),
                           pool, sc, tables[0], tables[1], d[:, :32], qo, err, max_blocks=3)
    assert lib.pkv_read_device_error(err) == 0
    assert np.array_equal(pool_bytes(pool), want[0]) and np.array_equal(sc.cpu().numpy(), want[1])
    assert np.array_equal(bits(qo), want[2])


@pytest.mark.parametrize("kind", KINDS)
def test_read_pages(lib, cuda_device, kind):
    dev = cuda_device
    codes, scales = random_pages(18, 9, kind)
    pool, sc = to_pool(codes, scales, kind, dev)
    ids = np.array([3, 3, 0, 8], np.int32)
    got = bits(lib.kv_read_bs8(pool, sc, to_dev_i32(ids, dev)))
    want = OB.from_f32_rne(O8.values(codes[ids], scales[ids], kind).astype(np.float32))
    assert np.array_equal(got, want)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out = lib.kv_read_bs8(pool, sc, to_dev_i32([-1, 9, 1], dev), d_err=err)
    assert lib.pkv_read_device_error(err) == lib.ERR_DEVICE_INDEX
    assert (out[:2] == 0).all() and np.array_equal(bits(out[2]), OB.from_f32_rne(
        O8.values(codes[1], scales[1], kind).astype(np.float32)))
    assert lib.kv_read_bs8(pool, sc, to_dev_i32([], dev)).shape[0] == 0


# ------------------------------------------------------------------ decode --

def decode(lib, dev, kind, q, codes, scales, bt, lens, scale=0.125, **kw):
    pool, sc = to_pool(codes, scales, kind, dev)
    qd = to_dev_bf16(q, dev)
    out = torch.full_like(qd, 5.0)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    lib.paged_gqa_decode_bs8(qd, pool, sc, to_dev_i32(bt, dev), to_dev_i32(lens, dev), out, scale, d_err=err, **kw)
    return out, lib.pkv_read_device_error(err)


def close(out, ref, size, reach, most, lens, what=""):
    got = OB.to_f64(bits(out))
    n = np.asarray(lens, np.float64).clip(0)[:, None, None]
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * (2.0 ** -17 * reach + 2.0 ** -21) + (n / 16 + 24) * 2.0 ** -23) * size
    tol += n * 2.0 ** -39 * most
    assert np.isfinite(got).all(), what
    over = np.abs(got - ref) - tol * (1 + 2.0 ** -8) - 1e-38
    assert (over <= 0).all(), f"{what}: {over.max():.3e} over at {np.unravel_index(over.argmax(), over.shape)}"


def check_decode(lib, dev, kind, q, codes, scales, bt, lens, scale=0.125, **kw):
    out, code = decode(lib, dev, kind, q, codes, scales, bt, lens, scale, **kw)
    assert code == 0
    close(out, *O8.attend(q, codes, scales, bt, lens, scale, kind), lens)
    return out


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens", [[1], [15], [16], [17], [31], [32], [33], [37], [49], [64], [65], [129], [2048], [2047],
                                  [0], [0, 0, 5, 0], [1] * 40, [2048, 1, 0, 700, 17, 1500, 2047, 129],
                                  [33, 600, 0, 16, 16, 16, 999], list(range(70))])
def test_decode_lengths(lib, cuda_device, kind, lens):
    pages = sum(-(-n // 16) for n in lens) + 2
    codes, scales = random_pages(30, pages, kind)
    bt = tables_for(31, lens, pages)
    codes[np.setdiff1d(np.arange(pages), bt)] = 0x7F    # pages of nobody: NaN as e4m3
    for s, n in enumerate(lens):                        # slots behind the end hold anything, NaN among it
        if n % 16:
            codes[bt[s, n // 16], :, :, n % 16:] = 0xFF if s % 2 else 0x7F
    out = check_decode(lib, cuda_device, kind, rows(32, len(lens), 32, 64), codes, scales, bt, lens, max_seq_len=max(lens))
    again = check_decode(lib, cuda_device, kind, rows(32, len(lens), 32, 64), codes, scales, bt, lens, max_seq_len=max(lens))
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    for s, n in enumerate(lens):
        if n == 0:
            assert (out[s] == 0).all()


@pytest.mark.parametrize("kind", KINDS)
def test_decode_long_sequence_and_wrong_bounds(lib, cuda_device, kind):
    lens = [20011, 3]
    codes, scales = random_pages(33, 1300, kind)
    bt = tables_for(34, lens, 1300, 1400)
    q = rows(35, 2, 32, 64, scale=0.5)
    check_decode(lib, cuda_device, kind, q, codes, scales, bt, lens)
    check_decode(lib, cuda_device, kind, q, codes, scales, bt, lens, max_seq_len=16)       # a bound far too small
    check_decode(lib, cuda_device, kind, q, codes, scales, bt, lens, max_blocks=1251, max_seq_len=0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("what", ["sharp", "tiny q", "huge q", "zero q", "no scale", "negative scale", "outlier page",
                                  "zero V blocks", "zero pages", "large scales", "small scales"])
def test_decode_values(lib, cuda_device, kind, what):
    lens = [150, 47]
    codes, scales = random_pages(36, 16, kind)
    bt = tables_for(37, lens, 16)
    q, scale = rows(38, 2, 32, 64), 0.125
    if what == "sharp":
        q = rows(38, 2, 32, 64, scale=20.0)
    elif what == "tiny q":
        q = rows(38, 2, 32, 64, scale=1e-36)
    elif what == "huge q":
        q, scale = rows(38, 2, 32, 64, scale=1e30), 1e-31
    elif what == "zero q":
        q = q & 0x8000
    elif what == "no scale":
        scale = 0.0
    elif what == "negative scale":
        scale = -0.2
    elif what == "outlier page":
        scales[bt[0, 3], 1] *= 4096
        scales[bt[0, 5], 0] *= 30
    elif what == "zero V blocks":
        scales[bt[0, ::2], 1] = 0
        codes[bt[0, ::2], 1] = 0
    elif what == "zero pages":
        codes[:] = 0
        scales[:] = 0
    elif what == "large scales":
        scales[:, 1] *= np.float32(1e30)
    elif what == "small scales":
        scales[:, 1] *= np.float32(1e-30)
        scales[:, 0] *= np.float32(1e-25)
    check_decode(lib, cuda_device, kind, q, codes, scales, bt, lens, scale)


@pytest.mark.parametrize("kind", KINDS)
def test_infinite_and_nan_queries_stay_in_their_head(lib, cuda_device, kind):
    lens = [150, 20]
    codes, scales = random_pages(55, 14, kind)
    bt = tables_for(56, lens, 14)
    q = rows(57, 2, 32, 64, scale=1e-3)
    ref = O8.attend(q, codes, scales, bt, lens, 0.125, kind)
    bad = q.copy()
    bad[0, 5, 3], bad[1, 30, 63] = 0x7F80, 0x7FC0          # inf, NaN
    out, code = decode(lib, cuda_device, kind, bad, codes, scales, bt, lens)
    assert code == 0
    keep = np.ones((2, 32), bool)
    keep[0, 5] = keep[1, 30] = False
    assert torch.isnan(out[1, 30].float()).all()
    out[0, 5], out[1, 30] = 0, 0
    close(out * torch.from_numpy(keep).to(out)[..., None], *[r * keep[..., None] for r in ref], lens)


def test_pages_behind_4_gib(lib, cuda_device, tables):
    """Offsets into a pool pass 32 bits: the last pages of 4.5 GB of codes."""
    dev, pages, n = cuda_device, 275000, 100
    pool, sc = lib.new_bs8_pool(pages, dev)
    bt = np.arange(pages - 7, pages, dtype=np.int32)[None, ::-1].copy()
    k, v, q = rows(58, n, 8, 64), rows(59, n, 8, 64), rows(60, 1, 32, 64)
    small = O8.append(np.zeros((7, 2, 8, 16, 64), np.uint8), np.zeros((7, 2, 8), np.float32), k, v, [0, n], [n],
                      np.arange(6, -1, -1, dtype=np.int32)[None], "int8")
    btd, lens = to_dev_i32(bt, dev), to_dev_i32([n], dev)
    lib.kv_append_rope_bs8(to_dev_bf16(k, dev), to_dev_bf16(v, dev), to_dev_i32([0, n], dev), lens, btd, pool, sc)
    assert np.array_equal(pool_bytes(pool[-7:]), small[0]) and np.array_equal(sc[-7:].cpu().numpy(), small[1])
    assert int((sc != 0).sum()) == int((small[1] != 0).sum())
    out = torch.empty(1, 32, 64, dtype=torch.bfloat16, device=dev)
    lib.paged_gqa_decode_bs8(to_dev_bf16(q, dev), pool, sc, btd, lens, out, 0.125)
    close(out, *O8.attend(q, small[0], small[1], np.arange(6, -1, -1, dtype=np.int32)[None], [n], 0.125, "int8"), [n])
    wide = lib.kv_read_bs8(pool, sc, to_dev_i32([pages - 1], dev))
    assert np.array_equal(bits(wide)[0], OB.from_f32_rne(O8.values(small[0][6], small[1][6], "int8").astype(np.float32)))


@pytest.mark.parametrize("kind", KINDS)
def test_decode_refuses_bad_sequences_alone(lib, cuda_device, kind):
    lens = [40, 300, -1, 7000, 2 ** 31 - 1, 500, 33, 20]
    codes, scales = random_pages(39, 60, kind)
    q = rows(40, len(lens), 32, 64)
    bt = np.full((len(lens), 32), -1, np.int32)
    perm = np.random.default_rng(41).permutation(60).astype(np.int32)
    bt[0, :3], bt[1, :19], bt[5, :32], bt[7, :2] = perm[:3], perm[3:22], perm[22:54], perm[54:56]
    bt[5, 17] = 60                                     # outside the pool, in the middle of a split sequence
    bt[6, :2] = perm[56:58]                            # and its third page missing
    out, code = decode(lib, cuda_device, kind, q, codes, scales, bt, lens)
    assert code == lib.ERR_DEVICE_INDEX
    good = [0, 1, 7]
    assert (out[[2, 3, 4, 5, 6]] == 0).all()
    ref = O8.attend(q[good], codes, scales, bt[good], np.array(lens)[good], 0.125, kind)
    close(out[good], *ref, np.array(lens)[good])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("S", [128, 129, 300])
def test_decode_many_sequences_long_short_empty_and_bad(lib, cuda_device, kind, S):
    """Sequences over many CTAs between ones that share a CTA, with all that is refused."""
    g = np.random.default_rng(60 + S)
    lens = g.integers(0, 500, S)
    lens[g.permutation(S)[:S // 3]] = g.integers(0, 18, S // 3)
    lens[[5, S - 2]] = 9001, 6007
    lens[[0, S - 1]] = 0, 700
    pages = int(sum(-(-n // 16) for n in lens)) + 1
    codes, scales = random_pages(61, pages, kind)
    bt = tables_for(62, lens, pages)
    q = rows(63, S, 32, 64)
    check_decode(lib, cuda_device, kind, q, codes, scales, bt, lens)
    bad = [5, 17, 18, 40, S - 1]
    lens[[17, 18, 40]] = -3, bt.shape[1] * 16 + 1, 480
    bt[5, 300], bt[S - 1, 43], bt[40, :30] = pages, -1, -1
    out, code = decode(lib, cuda_device, kind, q, codes, scales, bt, lens)
    assert code == lib.ERR_DEVICE_INDEX
    assert (out[bad] == 0).all()
    good = np.setdiff1d(np.arange(S), bad)
    close(out[good], *O8.attend(q[good], codes, scales, bt[good], lens[good], 0.125, kind), lens[good])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("S,bound", [(5, 64), (70, 128), (700, 64), (700, 384), (700, 400)])
def test_decode_short_by_the_bound(lib, cuda_device, kind, S, bound):
    """Whole sequences per CTA or shares, by the bound alone; lengths beyond it, empty
    and bad sequences among them."""
    g = np.random.default_rng(80 + S)
    lens = g.integers(0, bound, S)
    lens[g.permutation(S)[:S // 2]] = g.integers(0, 3, S // 2)
    lens[[0, S // 2, S - 1]] = 0, bound + 37, 700
    pages = int(sum(-(-n // 16) for n in lens)) + 1
    codes, scales = random_pages(81, pages, kind)
    bt = tables_for(82, lens, pages)
    q = rows(83, S, 32, 64)
    out = check_decode(lib, cuda_device, kind, q, codes, scales, bt, lens, max_seq_len=bound)
    assert (out[lens == 0] == 0).all()
    lens[[1, 3]] = -5, bt.shape[1] * 16 + 1
    bt[S - 1, 20], bad = -1, [1, 3, S - 1]
    out, code = decode(lib, cuda_device, kind, q, codes, scales, bt, lens, max_seq_len=bound)
    assert code == lib.ERR_DEVICE_INDEX and (out[bad] == 0).all()
    good = np.setdiff1d(np.arange(S), bad)
    close(out[good], *O8.attend(q[good], codes, scales, bt[good], lens[good], 0.125, kind), lens[good])


def test_decode_largest_batch_and_page_order(lib, cuda_device):
    S = 4096
    lens = np.random.default_rng(42).integers(0, 20, S).astype(np.int32)
    pages = int(sum(-(-n // 16) for n in lens))
    codes, scales = random_pages(43, pages, "int8")
    bt = tables_for(44, lens, pages)
    q = rows(45, S, 32, 64)
    out = check_decode(lib, cuda_device, "int8", q, codes, scales, bt, lens)
    perm = np.random.default_rng(46).permutation(pages)      # the same pages elsewhere
    moved, moved_sc = np.empty_like(codes), np.empty_like(scales)
    moved[perm], moved_sc[perm] = codes, scales
    bt2 = np.where(bt >= 0, perm[bt.clip(0)], -1).astype(np.int32)
    out2, _ = decode(lib, cuda_device, "int8", q, moved, moved_sc, bt2, lens)
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16))
    with pytest.raises(lib.PkvError):
        decode(lib, cuda_device, "int8", rows(45, S + 1, 32, 64), codes, scales, np.zeros((S + 1, 2), np.int32),
               np.zeros(S + 1, np.int32), workspace=torch.empty(1 << 27, dtype=torch.uint8, device=cuda_device))


@pytest.mark.parametrize("kind", KINDS)
def test_decode_of_odd_pages_after_a_call_that_leaves_nan(lib, cuda_device, kind):
    """Stages hold two pages; the missing one of an odd count must not matter,
    whatever an earlier call left in shared memory."""
    dev = cuda_device
    big = [4000] * 20
    codes, scales = random_pages(50, 5001, kind)
    bt = tables_for(51, big, 5001)
    lens = [3, 17, 33, 1, 48, 5, 81, 16] * 5
    q = rows(52, len(lens), 32, 64)
    bt2 = tables_for(53, lens, 5001)
    want = O8.attend(q, codes, scales, bt2, lens, 0.125, kind)
    nan = np.full_like(scales, np.nan)
    for _ in range(3):
        decode(lib, dev, kind, rows(54, 20, 32, 64), np.full_like(codes, 0x7F), nan, bt, big)
        out, code = decode(lib, dev, kind, q, codes, scales, bt2, lens)
        assert code == 0
        close(out, *want, lens)


def test_decode_workspace_streams_and_graphs(lib, cuda_device):
    """Any content of the workspace; two captured graphs with workspaces of
    their own on two streams at once; replays over other lengths."""
    dev, kind = cuda_device, "e4m3"
    lens = [700, 90, 1200, 3]
    codes, scales = random_pages(47, 200, kind)
    bt = tables_for(48, lens, 200, 100)
    q = rows(49, 4, 32, 64)
    want = check_decode(lib, dev, kind, q, codes, scales, bt, lens)
    pool, sc = to_pool(codes, scales, kind, dev)
    n = lib.paged_gqa_decode_bs8_workspace_bytes(4)
    graphs = []
    for fill in (0, 255):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=dev)
        a = dict(q=to_dev_bf16(q, dev), out=torch.zeros(4, 32, 64, dtype=torch.bfloat16, device=dev),
                 lens=to_dev_i32(lens, dev), bt=to_dev_i32(bt, dev), ws=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                lib.paged_gqa_decode_bs8(a["q"], pool, sc, a["bt"], a["lens"], a["out"], 0.125, workspace=ws)
        graphs.append((g, a, torch.cuda.Stream(dev)))
    torch.cuda.synchronize(dev)
    for _ in range(5):
        for g, a, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize(dev)
    for g, a, s in graphs:
        assert torch.equal(a["out"].view(torch.int16), want.view(torch.int16))
    short = [16, 90, 0, 3]
    graphs[0][1]["lens"].copy_(to_dev_i32(short, dev))
    graphs[0][0].replay()
    torch.cuda.synchronize(dev)
    close(graphs[0][1]["out"], *O8.attend(q, codes, scales, bt, short, 0.125, kind), short)


def test_refusals(lib, cuda_device):
    dev = cuda_device
    pool, sc = lib.new_bs8_pool(4, dev)
    q = torch.zeros(2, 32, 64, dtype=torch.bfloat16, device=dev)
    bt, lens = torch.zeros(2, 3, dtype=torch.int32, device=dev), torch.ones(2, dtype=torch.int32, device=dev)

    def call(**kw):
        a = dict(q=q, kv_pool=pool, kv_scales=sc, block_tables=bt, seq_lens=lens, out=torch.empty_like(q), scale=0.125) | kw
        lib.paged_gqa_decode_bs8(**a)
    call()
    for kw, e in ((dict(kv_pool=pool.view(torch.uint8)), TypeError), (dict(kv_pool=pool.cpu()), ValueError),
                  (dict(kv_pool=pool[:, :1]), ValueError), (dict(kv_scales=sc[:3]), ValueError),
                  (dict(kv_scales=sc.half()), TypeError), (dict(seq_lens=lens[:1]), ValueError),
                  (dict(block_tables=bt[:1]), ValueError), (dict(q=q.float()), TypeError),
                  (dict(scale=float("inf")), lib.PkvError), (dict(max_blocks=4), lib.PkvError),
                  (dict(workspace=torch.empty(64, dtype=torch.uint8, device=dev)), lib.PkvError)):
        with pytest.raises(e):
            call(**kw)
    k = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device=dev)
    cu = torch.arange(3, dtype=torch.int32, device=dev)
    cos = torch.zeros(16, 32, device=dev)
    for kw, e in ((dict(rope_cos=cos), ValueError), (dict(q_in=q, q_out=q), ValueError),
                  (dict(cu_new=cu[:2]), ValueError), (dict(k=k[:1]), ValueError),
                  (dict(rope_cos=cos, rope_sin=cos[:8]), ValueError),
                  (dict(k=k[:, :, :32]), ValueError), (dict(max_blocks=9), lib.PkvError)):
        a = dict(k=k, v=k, cu_new=cu, seq_lens=lens, block_tables=bt, kv_pool=pool, kv_scales=sc) | kw
        with pytest.raises(e):
            lib.kv_append_rope_bs8(**a)
    with pytest.raises(TypeError):
        lib.new_bs8_pool(1, dev, torch.float16)
    with pytest.raises(ValueError):
        lib.kv_read_bs8(pool, sc, bt[0], torch.empty(1, 2, 8, 16, 64, dtype=torch.bfloat16, device=dev))
