"""How exactly paged_gqa_decode_bs8 computes, where its bf16 result shows it:
values that cancel, queries and codes of very different sizes.

Every output may be off by its own rounding to bf16, 2^-8 of the value, and by
terms relative to A = sum p |v| / sum p:
  a probability   two fp16 values: the first leaves at most 2^-11 of it, a
                  difference that fp32 holds exactly, the second 2^-11 of that,
                  so 2^-22; with the factor 2^14 on it the least step of both is
                  2^-24, so half of it, 2^-39 of the largest p, is the least error:
                  n 2^-39 max |v| more;
  its exponent    a score is 64 exact products, their sum and its three scalings:
                  2^-17 of R = scale sum |q| |k| (67 roundings of 2^-24); its
                  exponential 2^-21; each in numerator and denominator;
  a query         values below 2^-31 of their head's largest are rounded to fp16
                  steps of 2^-24 under a scale that puts the largest at 2^14 or
                  more: 2^-39 max |q| scale sum |k| per score;
  the sums        (n / 16 + 24) 2^-23 of A.
"""
import numpy as np
import pytest
import torch

from oracle import bf16 as OB, bs8_kv as O8
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


def rows(seed, *shape, scale=1.0):
    g = np.random.default_rng(seed)
    return OB.from_f32_rne((scale * g.standard_normal(shape)).astype(np.float32))


def pages(seed, lens, kind, spare=1):
    """Random codes and scales, and tables of shuffled pages for these lengths."""
    g = np.random.default_rng(seed)
    need = [-(-n // 16) for n in lens]
    count = sum(need) + spare
    codes = g.integers(0, 256, (count, 2, 8, 16, 64)).astype(np.uint8)
    codes[codes == 0x80] = 0
    if kind == "e4m3":
        codes[(codes & 0x7F) == 0x7F] = 0x70
    scales = np.exp(g.normal(-4 if kind == "int8" else -5, 0.5, (count, 2, 8))).astype(np.float32)
    bt = np.full((len(lens), max(1, max(need))), -1, np.int32)
    perm, at = g.permutation(count).astype(np.int32), 0
    for s, m in enumerate(need):
        bt[s, :m] = perm[at:at + m]
        at += m
    return codes, scales, bt


def decode(lib, dev, kind, q, codes, scales, bt, lens, scale=0.125, **kw):
    pool = torch.from_numpy(codes.view(np.int8)).to(dev).view(TYPES[kind])
    qd = to_dev_bf16(q, dev)
    out = torch.full_like(qd, 5.0)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    lib.paged_gqa_decode_bs8(qd, pool, torch.from_numpy(scales).to(dev), to_dev_i32(bt, dev), to_dev_i32(lens, dev), out,
                             scale, d_err=err, **kw)
    assert lib.pkv_read_device_error(err) == 0
    return OB.to_f64(bits(out))


def tolerance(q, ref, size, reach, most, lens, top_k, scale):
    n = np.asarray(lens, np.float64)[:, None, None]
    qmax = np.abs(OB.to_f64(q)).max(-1, keepdims=True)
    score = 2.0 ** -17 * reach + 2.0 ** -39 * qmax * abs(scale) * 64 * top_k
    return 2.0 ** -8 * np.abs(ref) + (2.0 ** -22 + 2 * (score + 2.0 ** -21) + (n / 16 + 24) * 2.0 ** -23) * size + \
        n * 2.0 ** -39 * most


def check(lib, dev, kind, q, codes, scales, bt, lens, scale=0.125, **kw):
    got = decode(lib, dev, kind, q, codes, scales, bt, lens, scale, **kw)
    ref, size, reach, most = O8.attend(q, codes, scales, bt, lens, scale, kind)
    live = bt[bt >= 0]
    top_k = np.abs(O8.values(codes[live], scales[live], kind)[:, 0]).max()
    tol = tolerance(q, ref, size, reach, most, lens, top_k, scale)
    assert np.isfinite(got).all()
    over = np.abs(got - ref) - tol * (1 + 2.0 ** -8) - 1e-38
    assert (over <= 0).all(), f"{over.max():.3e} over at {np.unravel_index(over.argmax(), over.shape)}"


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens", [[2], [16, 2, 37], [300, 2, 64], [6000], [70] * 40])
def test_values_that_cancel(lib, cuda_device, kind, lens):
    """V of every second token is the negative of its neighbour's, and the scores are
    nearly equal: the output is the small difference of large sums, in which the
    rounding of a probability to 11 bits shows."""
    codes, scales, bt = pages(1, lens, kind)
    codes[:, 1, :, 1::2] = codes[:, 1, :, ::2]
    if kind == "int8":
        codes[:, 1, :, 1::2] = (-codes[:, 1, :, ::2].view(np.int8)).view(np.uint8)
    else:
        codes[:, 1, :, 1::2] ^= 0x80
    scales[:, 0] *= np.float32(0.02 if kind == "int8" else 0.005)
    check(lib, cuda_device, kind, rows(2, len(lens), 32, 64), codes, scales, bt, lens)


@pytest.mark.parametrize("kind", KINDS)
def test_heads_of_a_group_with_queries_of_different_sizes(lib, cuda_device, kind):
    """q heads of one KV head 2^44 apart: each is scaled by its own largest value."""
    lens = [150, 47]
    codes, scales, bt = pages(3, lens, kind)
    q = OB.to_f64(rows(4, 2, 32, 64))
    q[:, 1::4] *= 2.0 ** 44
    q[:, 2::4] *= 2.0 ** -44
    check(lib, cuda_device, kind, OB.from_f32_rne(q.astype(np.float32)), codes, scales, bt, lens)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [2.0 ** 127.9, 2.0 ** 110, 2.0 ** -70, 2.0 ** -100])
def test_values_next_to_the_ends_of_the_range(lib, cuda_device, kind, size):
    """V as large as bf16 goes, of one sign so that the sums grow with the length, and V
    whose sums come near the smallest numbers; in one CTA and over many."""
    lens = [3, 1500, 8000]
    codes, scales, bt = pages(5, lens, kind)
    codes[:, 1, :, :, ::2] &= 0x7F                     # every second dim of one sign
    top = 127 if kind == "int8" else 448
    scales[:, 1] = np.float32(size / top) * np.random.default_rng(6).uniform(0.5, 0.99, scales[:, 1].shape)
    scales[:, 0] *= np.float32(0.05)
    check(lib, cuda_device, kind, rows(7, 3, 32, 64), codes, scales, bt, lens)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("up", [-124, -110, 60, 110])
def test_queries_and_keys_at_opposite_ends_of_the_range(lib, cuda_device, kind, up):
    """Scores of ordinary size from q about 2^up and K about 2^-up."""
    lens = [33, 900]
    codes, scales, bt = pages(8, lens, kind)
    scales[:, 0] = np.ldexp(np.random.default_rng(9).uniform(0.5, 1, scales[:, 0].shape), -up - (7 if kind == "int8" else 9))
    q = OB.to_f64(rows(10, 2, 32, 64)) * 2.0 ** up
    check(lib, cuda_device, kind, OB.from_f32_rne(q.astype(np.float32)), codes, scales, bt, lens)
