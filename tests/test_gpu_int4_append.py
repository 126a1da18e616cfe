"""4-bit pages: kv_append_rope_int4 and kv_read_int4 against the FP64 oracle, bit
for bit (codes, scales, minima, rotated q, pages read back)."""
import numpy as np
import pytest
import torch

from oracle import bf16 as OB, int4_kv as O4, rope as OR
from tests._util import bits, cancelling_rows, to_dev_bf16, to_dev_i32
from tests.test_gpu_bs8 import rows, tables_for

pytestmark = pytest.mark.gpu


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


def random_pool(seed, pages):
    """Any bytes: what former owners left."""
    return np.random.default_rng(seed).integers(0, 256, (pages, 8, O4.BLOCK_BYTES)).astype(np.uint8)


def append(lib, dev, pool, k, v, cu, lens, bt, rope=None, q=None, **kw):
    pool, err = torch.from_numpy(pool).to(dev), torch.zeros(1, dtype=torch.int32, device=dev)
    if rope is not None:
        kw |= dict(rope_cos=rope[0], rope_sin=rope[1])
    if q is not None:
        kw |= dict(q_in=to_dev_bf16(q, dev), q_out=torch.zeros(q.shape, dtype=torch.bfloat16, device=dev))
    lib.kv_append_rope_int4(to_dev_bf16(k, dev), to_dev_bf16(v, dev), to_dev_i32(cu, dev), to_dev_i32(lens, dev),
                            to_dev_i32(bt, dev), pool, d_err=err, **kw)
    return pool.cpu().numpy(), kw.get("q_out"), lib.pkv_read_device_error(err)


def check(lib, dev, pool, k, v, cu, lens, bt, rope=None, q=None):
    cos, sin = (rope[2], rope[3]) if rope is not None else (None, None)
    want = O4.append(pool, k, v, cu, lens, bt, cos, sin, q)
    got, qo, code = append(lib, dev, pool, k, v, cu, lens, bt, rope, q)
    assert (code != 0) == want[2]
    assert np.array_equal(got, want[0])
    if q is not None:
        assert np.array_equal(bits(qo), want[1])
    return want


@pytest.mark.parametrize("new,held", [([1], [0]), ([1], [15]), ([1], [16]), ([17], [0]), ([40], [7]), ([3], [13]),
                                      ([1] * 33, list(range(33))), ([0, 5, 0, 0, 200, 1, 0], [9, 0, 3, 0, 31, 16, 2]),
                                      ([16, 16, 48], [0, 16, 8]), ([500], [50]), ([470, 8], [0, 0])])
def test_append(lib, cuda_device, tables, new, held):
    lens = [n + h for n, h in zip(new, held)]
    T, pages = sum(new), sum(-(-n // 16) for n in lens) + 3
    cu = np.concatenate([[0], np.cumsum(new)])
    bt = tables_for(1, lens, pages)
    pool = random_pool(2, pages)
    k, v, q = rows(3, T, 8, 64), rows(4, T, 8, 64, scale=0.3), rows(5, T, 32, 64)
    check(lib, cuda_device, pool, k, v, cu, lens, bt, tables, q)
    check(lib, cuda_device, pool, k, v, cu, lens, bt)                 # K as it is
    check(lib, cuda_device, pool, k, v, cu, lens, bt, tables)


def test_rotations_that_cancel(lib, cuda_device, tables):
    pos = np.arange(100)
    k, q = cancelling_rows(6, pos, 8, tables[2], tables[3]), cancelling_rows(7, pos, 32, tables[2], tables[3])
    check(lib, cuda_device, random_pool(8, 9), k, rows(9, 100, 8, 64), [0, 100], [100], tables_for(10, [100], 9), tables, q)


@pytest.mark.parametrize("T", [5, 32])
def test_values_at_the_ends(lib, cuda_device, T):
    """Rows of zeros of both signs, one value, subnormals, bf16's largest, steps of 2^-126
    and beside it, infinities and NaN in one place."""
    k, v = rows(11, T, 8, 64), rows(12, T, 8, 64, scale=1e-20)
    k[0] = 0
    k[1] = OB.from_f32_rne(np.float32(3e38))
    k[1, :, ::2] ^= 0x8000                                  # from one end to the other
    k[2, :, ::3] = 1                                        # the least subnormal
    k[2, :, 1::3] = 0
    k[2, :, 2::3] = 0x8001
    k[3] = 0x8000
    k[3, ::2, 5] = 0
    k[4] = OB.from_f32_rne(np.float32(-1.25))
    v[0] = 0x7F7F                                           # the largest, and its negative
    v[0, :, 9] = 0xFF7F
    for h, step in enumerate((0.99, 1.0, 1.01, 15, 16, 2.0 ** 100, 2.0 ** 200, 0.5)):   # times 2^-126
        v[1, h] = 0
        v[1, h, 17] = OB.from_f32_rne(np.float32(step * 15 * 2.0 ** -126))
    v[2, 0, 3], v[2, 1, 60], v[2, 2, 0], v[2, 3, 31] = 0x7F80, 0xFF80, 0x7FC0, 0xFFFF
    v[2, 4, 0], v[2, 4, 1] = 0x7F80, 0xFF80
    pool = random_pool(13, 9)
    check(lib, cuda_device, pool, k, v, [0, T], [T], np.array([[6, 2]], np.int32))
    if T == 5:
        for t in range(T):                                  # each on a page of its own
            check(lib, cuda_device, pool, k[t:t + 1], v[t:t + 1], [0, 1], [1], np.array([[t]], np.int32))


def test_values_where_a_code_changes(lib, cuda_device):
    """Values at and beside the middle between two codes, under scales of many
    significands and exponents."""
    g = np.random.default_rng(14)
    n, x = 256, None
    span = np.ldexp(1 + g.integers(0, 128, (2, n, 8)) / 128, g.integers(-90, 90, (2, n, 8)))
    lo = np.where(g.random(span.shape) < 0.5, 0.0, -span * g.integers(0, 33, span.shape) / 32)
    at = lo[..., None] + (g.integers(0, 15, (2, n, 8, 64)) + 0.5) * (span / 15)[..., None]
    x = ((at.astype(np.float32).view(np.uint32) >> 16).astype(np.int64) + g.integers(-1, 3, at.shape)).astype(np.uint16)
    x[..., 5] = OB.from_f32_rne(lo.astype(np.float32))
    x[..., 7] = OB.from_f32_rne((lo + span).astype(np.float32))
    bt = g.permutation(16).astype(np.int32)[None]
    check(lib, cuda_device, random_pool(15, 16), x[0], x[1], [0, n], [n], bt)


def test_bad_sequences_are_skipped(lib, cuda_device, tables):
    pool = random_pool(16, 6)
    k, v, q = rows(17, 60, 8, 64), rows(18, 60, 8, 64), rows(19, 60, 32, 64)
    bt = np.array([[0, 1], [2, 99], [-1, 3], [4, 5], [4, 5]], np.int32)
    #         fine; second page outside; first page missing; too long; fewer tokens than new ones
    want = check(lib, cuda_device, pool, k, v, [0, 20, 40, 50, 52, 55], [20, 20, 30, 33, 2], bt, tables, q)
    assert want[2]
    # rows behind the last sequence are left as they were; a range beyond the rows is refused
    got, qo, code = append(lib, cuda_device, pool, k, v, [0, 4], [4], bt, tables, q)
    assert code == 0 and (qo[4:] == 0).all() and (qo[:4] != 0).any()
    for cu, lens, b, rope in (([0, 61], [61], bt, tables), ([0, 1], [601], np.zeros((1, 64), np.int32), tables),
                              ([0, 1], [2 ** 31 - 1], bt, None), ([0, 1], [-1], bt, None), ([0, 1], [-2 ** 31], bt, None)):
        got, qo, code = append(lib, cuda_device, pool, k, v, cu, lens, b, rope, q if rope else None)
        assert code == lib.ERR_DEVICE_INDEX and np.array_equal(got, pool)


def test_many_sequences_and_strided_rows(lib, cuda_device, tables):
    """1500 sequences, rows of a fused projection, q rotated in place of another call's output."""
    dev, S = cuda_device, 1500
    g = np.random.default_rng(20)
    new, held = g.integers(0, 3, S), g.integers(0, 32, S)
    lens = new + held
    cu = np.concatenate([[0], np.cumsum(new)])
    T, pages = int(cu[-1]), int(sum(-(-n // 16) for n in lens)) + 1
    bt = tables_for(21, lens, pages, 5)
    pool, qkv = random_pool(22, pages), rows(23, T, 48, 64)
    want = O4.append(pool, qkv[:, 32:40], qkv[:, 40:], cu, lens, bt, tables[2], tables[3], qkv[:, :32])
    d, held_pool = to_dev_bf16(qkv, dev), torch.from_numpy(pool).to(dev)
    qo, err = torch.zeros(T, 32, 64, dtype=torch.bfloat16, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    lib.kv_append_rope_int4(d[:, 32:40], d[:, 40:], to_dev_i32(cu, dev), to_dev_i32(lens, dev), to_dev_i32(bt, dev),
                            held_pool, tables[0], tables[1], d[:, :32], qo, err, max_blocks=3)
    assert lib.pkv_read_device_error(err) == 0
    assert np.array_equal(held_pool.cpu().numpy(), want[0]) and np.array_equal(bits(qo), want[1])


def test_read_pages(lib, cuda_device):
    dev = cuda_device
    pool = random_pool(24, 700)
    pool[:, :, 1024:] = np.random.default_rng(25).integers(0x3C00, 0x4180, (700, 8, 64)).astype(np.uint16).view(np.uint8)
    pool[3, 2, 1024:1028] = np.array([0x7FC0, 0x7FC0], np.uint16).view(np.uint8)          # a NaN row
    d = torch.from_numpy(pool).to(dev)
    for ids in ([3, 3, 0, 8], list(range(700))):
        got = lib.kv_read_int4(d, to_dev_i32(ids, dev)).float().cpu().numpy()
        want = OB.to_f64(OB.from_f32_rne(O4.values(pool[ids]).astype(np.float32)))
        assert np.array_equal(got.astype(np.float64), want, equal_nan=True)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out = lib.kv_read_int4(d, to_dev_i32([-1, 700, 1], dev), d_err=err)
    assert lib.pkv_read_device_error(err) == lib.ERR_DEVICE_INDEX
    assert (out[:2] == 0).all() and np.array_equal(bits(out[2]), OB.from_f32_rne(O4.values(pool[1:2]).astype(np.float32))[0])
    assert lib.kv_read_int4(d, to_dev_i32([], dev)).shape[0] == 0


def test_pool_behind_4_gib(lib, cuda_device, tables):
    """Pages whose bytes lie behind 2^32."""
    dev, pages = cuda_device, 470000
    pool = torch.empty((pages, 8, O4.BLOCK_BYTES), dtype=torch.uint8, device=dev)
    bt = np.array([[pages - 1, 2, pages - 7]], np.int32)
    k, v = rows(26, 40, 8, 64), rows(27, 40, 8, 64)
    for i in (pages - 1, 2, pages - 7):
        pool[i] = 0
    lib.kv_append_rope_int4(to_dev_bf16(k, dev), to_dev_bf16(v, dev), to_dev_i32([0, 40], dev), to_dev_i32([40], dev),
                            to_dev_i32(bt, dev), pool)
    want, _, _ = O4.append(O4.new_pool(3), k, v, [0, 40], [40], np.array([[0, 1, 2]], np.int32))
    assert np.array_equal(pool[bt[0].tolist()].cpu().numpy(), want)
    got = bits(lib.kv_read_int4(pool, to_dev_i32(bt[0], dev)))
    assert np.array_equal(got, OB.from_f32_rne(O4.values(want).astype(np.float32)))
