"""kv_append_rope_bs8 on what the documentation leaves to the caller: orders of
cu_new that do not ascend, and (bit for bit against the FP64 oracle) what the
other append tests do not reach."""
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


def rows(seed, *shape, scale=1.0):
    g = np.random.default_rng(seed)
    return OB.from_f32_rne((scale * g.standard_normal(shape)).astype(np.float32))


def random_pages(seed, pages, kind):
    g = np.random.default_rng(seed)
    codes = g.integers(0, 256, (pages, 2, 8, 16, 64)).astype(np.uint8)
    codes[codes == 0x80] = 0
    if kind == "e4m3":
        codes[(codes & 0x7F) == 0x7F] = 0x70
    return codes, np.exp(g.normal(-5, 0.7, (pages, 2, 8))).astype(np.float32)


def append(lib, dev, kind, codes, scales, k, v, cu, lens, bt, rope=None, q=None, q_out=None):
    """The call on copies: (code bytes, scales, q_out, error word)."""
    pool, sc = torch.from_numpy(codes.view(np.int8)).to(dev).view(TYPES[kind]), torch.from_numpy(scales).to(dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    kw = {} if rope is None else dict(rope_cos=rope[0], rope_sin=rope[1])
    if q is not None:
        kw |= dict(q_in=q, q_out=q_out)
    lib.kv_append_rope_bs8(to_dev_bf16(k, dev), to_dev_bf16(v, dev), to_dev_i32(cu, dev), to_dev_i32(lens, dev),
                           to_dev_i32(bt, dev), pool, sc, d_err=err, **kw)
    code = lib.pkv_read_device_error(err)
    return pool.view(torch.int8).cpu().numpy().view(np.uint8), sc.cpu().numpy(), code


@pytest.mark.parametrize("cu,lens", [([99, 100, 0], [1, 0]), ([50, 99, 100, 0], [3, 1, 0]), ([100, 50, 0], [60, 60]),
                                     ([70, 90, 95, 100, 1, 1], [1, 1, 1, 2, 3])])
def test_cu_new_that_does_not_ascend(lib, cuda_device, cu, lens):
    """No row lies in the range that the search finds for it: everything is refused,
    and no table entry in front of a sequence's own is read."""
    codes, scales = random_pages(1, 12, "int8")
    T = 100
    bt = np.arange(12, dtype=np.int32)[None].repeat(len(lens), 0)
    got, sc, code = append(lib, cuda_device, "int8", codes, scales, rows(2, T, 8, 64), rows(3, T, 8, 64), cu, lens, bt)
    assert code == lib.ERR_DEVICE_INDEX
    assert np.array_equal(got, codes) and np.array_equal(sc, scales)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [0x7FC0, 0x7F80, 0xFF80])
@pytest.mark.parametrize("at", [0, 4, 9])
def test_rows_that_are_not_finite_show(lib, cuda_device, kind, bad, at):
    """A NaN or an infinity in one value of K of one head: every token of that block reads
    as NaN, before and after it, in this call and in later ones; the other blocks are
    what they would be without it."""
    codes, scales = random_pages(5, 2, kind)
    bt = np.array([[1]], np.int32)
    k, v = rows(6, 14, 8, 64), rows(7, 14, 8, 64)
    k[at + 1:, 5] = OB.from_f32_rne((40 * OB.to_f64(k[at + 1:, 5])).astype(np.float32))      # finite rows that would grow the scale
    k[at, 5, 33] = bad
    clean = k.copy()
    clean[:, 5] = 0
    got, want = (codes, scales), (codes, scales, None, False)
    for lo, hi in ((0, 4), (4, 9), (9, 10), (10, 14)):
        *got, code = append(lib, cuda_device, kind, *got[:2], k[lo:hi], v[lo:hi], [0, hi - lo], [hi], bt)
        want = O8.append(want[0], want[1], clean[lo:hi], v[lo:hi], [0, hi - lo], [hi], bt, kind)
        assert code == 0
        if at < hi:
            assert not np.isfinite(got[1][1, 0, 5])
            pool = torch.from_numpy(got[0].view(np.int8)).to(cuda_device).view(TYPES[kind])
            sc = torch.from_numpy(got[1]).to(cuda_device)
            read = lib.kv_read_bs8(pool, sc, to_dev_i32([1], cuda_device)).float()[0]
            assert torch.isnan(read[0, 5, :hi]).all()
            out = torch.zeros(1, 32, 64, dtype=torch.bfloat16, device=cuda_device)
            lib.paged_gqa_decode_bs8(to_dev_bf16(rows(8, 1, 32, 64), cuda_device), pool, sc, to_dev_i32(bt, cuda_device),
                                     to_dev_i32([hi], cuda_device), out, 0.125)
            assert torch.isnan(out[0, 20:24].float()).all()
            assert torch.isfinite(out[0, :20].float()).all() and torch.isfinite(out[0, 24:].float()).all()
    other = np.ones((2, 2, 8), bool)
    other[1, 0, 5] = False
    assert np.array_equal(got[0][other], want[0][other]) and np.array_equal(got[1][other], want[1][other])
