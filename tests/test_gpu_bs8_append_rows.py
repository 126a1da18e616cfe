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
