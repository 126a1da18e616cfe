"""A chunk of a prompt over a cached prefix in 4-bit pages: both appended, the pages read back as
bf16 pages (kv_read_int4), attention by paged_gqa_prefill over those, against the oracle's own
append, values and causal attention."""
import numpy as np
import pytest
import torch

from oracle import bf16 as OB, int4_kv as O4, paged_kv as OP, rope as OR
from tests._util import bf16_to_f64, bits, check_close, to_dev_bf16, to_dev_i32
from tests.test_gpu_bs8 import rows, tables_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib(cuda_device):
    from paged_kv_gqa_append_gb300 import build
    build.build()
    import paged_kv_gqa_append_gb300 as m
    return m


def test_prefill_over_pages_read_back(lib, cuda_device):
    dev, i32 = cuda_device, torch.int32
    lens, fresh = np.array([37, 300, 16, 129, 200]), np.array([37, 64, 1, 40, 200])
    held = lens - fresh
    pages = int(sum(-(-n // 16) for n in lens)) + 3
    bt = tables_for(90, lens, pages)
    cos_d, sin_d = lib.rope_tables_device(dev, 512)
    cos_o, sin_o = OR.table(OR.inv_freq_llama3(), 512)
    pool = torch.full((pages, 8, O4.BLOCK_BYTES), 0xFF, dtype=torch.uint8, device=dev)  # NaN where nothing is written
    want = pool.cpu().numpy()
    err = torch.zeros(1, dtype=i32, device=dev)
    for seed, new, total in ((91, held, held), (94, fresh, lens)):
        cu, T = np.concatenate([[0], np.cumsum(new)]), int(new.sum())
        k, v, q = rows(seed, T, 8, 64), rows(seed + 1, T, 8, 64), rows(seed + 2, T, 32, 64)
        want, want_q, bad = O4.append(want, k, v, cu, total, bt, cos_o, sin_o, q)
        assert not bad
        turned = torch.empty(T, 32, 64, dtype=torch.bfloat16, device=dev)
        lib.kv_append_rope_int4(to_dev_bf16(k, dev), to_dev_bf16(v, dev), to_dev_i32(cu, dev), to_dev_i32(total, dev),
                                to_dev_i32(bt, dev), pool, cos_d, sin_d, to_dev_bf16(q, dev), turned, err)
    # the sequences' pages, one after another, and the tables of that order
    used = bt[bt >= 0]
    order = np.full(bt.shape, -1, np.int32)
    order[bt >= 0] = np.arange(len(used))
    read = lib.kv_read_int4(pool, to_dev_i32(used, dev), d_err=err)
    want_read = OB.from_f64_via_f32(O4.values(want[used]))
    nan = np.isnan(OB.to_f64(want_read))
    assert np.array_equal(np.where(nan, 0, bits(read)), np.where(nan, 0, want_read))
    out = torch.empty_like(turned)
    lib.paged_gqa_prefill(turned, to_dev_i32(cu, dev), read, to_dev_i32(order, dev), to_dev_i32(lens, dev), out, 0.125, d_err=err)
    assert lib.pkv_read_device_error(err) == 0
    ref, bad = OP.prefill(want_q, cu, want_read, order, lens, 0.125)
    assert not bad
    check_close(bf16_to_f64(out), ref, "prefill over 4-bit pages read back")
