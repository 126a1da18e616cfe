"""paged_gqa_decode_bs8 where sequences are split over CTAs and merged: every number
of sequences at which the merge takes another form, with bounds above those that
keep sequences whole.  Tolerances are those of test_gpu_bs8_numbers.py."""
import numpy as np
import pytest
import torch

from oracle import bf16 as OB, bs8_kv as O8
from tests.test_gpu_bs8_numbers import KINDS, TYPES, lib, pages, rows, tolerance  # noqa: F401
from tests._util import bits, to_dev_bf16, to_dev_i32

pytestmark = pytest.mark.gpu


def decode(lib, dev, kind, q, codes, scales, bt, lens, **kw):  # noqa: F811
    pool = torch.from_numpy(codes.view(np.int8)).to(dev).view(TYPES[kind])
    qd = to_dev_bf16(q, dev)
    out = torch.full_like(qd, 5.0)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    lib.paged_gqa_decode_bs8(qd, pool, torch.from_numpy(scales).to(dev), to_dev_i32(bt, dev), to_dev_i32(lens, dev), out,
                             0.125, d_err=err, **kw)
    return out, lib.pkv_read_device_error(err)


def close(out, q, codes, scales, bt, lens, kind):
    ref, size, reach, most = O8.attend(q, codes, scales, bt, lens, 0.125, kind)
    live = bt[bt >= 0]
    top_k = np.nanmax(np.abs(O8.values(codes[live], scales[live], kind)[:, 0]))    # (NaN only behind the ends)
    tol = tolerance(q, ref, size, reach, most, lens, top_k, 0.125)
    got = OB.to_f64(bits(out))
    assert np.isfinite(got).all()
    over = np.abs(got - ref) - tol * (1 + 2.0 ** -8) - 1e-38
    assert (over <= 0).all(), f"{over.max():.3e} over at {np.unravel_index(over.argmax(), over.shape)}"


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("S", [2, 8, 9, 32, 33, 38, 39, 76, 77, 128, 129])
def test_shares_of_every_merge(lib, cuda_device, kind, S):  # noqa: F811
    """Long sequences over several CTAs, short ones that share a CTA, empty and bad ones."""
    g = np.random.default_rng(S)
    lens = g.integers(1, 900, S)
    lens[g.permutation(S)[:S // 4]] = g.integers(1, 40, S // 4)
    lens[[0, S - 1]] = 3001, 1777
    if S > 4:
        lens[[2, S // 2]] = 0
    codes, scales, bt = pages(40 + S, lens, kind, spare=2)
    for s, n in enumerate(lens):                        # slots behind the end hold NaN codes
        if n % 16:
            codes[bt[s, n // 16], :, :, n % 16:] = 0x7F
    q = rows(41, S, 32, 64)
    out, code = decode(lib, cuda_device, kind, q, codes, scales, bt, lens)
    assert code == 0 and (out[lens == 0] == 0).all()
    close(out, q, codes, scales, bt, lens, kind)
    again, _ = decode(lib, cuda_device, kind, q, codes, scales, bt, lens)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    if S < 8:
        return
    lens[[1, 3]] = -4, bt.shape[1] * 16 + 1             # refused lengths; a page that is none in a split sequence
    bt[0, 100] = len(codes)
    out, code = decode(lib, cuda_device, kind, q, codes, scales, bt, lens)
    assert code == lib.ERR_DEVICE_INDEX and (out[[0, 1, 3]] == 0).all()
    good = np.setdiff1d(np.arange(S), [0, 1, 3])
    close(out[good], q[good], codes, scales, bt[good], lens[good], kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bound", [81, 100000])
def test_odd_pages_in_shares_after_a_call_that_leaves_nan(lib, cuda_device, kind, bound):  # noqa: F811
    """The missing page of an odd last stage must not matter, whatever an earlier call left
    in shared memory: with sequences whole, and with a bound that forces shares."""
    lens = np.array([3, 17, 33, 1, 48, 5, 81, 16] * 5)
    codes, scales, bt = pages(50, lens, kind)
    q = rows(51, len(lens), 32, 64)
    big = np.full(20, 4000)
    junk_codes, junk_scales, junk_bt = pages(52, big, kind)
    junk_scales[:] = np.nan
    junk_codes[:] = 0x7F
    for _ in range(3):
        decode(lib, cuda_device, kind, rows(53, 20, 32, 64), junk_codes, junk_scales, junk_bt, big)
        out, code = decode(lib, cuda_device, kind, q, codes, scales, bt, lens, max_seq_len=bound)
        assert code == 0
        close(out, q, codes, scales, bt, lens, kind)
