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


# ------------------------------------------------- chunks of 16 tokens per CTA --

@pytest.fixture(scope="module")
def tables(lib, cuda_device):
    cos_d, sin_d = lib.rope_tables_device(cuda_device, 2500)
    cos_o, sin_o = OR.table(OR.inv_freq_llama3(), 2500)
    return cos_d, sin_d, cos_o, sin_o


def prompts(sms, seed, short=True):
    """New and held tokens of ragged prompts, of which the append takes 16 tokens per CTA:
    more than three tokens per SM and 16 per sequence.  Some are shorter than a chunk
    or empty, so that several begin in one; most begin inside a page."""
    g = np.random.default_rng(seed)
    new = [sms, 1, 0, 5, sms + 37, 0, 3, 2, 1, 16, 2 * sms, 32, 700] if short else [4 * sms + 3]
    held = g.integers(0, 50, len(new))
    if short:
        held[:4] = [0, 15, 3, 16]
    held[-1] = 9
    assert sum(new) >= 3 * sms and sum(new) // len(new) >= 16
    return np.array(new), held


def shuffled_tables(seed, lens, spare=2):
    need = [-(-int(n) // 16) for n in lens]
    perm = np.random.default_rng(seed).permutation(sum(need) + spare).astype(np.int32)
    bt = np.full((len(lens), max(1, max(need))), -1, np.int32)
    at = 0
    for s, m in enumerate(need):
        bt[s, :m] = perm[at:at + m]
        at += m
    return bt, len(perm)


def check_prompts(lib, dev, kind, new, lens, bt, pages, rope, q_kind, behind=0, seed=30):
    """Against the oracle; `behind` rows follow the last sequence's and stay as they are."""
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1]) + behind
    codes, scales = random_pages(seed, pages, kind)
    k, v = rows(seed + 1, T, 8, 64), rows(seed + 2, T, 8, 64, scale=0.3)
    q = q_in = q_out = None
    if q_kind:
        q = rows(seed + 3, T, 32, 64)
        q_in = to_dev_bf16(q, dev)
        q_out = q_in if q_kind == "in place" else torch.full_like(q_in, 3.0)
    before = None if q_out is None else bits(q_out).copy()
    want = O8.append(codes, scales, k, v, cu, lens, bt, kind, *(rope[2:] if rope is not None else (None, None)), q)
    got, sc, code = append(lib, dev, kind, codes, scales, k, v, cu, lens, bt, rope, q_in, q_out)
    assert (code != 0) == want[3]
    assert np.array_equal(sc.view(np.uint32), want[1].view(np.uint32))
    assert np.array_equal(got, want[0])
    if q_kind:
        n = int(cu[-1])
        assert np.array_equal(bits(q_out)[:n], want[2][:n])
        assert np.array_equal(bits(q_out)[n:], before[n:])
    return want


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q_kind", ["", "apart", "in place"])
@pytest.mark.parametrize("turn", [True, False])
def test_prompts_in_chunks(lib, cuda_device, tables, kind, q_kind, turn):
    if q_kind and not turn:
        return
    sms = torch.cuda.get_device_properties(cuda_device).multi_processor_count
    new, held = prompts(sms, 20)
    bt, pages = shuffled_tables(21, new + held)
    check_prompts(lib, cuda_device, kind, new, new + held, bt, pages, tables if turn else None, q_kind, behind=19)
    new, held = prompts(sms, 22, short=False)
    bt, pages = shuffled_tables(23, new + held)
    check_prompts(lib, cuda_device, kind, new, new + held, bt, pages, tables if turn else None, q_kind)


@pytest.mark.parametrize("kind", KINDS)
def test_bad_prompts_between_good_ones_in_chunks(lib, cuda_device, tables, kind):
    """Sequences refused as a whole and pages that are none, at the start, the middle and
    the end of chunks; the good ones around them are written."""
    sms = torch.cuda.get_device_properties(cuda_device).multi_processor_count
    new, held = prompts(sms, 24)
    lens = new + held
    bt, pages = shuffled_tables(25, lens)
    lens[[1, 4, 8]] = [-1, new[4] - 1, bt.shape[1] * 16 + 1]     # one token; more than a chunk; one token
    bt[0, 3], bt[9, 0], bt[12, 2], bt[12, -1] = pages, -1, -7, pages + 9
    want = check_prompts(lib, cuda_device, kind, new, lens, bt, pages, tables, "apart", behind=3)
    assert want[3]
    lens = new + held
    lens[12] = 2501                                              # more than the rotations have
    bt, pages = shuffled_tables(25, lens)
    assert check_prompts(lib, cuda_device, kind, new, lens, bt, pages, tables, "in place")[3]


def test_prompts_in_chunks_over_many_sequences(lib, cuda_device, tables):
    """1500 sequences of about 20 tokens: the search takes more than one round, and several
    begin in every other chunk; rows of a fused projection."""
    g = np.random.default_rng(26)
    new = g.integers(0, 44, 1500)
    held = g.integers(0, 20, 1500)
    assert new.sum() // 1500 >= 16
    bt, pages = shuffled_tables(27, new + held)
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1])
    codes, scales = random_pages(28, pages, "int8")
    k, v = rows(29, T, 8, 64), rows(30, T, 8, 64)
    want = O8.append(codes, scales, k, v, cu, new + held, bt, "int8", tables[2], tables[3])
    qkv = torch.empty(T, 48, 64, dtype=torch.bfloat16, device=cuda_device)
    qkv[:, 32:40], qkv[:, 40:] = to_dev_bf16(k, cuda_device), to_dev_bf16(v, cuda_device)
    pool, sc = torch.from_numpy(codes.view(np.int8)).to(cuda_device), torch.from_numpy(scales).to(cuda_device)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    lib.kv_append_rope_bs8(qkv[:, 32:40], qkv[:, 40:], to_dev_i32(cu, cuda_device), to_dev_i32(new + held, cuda_device),
                           to_dev_i32(bt, cuda_device), pool, sc, tables[0], tables[1], d_err=err)
    assert lib.pkv_read_device_error(err) == 0
    assert np.array_equal(pool.cpu().numpy().view(np.uint8), want[0]) and np.array_equal(sc.cpu().numpy(), want[1])


@pytest.mark.parametrize("kind", KINDS)
def test_more_pages_read_than_sms(lib, cuda_device, kind):
    sms = torch.cuda.get_device_properties(cuda_device).multi_processor_count
    codes, scales = random_pages(31, 200, kind)
    ids = np.random.default_rng(32).integers(0, 200, 2 * sms + 5).astype(np.int32)
    ids[[3, 7, sms + 1]] = -1, 200, 2 ** 31 - 1
    pool, sc = torch.from_numpy(codes.view(np.int8)).to(cuda_device).view(TYPES[kind]), torch.from_numpy(scales).to(cuda_device)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    out = bits(lib.kv_read_bs8(pool, sc, to_dev_i32(ids, cuda_device), d_err=err))
    assert lib.pkv_read_device_error(err) == lib.ERR_DEVICE_INDEX
    ok = (ids >= 0) & (ids < 200)
    assert (out[~ok] == 0).all()
    assert np.array_equal(out[ok], OB.from_f32_rne(O8.values(codes, scales, kind).astype(np.float32))[ids[ok]])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("least,most,per_sm", [(0, 9, 20), (4, 14, 20), (10, 30, 3)])
def test_drafts_of_several_tokens_in_chunks(lib, cuda_device, tables, kind, least, most, per_sm):
    """A few tokens for each of many sequences, behind held ones: up to 16 runs, and more
    sequences than that, in a chunk."""
    sms = torch.cuda.get_device_properties(cuda_device).multi_processor_count
    g = np.random.default_rng(35 + least)
    new = g.integers(least, most + 1, per_sm * sms * 2 // (least + most) + 40)
    assert new.sum() >= per_sm * sms and new.sum() // len(new) >= (16 if per_sm == 3 else 4)
    held = g.integers(0, 40, len(new))
    bt, size = shuffled_tables(36, new + held)
    check_prompts(lib, cuda_device, kind, new, new + held, bt, size, tables, "apart", behind=5)
