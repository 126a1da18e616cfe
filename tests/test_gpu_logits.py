"""process_logits against the oracle: ids and logits equal bit for bit (every
operation of the definition is one rounded fp32 operation on both sides)."""
import numpy as np
import pytest
import torch

from oracle import bf16 as OB, logits as OL

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib(cuda_device):
    from paged_kv_gqa_append_gb300 import build
    build.build()
    import paged_kv_gqa_append_gb300 as m
    return m


def case(seed, rows, vocab, hist, bias, dtype="float32", specials=True):
    g = np.random.default_rng(seed)
    x = (4 * g.standard_normal((rows, vocab))).astype(np.float32)
    if specials:
        for r in range(rows):
            at = g.integers(0, vocab, 6)
            x[r, at] = [np.nan, np.inf, -np.inf, 0.0, -0.0, np.float32(np.nanmax(x[r]))][: len(at)]
    t = torch.from_numpy(x).to(getattr(torch, dtype))
    c = dict(x=t, wide=t.float().numpy())
    c["history"] = g.integers(-3, vocab + 3, (rows, hist)).astype(np.int32)     # padding among them
    c["history"][:, ::2] = g.integers(0, min(vocab, 5), c["history"][:, ::2].shape)   # and repeats
    c["history_lens"] = g.integers(-1, hist + 3, rows).astype(np.int32)
    c["prompt_lens"] = g.integers(0, hist + 1, rows).astype(np.int32)
    c["repetition"] = g.uniform(0.7, 1.9, rows).astype(np.float32)
    c["presence"] = g.uniform(-1, 1, rows).astype(np.float32)
    c["frequency"] = g.uniform(-1, 1, rows).astype(np.float32)
    if bias:
        c["bias_ids"] = g.integers(-2, vocab + 2, (rows, bias)).astype(np.int32)
        c["bias_ids"][:, -1] = c["bias_ids"][:, 0]                               # the same id twice
        c["bias_values"] = (3 * g.standard_normal((rows, bias))).astype(np.float32)
    c["mask"] = g.integers(-2 ** 31, 2 ** 31, (rows, (vocab + 31) // 32 + seed % 2)).astype(np.int32)
    return c


NAMES = ["history", "history_lens", "prompt_lens", "repetition", "presence", "frequency", "bias_ids", "bias_values", "mask"]


def run(lib, dev, c, names, out=True, **kw):
    put = {("allow_mask" if n == "mask" else n): torch.from_numpy(c[n]).to(dev) for n in names if n in c}
    x = c["x"].to(dev)
    o = torch.full(x.shape, 7.0, device=dev) if out is True else out
    ids = lib.process_logits(x, out=o, **put, **kw)
    want, want_ids = OL.process(c["wide"], **{n: c[n] for n in names if n in c})
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    if o is not None:
        got = o.cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(want))
        ok = ~np.isnan(want)
        assert np.array_equal(got[ok].view(np.uint32), want[ok].view(np.uint32))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("rows,vocab,hist,bias", [(1, 1, 1, 1), (3, 7, 5, 2), (2, 31, 40, 0), (5, 257, 64, 9),
                                                  (4, 1000, 3, 700), (33, 4099, 129, 33), (2, 128256, 2048, 300),
                                                  (61, 4099, 129, 33), (150, 1003, 2500, 7)])
def test_everything(lib, cuda_device, dtype, rows, vocab, hist, bias):
    c = case(rows + vocab, rows, vocab, hist, bias, dtype)
    run(lib, cuda_device, c, NAMES)
    run(lib, cuda_device, c, NAMES, out=None)


@pytest.mark.parametrize("names", [[], ["mask"], ["bias_ids", "bias_values"], ["history", "history_lens"],
                                   ["history", "history_lens", "frequency"],
                                   ["history", "history_lens", "prompt_lens", "presence", "mask"]])
def test_each_alone(lib, cuda_device, names):
    run(lib, cuda_device, case(5, 6, 2500, 77, 12), names)
    run(lib, cuda_device, case(6, 6, 2500, 77, 12), names, out=None)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("vocab,hist,bias", [(20011, 30000, 0), (9001, 5, 6000), (16500, 12000, 4000), (8200, 20000, 1)])
def test_more_changed_tokens_than_a_pass_holds(lib, cuda_device, dtype, vocab, hist, bias):
    """Over 1024 distinct tokens in an eighth of the vocabulary: smaller passes."""
    c = case(vocab, 3, vocab, hist, bias, dtype)
    c["history"][:, ::2] = np.random.default_rng(vocab).integers(0, vocab, c["history"][:, ::2].shape)
    c["history_lens"][:] = [hist, hist // 2, hist]
    run(lib, cuda_device, c, NAMES)
    run(lib, cuda_device, c, NAMES, out=None)
    many = {n: np.concatenate([a] * 17) for n, a in c.items() if n not in ("x", "wide")}     # CTAs of the other shape
    many["x"], many["wide"] = c["x"].repeat(17, 1), np.concatenate([c["wide"]] * 17)
    many["repetition"][3:] += 0.25
    dev = cuda_device
    got = lib.process_logits(many["x"].to(dev), **{("allow_mask" if n == "mask" else n): torch.from_numpy(many[n]).to(dev)
                                                    for n in NAMES if n in many}).cpu().numpy()
    sub = [0, 1, 2, 30, 31, 50]
    _, want = OL.process(many["wide"][sub], **{n: many[n][sub] for n in NAMES if n in many})
    assert np.array_equal(got[sub], want)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,vocab,hist,bias", [(160, 1777, 30, 3), (320, 1001, 40, 5), (700, 515, 900, 2), (700, 16500, 5, 0),
                                                  (310, 2048, 3000, 40)])
def test_many_rows(lib, cuda_device, dtype, rows, vocab, hist, bias):
    """Fewer CTAs per row, and more of them again where lists are long."""
    c = case(vocab, rows, vocab, hist, bias, dtype)
    run(lib, cuda_device, c, NAMES)
    run(lib, cuda_device, c, ["mask"], out=None)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("vocab,at", [(1, 0), (9, 1), (4099, 3), (20011, 5), (257, 7)])
def test_equal_logits_at_any_alignment(lib, cuda_device, dtype, vocab, at):
    """The first of equal logits, wherever 16-byte loads begin; -0 equals 0."""
    x = torch.zeros((9, vocab + at), dtype=getattr(torch, dtype))
    x[:, ::2] = -0.0
    x = x.to(cuda_device)[:, at:]
    assert (lib.process_logits(x).cpu() == 0).all()
    mask = torch.zeros((9, (vocab + 31) // 32), dtype=torch.int32)
    last = vocab - 1
    mask[:, last // 32] = -2 ** 31 if last % 32 == 31 else 1 << (last % 32)
    mask[:, 0] |= 1 << min(4, last)
    out = torch.full((9, vocab + 3), 5.0, device=cuda_device)
    ids = lib.process_logits(x, out=out[:, 1:vocab + 1], allow_mask=mask.to(cuda_device))
    assert (ids.cpu() == min(4, last)).all()
    got = out.cpu().numpy()
    want = np.full((9, vocab), -np.inf, np.float32)
    want[:, [min(4, last), last]] = 0
    assert np.array_equal(got[:, 1:vocab + 1], want) and (got[:, 0] == 5).all() and (got[:, vocab + 1:] == 5).all()


@pytest.mark.parametrize("rows", [2, 80])
@pytest.mark.parametrize("hist,bias,distinct", [(9000, 0, 40), (2500, 1500, 900), (700, 131200, 300), (5, 66000, 2400)])
def test_long_lists_of_few_tokens(lib, cuda_device, rows, hist, bias, distinct):
    """Lists far longer than what is entered at a time, of tokens of one part;
    a bias entry's number needs more than 16 bits."""
    c = case(rows, rows, 20011, hist, bias)
    g = np.random.default_rng(rows + distinct)
    some = np.sort(g.permutation(2500)[:distinct]).astype(np.int32)     # one CTA's tokens
    c["history"] = some[g.integers(0, distinct, c["history"].shape)]
    c["history_lens"] = np.full(rows, hist, np.int32)
    if bias:
        c["bias_ids"] = some[g.integers(0, distinct, c["bias_ids"].shape)]
        c["bias_ids"][:, 65530:65540] = 19999                           # beside the 2^16th entry, in the last part
    run(lib, cuda_device, c, NAMES)
    x = c["x"].to(cuda_device)
    run(lib, cuda_device, dict(c, x=x), NAMES, out=None)
    put = {("allow_mask" if n == "mask" else n): torch.from_numpy(c[n]).to(cuda_device) for n in NAMES if n in c}
    other = torch.empty_like(x)
    ids = lib.process_logits(x, out=other, **put)
    same = x.clone()
    assert torch.equal(lib.process_logits(same, out=same, **put), ids)
    assert torch.equal(same.view(torch.int32), other.view(torch.int32))


def test_large_vocabulary(lib, cuda_device):
    """Over 8 x 16384 tokens the parts go in passes; the last one is ragged."""
    c = case(7, 2, 300001, 500, 50)
    c["history"][:, :100] = np.random.default_rng(1).integers(0, 300001, (2, 100))
    c["history_lens"][:] = 500
    run(lib, cuda_device, c, NAMES)


def test_strided_unaligned_rows_and_in_place(lib, cuda_device):
    dev = cuda_device
    c = case(8, 5, 1001, 30, 5)
    put = {("allow_mask" if n == "mask" else n): torch.from_numpy(c[n]).to(dev) for n in NAMES}
    want, want_ids = OL.process(c["wide"], **{n: c[n] for n in NAMES})
    buf = torch.full((5, 1009), 3.0, device=dev)
    buf[:, 3:1004] = c["x"].to(dev)
    rows = buf[:, 3:1004]
    ids = lib.process_logits(rows, out=rows, **put)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert np.array_equal(rows.cpu().numpy(), want, equal_nan=True)
    assert (buf[:, :3] == 3).all() and (buf[:, 1004:] == 3).all()
    half = torch.zeros((5, 1005), dtype=torch.float16, device=dev)
    c16 = case(9, 5, 1001, 30, 5, "float16")
    half[:, 1:1002] = c16["x"].to(dev)
    out = torch.zeros((5, 1003), device=dev)
    ids = lib.process_logits(half[:, 1:1002], out=out[:, 2:], allow_mask=torch.from_numpy(c16["mask"]).to(dev))
    want, want_ids = OL.process(c16["wide"], mask=c16["mask"])
    assert np.array_equal(ids.cpu().numpy(), want_ids) and np.array_equal(out[:, 2:].cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("copies", [1, 12])
def test_rows_with_nothing_left(lib, cuda_device, copies):
    dev = cuda_device
    x = torch.randn(4, 100, device=dev)
    x[1] = float("nan")
    x[2] = float("-inf")
    mask = torch.full((4, 4), -1, dtype=torch.int32, device=dev)
    mask[0] = 0
    mask[3] = 0
    mask[3, 3] = 1 << 30                                   # a bit behind the vocabulary: token 126
    x, mask = x.repeat(copies, 1), mask.repeat(copies, 1)
    out = torch.empty_like(x)
    ids = lib.process_logits(x, out=out, allow_mask=mask)
    assert ids.tolist() == [-1, -1, 0, -1] * copies
    # everything is -inf but for what the history makes of it: a penalty cannot raise it, a bias can
    low = torch.full((4 * copies, 100), float("-inf"), device=dev)
    hist = torch.full((4 * copies, 2), 7, dtype=torch.int32, device=dev)
    lens = torch.full((4 * copies,), 2, dtype=torch.int32, device=dev)
    bias = torch.full((4 * copies, 1), 40, dtype=torch.int32, device=dev)
    up = torch.full((4 * copies, 1), float("inf"), device=dev)
    first = lib.process_logits(low, history=hist, history_lens=lens)
    assert first.tolist() == [0] * (4 * copies)
    first = lib.process_logits(low, bias_ids=bias, bias_values=up)                 # -inf + inf is NaN: never chosen
    assert first.tolist() == [0] * (4 * copies)
    only = torch.zeros((4 * copies, 4), dtype=torch.int32, device=dev)
    only[:, 0] = 1 << 7
    assert lib.process_logits(low, history=hist, history_lens=lens, allow_mask=only).tolist() == [7] * (4 * copies)
    assert torch.isinf(out[0]).all() and torch.isnan(out[1]).all()


def test_matches_the_plain_argmax(lib, cuda_device):
    x = torch.randn(64, 128256, device=cuda_device)
    assert torch.equal(lib.process_logits(x), lib.argmax_rows(x))


def test_graph_replay_and_another_stream(lib, cuda_device):
    dev = cuda_device
    c = case(10, 3, 5000, 64, 8)
    put = {("allow_mask" if n == "mask" else n): torch.from_numpy(c[n]).to(dev) for n in NAMES}
    x, out = c["x"].to(dev), torch.empty(3, 5000, device=dev)
    ids = torch.empty(3, dtype=torch.int32, device=dev)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    lib.process_logits(x, out=out, ids=ids, stream=side, **put)
    side.synchronize()
    first = (ids.clone(), out.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.process_logits(x, out=out, ids=ids, **put)
    for _ in range(2):
        out.zero_()
        ids.zero_()
        g.replay()
        assert torch.equal(ids, first[0]) and torch.equal(out.nan_to_num(9.0), first[1].nan_to_num(9.0))


def test_refusals(lib, cuda_device):
    dev = cuda_device
    x = torch.randn(2, 50, device=dev)
    i = torch.zeros(2, 4, dtype=torch.int32, device=dev)
    one = torch.ones(2, dtype=torch.int32, device=dev)
    for kw, e in ((dict(history=i), ValueError), (dict(repetition=torch.ones(2, device=dev)), ValueError),
                  (dict(history=i, history_lens=one[:1]), ValueError), (dict(bias_ids=i), ValueError),
                  (dict(bias_ids=i, bias_values=torch.ones(2, 3, device=dev)), ValueError),
                  (dict(allow_mask=i[:, :1].contiguous()), ValueError), (dict(out=x.half()), TypeError),
                  (dict(out=torch.empty(2, 49, device=dev)), ValueError),
                  (dict(history=i.cpu(), history_lens=one), ValueError),
                  (dict(ids=torch.zeros(2, dtype=torch.int64, device=dev)), TypeError)):
        with pytest.raises(e):
            lib.process_logits(x, **kw)
    with pytest.raises(ValueError):
        lib.process_logits(x.cpu())
    with pytest.raises(TypeError):
        lib.process_logits(x.double())
    with pytest.raises(ValueError):
        lib.process_logits(x.t())
    assert lib.process_logits(x[:0]).numel() == 0
    # an empty history counts nothing
    h0 = torch.zeros(2, 0, dtype=torch.int32, device=dev)
    assert torch.equal(lib.process_logits(x, history=h0, history_lens=one), lib.argmax_rows(x))
