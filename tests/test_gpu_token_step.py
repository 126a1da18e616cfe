"""A decode loop of the cache and token operators together, as a model with
normalised heads would run them on block-scaled 8-bit pages: prompt append,
then steps of qk_norm_rope, kv_append_rope_bs8, paged_gqa_decode_bs8 and
process_logits, eager and as one captured graph; and a prompt continued by
paged_gqa_prefill over pages read back as bf16."""
import numpy as np
import pytest
import torch

from oracle import bf16 as OB, bs8_kv as O8, logits as OL, paged_kv as OP
from tests._util import bits, check_close, bf16_to_f64, to_dev_bf16, to_dev_i32
from tests.test_gpu_bs8 import close, pool_bytes, rows, tables_for

pytestmark = pytest.mark.gpu
VOCAB = 999


@pytest.fixture(scope="module")
def lib(cuda_device):
    from paged_kv_gqa_append_gb300 import build
    build.build()
    import paged_kv_gqa_append_gb300 as m
    return m


@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("graph", [False, True])
def test_decode_loop(lib, cuda_device, dtype, graph):
    dev, kind = cuda_device, "int8" if dtype == torch.int8 else "e4m3"
    S, steps = 3, 19
    prompt = np.array([5, 0, 30], np.int32)
    pages = 12
    bt = tables_for(1, prompt + steps, pages, 4)
    f, mul = lib.pkv_rope_inv_freq_scaled(32, 10000.0, "yarn", 4.0, 16)        # half of the head
    cos, sin = lib.rope_tables_scaled_device(dev, 64, f, mul)
    w = [to_dev_bf16(OB.from_f32_rne(np.random.default_rng(i).uniform(0.5, 1.5, 64).astype(np.float32)), dev) for i in (2, 3)]
    pool, sc = lib.new_bs8_pool(pages, dev, dtype)
    btd, err = to_dev_i32(bt, dev), torch.zeros(1, dtype=torch.int32, device=dev)
    # the prompt
    T = int(prompt.sum())
    kp, vp, kr = to_dev_bf16(rows(4, T, 8, 64), dev), to_dev_bf16(rows(5, T, 8, 64), dev), torch.empty(T, 8, 64, dtype=torch.bfloat16, device=dev)
    pos = np.concatenate([np.arange(n) for n in prompt]).astype(np.int32)
    lib.qk_norm_rope(None, kp, to_dev_i32(pos, dev), cos, sin, None, kr, k_weight=w[1], interleaved=True, d_err=err)
    cu = np.concatenate([[0], np.cumsum(prompt)])
    lib.kv_append_rope_bs8(kr, vp, to_dev_i32(cu, dev), to_dev_i32(prompt, dev), btd, pool, sc, d_err=err)
    codes = np.zeros((pages, 2, 8, 16, 64), np.uint8)
    codes, scales, _, _ = O8.append(codes, np.zeros((pages, 2, 8), np.float32), bits(kr), bits(vp), cu, prompt, bt, kind)
    # the step's buffers: q, k, v as slices of one projection
    qkv = torch.empty(S, 48, 64, dtype=torch.bfloat16, device=dev)
    q, k, v = qkv[:, :32], qkv[:, 32:40], qkv[:, 40:]
    qo, ko, out = (torch.empty(S, n, 64, dtype=torch.bfloat16, device=dev) for n in (32, 8, 32))
    positions, lens = torch.empty(S, dtype=torch.int32, device=dev), torch.empty(S, dtype=torch.int32, device=dev)
    one = torch.arange(S + 1, dtype=torch.int32, device=dev)
    head = torch.randn(32 * 64, VOCAB, generator=torch.Generator("cpu").manual_seed(6)).to(dev, torch.bfloat16)
    logits = torch.empty(S, VOCAB, dtype=torch.bfloat16, device=dev)
    ids = torch.empty(S, dtype=torch.int32, device=dev)
    history = torch.full((S, steps), -1, dtype=torch.int32, device=dev)
    made = torch.zeros(S, dtype=torch.int32, device=dev)
    freq = torch.full((S,), 0.5, device=dev)
    mask = to_dev_i32(np.random.default_rng(7).integers(-2 ** 31, 2 ** 31, (S, 32)).astype(np.int32), dev)
    ws = lib.alloc_bs8_workspace(S, dev)

    def step():
        lib.qk_norm_rope(q, k, positions, cos, sin, qo, ko, q_weight=w[0], k_weight=w[1], interleaved=True, d_err=err)
        lib.kv_append_rope_bs8(ko, v, one, lens, btd, pool, sc, d_err=err)
        lib.paged_gqa_decode_bs8(qo, pool, sc, btd, lens, out, 0.125, workspace=ws, d_err=err)
        torch.mm(out.view(S, -1), head, out=logits)
        lib.process_logits(logits, ids=ids, history=history, history_lens=made, frequency=freq, allow_mask=mask)

    run = step
    for t in range(steps):
        n = prompt + t + 1
        qkv.copy_(to_dev_bf16(rows(100 + t, S, 48, 64, scale=1 + t % 3), dev))
        positions.copy_(to_dev_i32(n - 1, dev))
        lens.copy_(to_dev_i32(n, dev))
        if graph and t == 1:
            keep = pool.view(torch.int8).clone(), sc.clone()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
            assert torch.equal(pool.view(torch.int8), keep[0]) and torch.equal(sc, keep[1])  # a capture runs nothing
            run = g.replay
        run()
        torch.cuda.synchronize(dev)
        codes, scales, _, bad = O8.append(codes, scales, bits(ko), bits(v.contiguous()), np.arange(S + 1), n, bt, kind)
        assert not bad and np.array_equal(pool_bytes(pool), codes)
        assert np.array_equal(sc.cpu().numpy().view(np.uint32), scales.view(np.uint32))
        close(out, *O8.attend(bits(qo), codes, scales, bt, n, 0.125, kind), n, f"step {t}")
        _, want = OL.process(logits.float().cpu().numpy(), history.cpu().numpy(), made.cpu().numpy(), None, None, None,
                             freq.cpu().numpy(), mask=mask.cpu().numpy())
        assert np.array_equal(ids.cpu().numpy(), want)
        history[:, t] = ids
        made += 1
    assert lib.pkv_read_device_error(err) == 0


def test_prefill_over_a_cached_prefix_read_back(lib, cuda_device):
    """40 cached tokens in 8 bits and a chunk of 9 more: the pages read back as
    a bf16 pool, the chunk appended there, attention by paged_gqa_prefill."""
    dev = cuda_device
    bt = np.array([[3, 0, 2, 5]], np.int32)
    pool, sc = lib.new_bs8_pool(6, dev)
    cos, sin = lib.rope_tables_device(dev, 64)
    k, v, q = to_dev_bf16(rows(8, 49, 8, 64), dev), to_dev_bf16(rows(9, 49, 8, 64), dev), to_dev_bf16(rows(10, 9, 32, 64), dev)
    lib.kv_append_rope_bs8(k[:40], v[:40], to_dev_i32([0, 40], dev), to_dev_i32([40], dev), to_dev_i32(bt, dev), pool, sc, cos, sin)
    wide = lib.kv_read_bs8(pool, sc, to_dev_i32(bt[0], dev))
    here = torch.arange(4, dtype=torch.int32, device=dev)[None]
    qr = torch.empty_like(q)
    lib.kv_append_rope(k[40:].contiguous(), v[40:].contiguous(), torch.arange(40, 49, dtype=torch.int32, device=dev), here, wide,
                       cos, sin, token_seq=torch.zeros(9, dtype=torch.int32, device=dev), q_in=q, q_out=qr)
    out = torch.empty_like(q)
    lib.paged_gqa_prefill(qr, to_dev_i32([0, 9], dev), wide, here, to_dev_i32([49], dev), out, 0.125)
    for i in range(9):
        ref, bad = OP.decode(bits(qr[i:i + 1]), bits(wide), np.arange(4, dtype=np.int32)[None], [41 + i], 0.125)
        check_close(bf16_to_f64(out[i:i + 1]), ref, f"row {i}")


def test_usual_calls_are_marshalled_natively_and_equal_the_others(lib, cuda_device, monkeypatch):
    """The calls of a step never reach the ctypes way; through it (a stream
    given) they give the same bits."""
    dev, S = cuda_device, 5
    cos, sin = lib.rope_tables_device(dev, 64)
    qkv = to_dev_bf16(rows(20, S, 48, 64), dev)
    q, k, v = qkv[:, :32], qkv[:, 32:40], qkv[:, 40:]
    w = torch.ones(64, device=dev)
    bt = to_dev_i32(np.arange(S * 2).reshape(S, 2), dev)
    pos, lens, cu = (to_dev_i32(x, dev) for x in ([3, 16, 0, 31, 7], [4, 17, 1, 32, 8], np.arange(S + 1)))
    logits = torch.randn(S, 500, generator=torch.Generator("cpu").manual_seed(1)).to(dev)
    hist, hl = to_dev_i32(np.arange(S * 4).reshape(S, 4), dev), to_dev_i32([4] * S, dev)
    seen = []
    real = lib._call
    monkeypatch.setattr(lib, "_call", lambda dev, stream, where, args: (seen.append(where), real(dev, stream, where, args)))
    got = []
    for stream in (None, torch.cuda.current_stream(dev)):
        pool16 = torch.zeros((S * 2, 2, 8, 16, 64), dtype=torch.bfloat16, device=dev)
        pool, sc = lib.new_bs8_pool(S * 2, dev, torch.float8_e4m3fn)
        qo, ko, out = (torch.zeros(S, n, 64, dtype=torch.bfloat16, device=dev) for n in (32, 8, 32))
        ws = lib.alloc_bs8_workspace(S, dev)
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        lib.kv_append_norm_rope(k, v, pos, bt, pool16, cos, sin, q_in=q, q_out=qo, q_weight=w, k_weight=w, d_err=err, stream=stream)
        lib.qk_norm_rope(q, k, pos, cos, sin, qo, ko, q_weight=w, d_err=err, stream=stream)
        lib.kv_append_rope_bs8(k, v, cu, lens, bt, pool, sc, cos, sin, q, qo, err, stream=stream)
        wide = lib.kv_read_bs8(pool, sc, bt[0].contiguous(), torch.empty((2, 2, 8, 16, 64), dtype=torch.bfloat16, device=dev), err, stream=stream)
        lib.paged_gqa_decode_bs8(qo, pool, sc, bt, lens, out, 0.125, workspace=ws, max_seq_len=32, d_err=err, stream=stream)
        ids = lib.process_logits(logits, history=hist, history_lens=hl, frequency=torch.ones(S, device=dev), stream=stream)
        torch.cuda.synchronize(dev)
        assert lib.pkv_read_device_error(err) == 0
        got.append([pool16, qo, ko, pool.view(torch.int8), sc, wide, out, ids])
        assert len(seen) == (0 if stream is None else 6), seen
    for a, b in zip(*got):
        assert torch.equal(a, b)
    # what is refused is refused by the Python checks, with their words
    with pytest.raises(ValueError, match="positions must have 5 elements"):
        lib.qk_norm_rope(q, k, pos[:3], cos, sin, qo, ko)
    with pytest.raises(ValueError, match="num_seqs"):
        lib.paged_gqa_decode_bs8(qo, pool, sc, bt[:3], lens, out, 0.125)
    with pytest.raises(lib.PkvError, match="WORKSPACE"):
        lib.paged_gqa_decode_bs8(qo, pool, sc, bt, lens, out, 0.125, workspace=ws[:16])
