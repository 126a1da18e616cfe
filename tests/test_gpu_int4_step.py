"""A decode loop that stays on the GPU: tables grown by grow_block_tables, prompts and
steps into 4-bit pages, attention, logits processing and sampling, eager and as one
captured graph, against the oracles step by step; finished rows released and their pages
used again; and the two ways that a call is marshalled."""
import numpy as np
import pytest
import torch

from oracle import int4_kv as O4, logits as OL, page_stack as PS, rope as OR, sampling as OS
from tests._util import bits, to_dev_bf16, to_dev_i32
from tests.test_gpu_bs8 import rows
from tests.test_gpu_int4 import close

pytestmark = pytest.mark.gpu
VOCAB = 999


@pytest.fixture(scope="module")
def lib(cuda_device):
    from paged_kv_gqa_append_gb300 import build
    build.build()
    import paged_kv_gqa_append_gb300 as m
    return m


@pytest.mark.parametrize("graph", [False, True])
def test_decode_loop(lib, cuda_device, graph):
    dev, S, layers, width, pages, steps = cuda_device, 3, 2, 4, 24, 22
    prompt = np.array([5, 30, 17], np.int32)
    cos, sin = lib.rope_tables_device(dev, 64)
    cos_o, sin_o = OR.table(OR.inv_freq_llama3(), 64)
    i32 = torch.int32
    stack, count = lib.new_free_pages(pages, dev)
    tables = torch.full((layers, S, width), -1, dtype=i32, device=dev)
    lens, new = torch.zeros(S, dtype=i32, device=dev), to_dev_i32(prompt, dev)
    done = torch.zeros(S, dtype=torch.bool, device=dev)
    pool, err = lib.new_int4_pool(pages, dev), torch.zeros(1, dtype=i32, device=dev)
    T = int(prompt.sum())
    cu = torch.empty(S + 1, dtype=i32, device=dev)
    slots = torch.empty((layers, T), dtype=i32, device=dev)
    # prompts and steps share buffers of T rows; a step fills the first of them
    q, qr = (torch.zeros(layers, T, 32, 64, dtype=torch.bfloat16, device=dev) for _ in range(2))
    k, v = (torch.zeros(layers, T, 8, 64, dtype=torch.bfloat16, device=dev) for _ in range(2))
    out = torch.empty(layers, S, 32, 64, dtype=torch.bfloat16, device=dev)
    ws = lib.alloc_int4_workspace(S, dev)
    head = torch.randn(32 * 64, VOCAB, generator=torch.Generator("cpu").manual_seed(6)).to(dev, torch.bfloat16)
    logits, kept = torch.empty(S, VOCAB, dtype=torch.bfloat16, device=dev), torch.empty(S, VOCAB, device=dev)
    noise = torch.empty(S, VOCAB, device=dev)
    ids, lp = torch.zeros(S, dtype=i32, device=dev), torch.zeros(S, device=dev)
    history, made = torch.full((S, steps + 1), -1, dtype=i32, device=dev), torch.zeros(S, dtype=i32, device=dev)
    freq, temp = torch.full((S,), 0.5, device=dev), to_dev_f32([0.8, 0.0, 1.5], dev)
    top_k, top_p = to_dev_i32([20, 0, 0], dev), to_dev_f32([1.0, 1.0, 0.8], dev)

    def tokens():
        lib.release_pages(lens, done, tables, stack, count, d_err=err)
        lib.grow_block_tables(lens, new, tables, stack, count, cu_new=cu, slots=slots, d_err=err)
        for l in range(layers):
            lib.kv_append_rope_int4(k[l], v[l], cu, lens, tables[l], pool, cos, sin, q[l], qr[l], err)

    def step():
        tokens()
        for l in range(layers):
            lib.paged_gqa_decode_int4(qr[l, :S], pool, tables[l], lens, out[l], 0.125, workspace=ws, d_err=err)
        torch.mm(out[-1].view(S, -1), head, out=logits)
        lib.process_logits(logits, out=kept, history=history, history_lens=made, frequency=freq)
        lib.sample_logits(kept, noise, temp, top_k=top_k, top_p=top_p, ids=ids, logprobs=lp)

    # the same on the host
    h_lens, h_tables, h_stack, h_count = np.zeros(S, np.int32), np.full((layers, S, width), -1, np.int32), np.arange(pages - 1, -1, -1, dtype=np.int32), pages
    h_pool = O4.new_pool(pages)
    run = step
    for t in range(steps + 1):
        fresh = prompt if t == 0 else np.ones(S, np.int32)
        finished = np.zeros(S, bool)
        if t == 12:  # the second row ends, and a prompt of 9 tokens takes its place
            finished[1], fresh[1] = True, 9
        n = int(fresh.sum())
        new.copy_(to_dev_i32(fresh, dev))
        done.copy_(torch.from_numpy(finished))
        for i, (x, heads) in enumerate(((q, 32), (k, 8), (v, 8))):
            x[:, :n].copy_(to_dev_bf16(rows(100 * t + i, layers, n, heads, 64), dev))
        noise.exponential_(generator=torch.Generator(dev).manual_seed(t))
        if t == 0:
            tokens()
        else:
            if graph and t == 2:
                keep = pool.clone(), tables.clone(), lens.clone()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    step()
                assert all(torch.equal(a, b) for a, b in zip(keep, (pool, tables, lens)))  # a capture runs nothing
                run = g.replay
            run()
        torch.cuda.synchronize(dev)
        h_stack, h_lens, h_count, bad = PS.release(h_lens, finished, h_tables, h_stack, h_count)
        assert not bad
        h_tables, h_lens, h_count, h_cu, _, _, h_slots, bad = PS.grow(h_lens, fresh, h_tables, h_stack, h_count, T)
        assert not bad
        for got, want in ((lens, h_lens), (tables, h_tables), (cu, h_cu), (slots, h_slots), (count, [h_count])):
            assert np.array_equal(got.cpu().numpy(), want), t
        for l in range(layers):
            h_pool, h_q, bad = O4.append(h_pool, bits(k[l]), bits(v[l]), h_cu, h_lens, h_tables[l], cos_o, sin_o, bits(q[l]))
            assert not bad and np.array_equal(bits(qr[l, :n]), h_q[:n])
        assert np.array_equal(pool.cpu().numpy(), h_pool)
        if t == 0:
            continue
        for l in range(layers):
            close(out[l], *O4.attend(bits(qr[l, :S]), h_pool, h_tables[l], h_lens, 0.125), h_lens, f"step {t}")
        want, _ = OL.process(logits.float().cpu().numpy(), history.cpu().numpy(), made.cpu().numpy(), None, None, None, freq.cpu().numpy())
        assert np.array_equal(kept.cpu().numpy(), want)
        e = noise.cpu().numpy()
        for r in range(S):
            assert OS.acceptable(int(ids[r]), want[r], e[r], float(temp[r]), int(top_k[r]), float(top_p[r])), (t, r)
        history[:, t - 1] = ids
        made += 1
    assert lib.pkv_read_device_error(err) == 0


def to_dev_f32(x, dev):
    return torch.tensor(x, dtype=torch.float32).to(dev)


def test_both_ways_of_a_call_give_the_same_bits(lib, cuda_device, monkeypatch):
    dev, S = cuda_device, 5
    cos, sin = lib.rope_tables_device(dev, 64)
    qkv = to_dev_bf16(rows(20, S, 48, 64), dev)
    q, k, v = qkv[:, :32], qkv[:, 32:40], qkv[:, 40:]
    x = torch.randn(S, 500, generator=torch.Generator("cpu").manual_seed(1)).to(dev)
    e = torch.empty(S, 500).exponential_(generator=torch.Generator("cpu").manual_seed(2)).to(dev)
    seen, got = [], []
    real = lib._call
    monkeypatch.setattr(lib, "_call", lambda dev, stream, where, args: (seen.append(where), real(dev, stream, where, args)))
    for stream in (None, torch.cuda.current_stream(dev)):
        lens, new = to_dev_i32([3, 15, 0, 31, 7], dev), torch.ones(S, dtype=torch.int32, device=dev)
        tables = torch.zeros((2, S, 3), dtype=torch.int32, device=dev)
        tables[:, 3, 1], tables[:, :, 0] = 4, torch.arange(S, dtype=torch.int32, device=dev)
        stack, count = lib.new_free_pages(20, dev)
        count -= 6
        pos, seq = (torch.zeros(S, dtype=torch.int32, device=dev) for _ in range(2))
        slots = torch.zeros((2, S), dtype=torch.int32, device=dev)
        pool, err = lib.new_int4_pool(20, dev), torch.zeros(1, dtype=torch.int32, device=dev)
        qo, out = (torch.zeros(S, 32, 64, dtype=torch.bfloat16, device=dev) for _ in range(2))
        ws = lib.alloc_int4_workspace(S, dev)
        cu = lib.grow_block_tables(lens, new, tables, stack, count, positions=pos, token_seq=seq, slots=slots, d_err=err, stream=stream)
        lib.kv_append_rope_int4(k, v, cu, lens, tables[0], pool, cos, sin, q, qo, err, stream=stream)
        wide = lib.kv_read_int4(pool, tables[0, 3].contiguous(), torch.empty((3, 2, 8, 16, 64), dtype=torch.bfloat16, device=dev), err, stream=stream)
        lib.paged_gqa_decode_int4(qo, pool, tables[0], lens, out, 0.125, workspace=ws, max_seq_len=48, d_err=err, stream=stream)
        ids = lib.sample_logits(x, e, top_p=torch.full((S,), 0.5, device=dev), logprobs=(lp := torch.empty(S, device=dev)), stream=stream)
        kept_lens = lens.clone()
        lib.release_pages(lens, to_dev_i32([0, 1, 0, 0, 1], dev) > 0, tables, stack, count, d_err=err, stream=stream)
        torch.cuda.synchronize(dev)
        assert lib.pkv_read_device_error(err) == 0
        got.append([kept_lens, lens, tables, stack, count, pos, seq, slots, cu, pool, qo, out, wide, ids, lp])
        assert len(seen) == (0 if stream is None else 6), seen
    for a, b in zip(*got):
        assert torch.equal(a, b)
    with pytest.raises(ValueError, match="num_seqs"):
        lib.paged_gqa_decode_int4(qo, pool, tables[0, :3].contiguous(), lens, out, 0.125)
    with pytest.raises(lib.PkvError, match="WORKSPACE"):
        lib.paged_gqa_decode_int4(qo, pool, tables[0], lens, out, 0.125, workspace=ws[:16])
    with pytest.raises(ValueError, match="slots must have"):
        lib.grow_block_tables(lens, new, tables, stack, count, positions=pos, slots=slots[:, :2].contiguous())
    with pytest.raises(ValueError, match="overlap"):
        lib.grow_block_tables(lens, new, tables[:1].expand(2, -1, -1), stack, count)
    with pytest.raises(TypeError, match="finished"):
        lib.release_pages(lens, lens, tables, stack, count)
