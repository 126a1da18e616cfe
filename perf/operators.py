"""Cases and plain forms of the cache and token operators.

Four operators of a decode loop over 16-token pages (32 query heads, 8 KV
heads of dimension 64):

  norm_rope  the heads of q and k normalised (RMS) and rotated in one pass --
             part of the head, either pair layout, tables scaled for long
             contexts -- and k, v written into bf16 pages
  append     k, v written into pages of 8-bit codes with one scale for each
             block of 16 tokens, head and K or V; the written pages read back
             as bf16 pages
  decode     attention of one query token per sequence over such pages
  logits     repetition, presence and frequency penalties, sparse biases and
             a grammar's bit mask on the logits, and the next token

Where `own` is false, run() computes them from elementary torch operations in
32 bits; where it is true, by the package's calls.  exact() computes them in
64 bits from the definitions.
"""
import math
import random

import torch

own = False

HQ, HKV, D, PAGE = 32, 8, 64, 16
VOCAB = 128256
CODE_MAX = {"int8": 127.0, "e4m3": 448.0}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one sequence's token: only latency counts
        dict(name="norm_rope token", op="norm_rope", tokens=1, pairs=32, interleaved=False, norm=True,
             append=True, fused_rows=True, scaling="none", ctx=2048),
        # a decode step of 257 sequences, q/k/v as slices of the projection's rows, half of the head rotated
        dict(name="norm_rope step", op="norm_rope", tokens=257, pairs=16, interleaved=True, norm=True,
             append=True, fused_rows=True, scaling="none", ctx=2048),
        # prompts of a long-context model into the cache
        dict(name="norm_rope prompt", op="norm_rope", tokens=32768, pairs=32, interleaved=False, norm=True,
             append=True, fused_rows=False, scaling="yarn", ctx=32768),
        # the new token of each of 32 sequences, inside pages that are partly filled
        dict(name="append step", op="append", seqs=32, new=1, held=2047, ragged=True, codes="int8", rope=True),
        # eight ragged prompts, the longest 4095 tokens, one of them continuing a page
        dict(name="append prompts", op="append", seqs=8, new=4095, held=9, ragged=True, codes="e4m3", rope=True),
        # a single short request
        dict(name="decode single", op="decode", seqs=1, tokens=37, ragged=False, codes="e4m3"),
        # the batch of the decode benchmark
        dict(name="decode batch", op="decode", seqs=32, tokens=2048, ragged=False, codes="int8"),
        # mixed lengths, an empty sequence among them
        dict(name="decode mixed", op="decode", seqs=97, tokens=8191, ragged=True, codes="e4m3"),
        # one long document
        dict(name="decode long", op="decode", seqs=1, tokens=131071, ragged=False, codes="int8"),
        # greedy decoding of one request under a grammar
        dict(name="logits one row", op="logits", rows=1, vocab=VOCAB, dtype="float32", history=500, bias=0,
             mask=True, penalties=True, write=False),
        # a batch of half-precision logits with every feature, logits kept for sampling
        dict(name="logits batch", op="logits", rows=32, vocab=VOCAB, dtype="bfloat16", history=2048, bias=17,
             mask=True, penalties=True, write=True),
        # a large batch in 32 bits
        dict(name="logits large", op="logits", rows=256, vocab=VOCAB, dtype="float32", history=1024, bias=300,
             mask=False, penalties=True, write=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "decode", "logits"])
    if op == "norm_rope":
        t = _log(rng, 1, 32768)
        return dict(op=op, tokens=t, pairs=rng.choice([4, 8, 11, 16, 20, 24, 32]),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.7, append=rng.random() < 0.7,
                    fused_rows=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "yarn"]),
                    ctx=max(t, _log(rng, 2048, 65536)))
    if op == "append":
        s = _log(rng, 1, 128)
        return dict(op=op, seqs=s, new=_log(rng, 1, max(1, min(4096, 32768 // s))), held=rng.randint(0, 3000),
                    ragged=rng.random() < 0.7, codes=rng.choice(["int8", "e4m3"]), rope=rng.random() < 0.7)
    if op == "decode":
        s = _log(rng, 1, 256)
        return dict(op=op, seqs=s, tokens=_log(rng, 1, max(16, min(131072, 390000 // s))),
                    ragged=rng.random() < 0.6, codes=rng.choice(["int8", "e4m3"]))
    r = _log(rng, 1, 200)
    return dict(op=op, rows=r, vocab=_log(rng, 1000, 160000), dtype=rng.choice(["float32", "bfloat16", "float16"]),
                history=_log(rng, 1, 4096), bias=rng.choice([0, 1, 33, 300]), mask=rng.random() < 0.6,
                penalties=rng.random() < 0.8, write=rng.random() < 0.6)


def _spread(case, count, most):
    """`count` whole numbers of 0..most, the largest of them `most`, the same for the same case."""
    if not case["ragged"]:
        return [most] * count
    r = random.Random("%d %d" % (count, most))
    got = [r.randint(0, most) for _ in range(count)]
    got[r.randrange(count)] = most
    if count > 4:
        got[(got.index(most) + 1) % count] = 0
    return got


def _append_lens(case):
    """New tokens and tokens held before, for each sequence."""
    if case["new"] == 1:
        new = [1] * case["seqs"]
    else:
        new = _spread(case, case["seqs"], case["new"])
    r = random.Random("held %d %d" % (case["seqs"], case["held"]))
    held = [r.randint(0, case["held"]) if case["ragged"] else case["held"] for _ in new]
    return new, held


def work(case):
    if case["op"] == "norm_rope":
        t, heads = case["tokens"], HQ + HKV + (HKV if case["append"] else 0)
        return {"bytes": t * (heads * D * 2 * 2 + 8 * case["pairs"] + 8) + 512, "flops": t * (HQ + HKV) * D * 8}
    if case["op"] == "append":
        new, held = _append_lens(case)
        t, pages = sum(new), sum(-(-(n + h) // PAGE) - h // PAGE for n, h in zip(new, held) if n)
        old = sum(h % PAGE for n, h in zip(new, held) if n)
        return {"bytes": t * HKV * D * 2 * (2 + 1) + old * HKV * D * 2 * 2 +  # rows read, codes written, held codes
                (t * (HQ * D * 2 * 2 + 8 * 32) if case["rope"] else 0) +  # q and the tables' rows
                pages * HKV * D * PAGE * 2 * 3,  # pages read back
                "flops": t * HKV * D * 2 * 4}
    if case["op"] == "decode":
        lens = _spread(case, case["seqs"], case["tokens"])
        pages = sum(-(-n // PAGE) for n in lens)
        return {"bytes": sum(lens) * HKV * D * 2 + pages * (HKV * 2 * 4 + 4) + len(lens) * (HQ * D * 2 * 2 + 4),
                "flops": 4 * HQ * D * sum(lens)}
    n = case["rows"] * case["vocab"]
    es = 4 if case["dtype"] == "float32" else 2
    return {"bytes": n * (es + (4 if case["write"] else 0)) + (n // 8 if case["mask"] else 0) +
            case["rows"] * ((case["history"] * 2 if case["penalties"] else 0) + case["bias"] * 8 + 4),
            "flops": n * 2}


# ------------------------------------------------------------------ inputs --

def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _int(values, dev):
    return torch.tensor(values, dtype=torch.int32).to(dev)


def _tables(pairs, ctx, scaling, dev):
    """cos and sin [ctx][pairs] of plain, linearly scaled or YaRN-scaled frequencies (a context eight times the original)."""
    theta, factor = 500000.0, 8.0
    i = torch.arange(pairs, dtype=torch.float64, device=dev)
    f, mul = theta ** (-i / pairs), 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        orig = max(1.0, ctx / factor)
        at = [pairs * math.log(orig / (turns * 2 * math.pi)) / math.log(theta) for turns in (32.0, 1.0)]
        lo, hi = max(0, math.floor(at[0])), min(2 * pairs - 1, math.ceil(at[1]))
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f, mul = f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    a = torch.arange(ctx, dtype=torch.float64, device=dev)[:, None] * f
    return (a.cos() * mul).float(), (a.sin() * mul).float()


def _block_tables(lens, spare, gen, dev):
    """Shuffled pages for sequences of these lengths, -1 behind them, and the number of pages."""
    need = [-(-n // PAGE) for n in lens]
    width = max(1, max(need))
    total = sum(need) + spare
    perm = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    n = _int(need, dev).long()
    start = torch.cumsum(n, 0) - n
    col = torch.arange(width, device=dev)
    at = (start[:, None] + col).clamp(max=total - 1)
    return torch.where(col < n[:, None], perm[at], torch.full_like(perm[at], -1)), total


def _code_type(case):
    return torch.int8 if case["codes"] == "int8" else torch.float8_e4m3fn


def _random_codes(pages, case, gen, dev):
    """Codes and scales of pages as normal K and V rows leave them."""
    top = CODE_MAX[case["codes"]]
    x = torch.randn((pages, 2, HKV, PAGE, D), generator=gen, device=dev)
    x.mul_(top / 3.7).clamp_(-top, top)
    codes = x.round_().to(torch.int8) if case["codes"] == "int8" else x.to(torch.float8_e4m3fn)
    scales = torch.exp(0.5 * torch.randn((pages, 2, HKV), generator=gen, device=dev)) * (3.7 / top)
    return codes, scales


def prepare(case, seed):
    dev = _dev()
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    bf = torch.bfloat16

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev).to(bf)

    st = {"case": case}
    if case["op"] == "norm_rope":
        t = case["tokens"]
        st["cos"], st["sin"] = _tables(case["pairs"], case["ctx"], case["scaling"], dev)
        # a prompt: the tokens of one row in order; a step: one token of each row, anywhere
        prompt = t > 1024
        pos = (torch.arange(t, device=dev) if prompt else torch.randint(0, case["ctx"], (t,), generator=g, device=dev))
        st["positions"] = pos.to(torch.int32)
        st["token_seq"] = torch.zeros(t, dtype=torch.int32, device=dev) if prompt else None
        if case["fused_rows"]:
            qkv = normal(t, HQ + 2 * HKV, D)
            st["q"], st["k"], st["v"] = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
        else:
            st["q"], st["k"], st["v"] = normal(t, HQ, D), normal(t, HKV, D), normal(t, HKV, D)
        st["qw"], st["kw"] = ((1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(bf) if case["norm"] else None
                              for _ in range(2))
        st["q_out"] = torch.zeros((t, HQ, D), dtype=bf, device=dev)
        st["k_out"] = None if case["append"] else torch.zeros((t, HKV, D), dtype=bf, device=dev)
        if case["append"]:
            if prompt:
                st["tables"], pages = _block_tables([t], 3, g, dev)
            else:  # each row's only allocated page is the one that its token goes to
                pages = t + 3
                perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
                st["tables"] = torch.full((t, -(-case["ctx"] // PAGE)), -1, dtype=torch.int32, device=dev)
                st["tables"].scatter_(1, (pos // PAGE)[:, None], perm[:t, None])
            st["pool"] = torch.zeros((pages, 2, HKV, PAGE, D), dtype=bf, device=dev)
        st["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
    elif case["op"] == "append":
        new, held = _append_lens(case)
        total = [n + h for n, h in zip(new, held)]
        t = sum(new)
        st["k"], st["v"] = normal(t, HKV, D), normal(t, HKV, D)
        st["cu"] = _int([0] + [sum(new[:i + 1]) for i in range(len(new))], dev)
        st["lens"] = _int(total, dev)
        if case["rope"]:
            st["q"], st["q_out"] = normal(t, HQ, D), torch.zeros((t, HQ, D), dtype=bf, device=dev)
            st["cos"], st["sin"] = _tables(32, max(16, max(total)), "none", dev)
        # pages before the first one that is written stay unread: the sequences' tables start there with any page
        first = [h // PAGE for h in held]
        need = [max(0, -(-n // PAGE) - f) if m else 0 for n, f, m in zip(total, first, new)]
        tb, pages = _block_tables([n * PAGE for n in need], 3, g, dev)
        width = max(1, max(f + n for f, n in zip(first, need)))
        full = torch.zeros((len(new), width + 1), dtype=torch.int32, device=dev)
        col = torch.arange(tb.shape[1], device=dev)[None]
        at = torch.where(tb >= 0, col + _int(first, dev).long()[:, None], torch.full_like(col, width))
        full.scatter_(1, at, tb.clamp(min=0))
        st["tables"] = full[:, :width].contiguous()
        st["pages"] = tb[tb >= 0].contiguous()  # the pages written
        st["pool"], st["scales"] = _random_codes(pages, case, g, dev)
        st["read"] = torch.zeros((st["pages"].numel(), 2, HKV, PAGE, D), dtype=bf, device=dev)
        st["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
    elif case["op"] == "decode":
        lens = _spread(case, case["seqs"], case["tokens"])
        st["tables"], pages = _block_tables(lens, 3, g, dev)
        st["pool"], st["scales"] = _random_codes(pages, case, g, dev)
        st["lens"] = _int(lens, dev)
        st["q"] = normal(case["seqs"], HQ, D)
        st["out"] = torch.zeros((case["seqs"], HQ, D), dtype=bf, device=dev)
        st["longest"] = max(lens)
        st["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
    else:
        r, v, h = case["rows"], case["vocab"], case["history"]
        st["logits"] = (3 * torch.randn((r, v), generator=g, device=dev)).to(getattr(torch, case["dtype"]))
        if case["penalties"]:
            # tokens repeat as text does: squares of uniforms gather at the low ids
            st["history"] = (torch.rand((r, h), generator=g, device=dev).square() * v).long().clamp(0, v - 1).to(torch.int32)
            st["hist_lens"] = torch.randint(0, h + 1, (r,), generator=g, device=dev).to(torch.int32)
            st["prompt_lens"] = (st["hist_lens"] * torch.rand(r, generator=g, device=dev)).to(torch.int32)
            st["rep"] = 1 + 0.3 * torch.rand(r, generator=g, device=dev)
            st["pres"] = torch.rand(r, generator=g, device=dev) - 0.2
            st["freq"] = 0.5 * torch.rand(r, generator=g, device=dev)
        if case["bias"]:
            st["bias_ids"] = torch.randint(-1, v, (r, case["bias"]), generator=g, device=dev).to(torch.int32)
            st["bias"] = 2 * torch.randn((r, case["bias"]), generator=g, device=dev)
        if case["mask"]:
            words = -(-v // 32)
            st["mask"] = torch.randint(-2 ** 31, 2 ** 31, (r, words), generator=g, device=dev).to(torch.int32)
        st["out"] = torch.zeros((r, v), device=dev) if case["write"] else None
        st["ids"] = torch.zeros(r, dtype=torch.int32, device=dev)
    return st


# -------------------------------------------------------------- plain forms --

def _norm(x, w):
    x = x.float()
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()


def _rotate(x, c, s, interleaved):
    """x [T, heads, 64] with the first 2 * pairs dims rotated; c, s [T, pairs]."""
    c, s, p = c[:, None], s[:, None], c.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * p:2], x[..., 1:2 * p:2]
        turned = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    else:
        a, b = x[..., :p], x[..., p:2 * p]
        turned = torch.cat((a * c - b * s, a * s + b * c), -1)
    return torch.cat((turned, x[..., 2 * p:]), -1)


def _plain_norm_rope(st):
    pos = st["positions"].long()
    c, s = st["cos"][pos], st["sin"][pos]
    turn = st["case"]["interleaved"]
    q = _rotate(_norm(st["q"], st["qw"]), c, s, turn).to(torch.bfloat16)
    k = _rotate(_norm(st["k"], st["kw"]), c, s, turn).to(torch.bfloat16)
    if not st["case"]["append"]:
        return {"q": q, "k": k}
    row = torch.arange(len(pos), device=pos.device) if st["token_seq"] is None else st["token_seq"].long()
    page = st["tables"][row, pos // PAGE].long()
    st["pool"][page, 0, :, pos % PAGE] = k
    st["pool"][page, 1, :, pos % PAGE] = st["v"]
    return {"q": q, "pool": st["pool"]}


def _quantise(x, scale, codes):
    """Codes of x under a scale that broadcasts, as 32-bit values."""
    y = torch.where(scale > 0, x / scale, torch.zeros_like(x))
    if codes == "int8":
        return y.round().clamp(-127, 127)
    return y.clamp(-448, 448).to(torch.float8_e4m3fn).float()


def _store(pool, page, slot, rows):
    """rows [n, 2, heads, D] of code values into the pool (seen as bytes: 8-bit floats have no indexed writes)."""
    rows = rows.to(pool.dtype)
    pool.view(torch.int8)[page, :, :, slot] = rows.view(torch.int8)


def _plain_append(st):
    case, pool, scales = st["case"], st["pool"], st["scales"]
    cu, lens = st["cu"].long(), st["lens"].long()
    t, dev = st["k"].shape[0], st["k"].device
    tok = torch.arange(t, device=dev)
    row = torch.searchsorted(cu, tok, right=True) - 1
    held = lens - (cu[1:] - cu[:-1])
    pos = held[row] + tok - cu[row]
    k, got = st["k"].float(), {}
    if case["rope"]:
        c, s = st["cos"][pos], st["sin"][pos]
        got["q"] = _rotate(st["q"].float(), c, s, False).to(torch.bfloat16)
        k = _rotate(k, c, s, False).to(torch.bfloat16).float()
    x = torch.stack((k, st["v"].float()), 1)  # [T, 2, heads, D]
    page, slot = st["tables"][row, pos // PAGE].long(), pos % PAGE
    top = torch.full((1,), CODE_MAX[case["codes"]], device=dev)
    amax = torch.zeros_like(scales)
    amax.scatter_reduce_(0, page[:, None, None].expand(t, 2, HKV), x.abs().amax(-1), "amax")
    fresh = amax / top
    # sequences whose first new token continues a page
    part = (held % PAGE > 0) & (cu[1:] > cu[:-1])
    p0 = st["tables"].gather(1, (held // PAGE).clamp(max=st["tables"].shape[1] - 1)[:, None])[:, 0].long()[part]
    old = scales[p0]
    fresh[p0] = torch.maximum(old, fresh[p0])
    grown = fresh[p0] > old
    value = pool.view(torch.int8)[p0].view(pool.dtype).float() * old[..., None, None]
    again = _quantise(value, fresh[p0][..., None, None], case["codes"]).to(pool.dtype).view(torch.int8)
    keep = pool.view(torch.int8)[p0]
    was = torch.arange(PAGE, device=dev)[:, None] < (held[part] % PAGE)[:, None, None, None, None]
    pool.view(torch.int8)[p0] = torch.where(grown[..., None, None] & was, again, keep)
    scales[page] = fresh[page]
    _store(pool, page, slot, _quantise(x, fresh[page][..., None], case["codes"]))
    at = st["pages"].long()
    got["scales"] = scales
    got["read"] = (pool.view(torch.int8)[at].view(pool.dtype).float() * scales[at][..., None, None]).to(torch.bfloat16)
    return got


def _plain_decode(st):
    tb, lens = st["tables"].long(), st["lens"].long()
    s, m = tb.shape
    n = m * PAGE
    at = tb.clamp(min=0)
    x = st["pool"].view(torch.int8)[at].view(st["pool"].dtype).float() * st["scales"][at][..., None, None]
    x = x.permute(2, 0, 3, 1, 4, 5).reshape(2, s, HKV, n, D)  # K, V by sequence and head
    q = st["q"].float().view(s, HKV, HQ // HKV, D)
    live = (torch.arange(n, device=tb.device) < lens[:, None])[:, None, None]
    score = (q @ x[0].transpose(-1, -2)) * 0.125
    score = torch.where(live, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top.isinf(), torch.zeros_like(top), top))
    v = torch.where(live[:, :, 0, :, None], x[1], torch.zeros_like(x[1]))
    out = (p @ v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return out.reshape(s, HQ, D).to(torch.bfloat16)


def _plain_logits(st):
    case, x = st["case"], st["logits"].float()
    r, v = x.shape
    dev = x.device
    if case["penalties"]:
        at = torch.arange(case["history"], device=dev)
        ids = torch.where(at < st["hist_lens"][:, None], st["history"], v).long()
        made = ((at >= st["prompt_lens"][:, None]) & (ids < v)).float()
        seen = torch.zeros((r, v + 1), dtype=torch.bool, device=dev).scatter_(1, ids, True)[:, :v]
        count = torch.zeros((r, v + 1), device=dev).scatter_add_(1, ids, made)[:, :v]
        rep = st["rep"][:, None]
        x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
        x = x - st["freq"][:, None] * count
        x = x - torch.where(count > 0, st["pres"][:, None], torch.zeros_like(x))
    if case["bias"]:
        ids = torch.where(st["bias_ids"] >= 0, st["bias_ids"], v).long()
        entry = torch.arange(1, case["bias"] + 1, device=dev).expand(r, -1)  # the last entry of an id counts
        last = torch.zeros((r, v + 1), dtype=torch.int64, device=dev).scatter_reduce_(1, ids, entry, "amax")[:, :v]
        value = torch.cat((torch.zeros((r, 1), device=dev), st["bias"]), 1).gather(1, last)
        x = torch.where(last > 0, x + value, x)
    ok = ~x.isnan()
    if case["mask"]:
        i = torch.arange(v, device=dev)
        allowed = (st["mask"][:, i >> 5] >> (i & 31)) & 1 != 0
        x, ok = torch.where(allowed, x, torch.full_like(x, -math.inf)), ok & allowed
    top = torch.where(ok, x, torch.full_like(x, -math.inf)).amax(1, keepdim=True)
    first = torch.where(ok & (x == top), torch.arange(v, device=dev), v).amin(1)
    ids = torch.where(first < v, first, -1).to(torch.int32)
    return {"ids": ids, "logits": x} if case["write"] else {"ids": ids}


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    if op == "norm_rope":
        return _plain_norm_rope(state)
    if op == "append":
        return _plain_append(state)
    if op == "decode":
        return _plain_decode(state)
    return _plain_logits(state)


# ---------------------------------------------------- the package's own calls --

def _own(op, st):
    import paged_kv_gqa_append_gb300 as pkv
    case = st["case"]
    if op == "norm_rope":
        opts = dict(q_weight=st["qw"], k_weight=st["kw"], eps=1e-6, interleaved=case["interleaved"], d_err=st["err"])
        if not case["append"]:
            pkv.qk_norm_rope(st["q"], st["k"], st["positions"], st["cos"], st["sin"], st["q_out"], st["k_out"], **opts)
            return {"q": st["q_out"], "k": st["k_out"]}
        pkv.kv_append_norm_rope(st["k"], st["v"], st["positions"], st["tables"], st["pool"], st["cos"], st["sin"],
                                token_seq=st["token_seq"], q_in=st["q"], q_out=st["q_out"], **opts)
        return {"q": st["q_out"], "pool": st["pool"]}
    if op == "append":
        turn = dict(rope_cos=st["cos"], rope_sin=st["sin"], q_in=st["q"], q_out=st["q_out"]) if case["rope"] else {}
        pkv.kv_append_rope_bs8(st["k"], st["v"], st["cu"], st["lens"], st["tables"], st["pool"], st["scales"],
                               d_err=st["err"], **turn)
        pkv.kv_read_bs8(st["pool"], st["scales"], st["pages"], st["read"], d_err=st["err"])
        got = {"scales": st["scales"], "read": st["read"]}
        return dict(got, q=st["q_out"]) if case["rope"] else got
    if op == "decode":
        if "workspace" not in st:
            st["workspace"] = pkv.alloc_bs8_workspace(case["seqs"], st["q"].device)
        pkv.paged_gqa_decode_bs8(st["q"], st["pool"], st["scales"], st["tables"], st["lens"], st["out"], 0.125,
                                 workspace=st["workspace"], max_seq_len=st["longest"], d_err=st["err"])
        return st["out"]
    ids = pkv.process_logits(st["logits"], out=st["out"], ids=st["ids"], history=st.get("history"),
                             history_lens=st.get("hist_lens"), prompt_lens=st.get("prompt_lens"),
                             repetition=st.get("rep"), presence=st.get("pres"), frequency=st.get("freq"),
                             bias_ids=st.get("bias_ids"), bias_values=st.get("bias"), allow_mask=st.get("mask"))
    return {"ids": ids, "logits": st["out"]} if case["write"] else {"ids": ids}


# ------------------------------------------------------------ in 64 bits --

def _exact_heads(x, w, cos, sin, interleaved):
    """One tensor's heads normalised and rotated, as complex products."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + 1e-6) * w.double()
    p = cos.shape[1]
    turn = torch.complex(cos.double(), sin.double())[:, None]
    y = x.clone()
    if interleaved:
        z = torch.view_as_complex(x[..., :2 * p].reshape(*x.shape[:-1], p, 2).contiguous()) * turn
        y[..., :2 * p] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :p].contiguous(), x[..., p:2 * p].contiguous()) * turn
        y[..., :p], y[..., p:2 * p] = z.real, z.imag
    return y


def _exact_codes(x, scale, codes):
    # the definition's quotient is a 32-bit one: a tie between two codes is decided by it
    y = torch.where(scale > 0, x / scale, 0.0).float().double()
    if codes == "int8":
        return torch.round(y).clamp(-127, 127)
    # e4m3: three bits behind the leading one, the smallest step 2^-9
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def exact(case, seed):
    st = prepare(case, seed)
    dev = st["q"].device if "q" in st else _dev()
    if case["op"] == "norm_rope":
        pos = st["positions"].long()
        c, s = st["cos"][pos], st["sin"][pos]
        q = _exact_heads(st["q"], st["qw"], c, s, case["interleaved"])
        k = _exact_heads(st["k"], st["kw"], c, s, case["interleaved"])
        if not case["append"]:
            return {"q": q, "k": k}
        pool = st["pool"].double()
        row = st["token_seq"].long() if st["token_seq"] is not None else torch.arange(len(pos), device=dev)
        flat = pool.permute(0, 3, 1, 2, 4).reshape(-1, 2, HKV, D)  # one row for each slot of the pool
        flat[st["tables"][row, pos // PAGE].long() * PAGE + pos % PAGE] = torch.stack((k, st["v"].double()), 1)
        return {"q": q, "pool": flat.reshape(-1, PAGE, 2, HKV, D).permute(0, 2, 3, 1, 4).contiguous()}
    if case["op"] == "append":
        new, held = _append_lens(case)
        if case["seqs"] > 256:
            return None
        top = CODE_MAX[case["codes"]]
        value, scales = st["pool"].to(torch.float64), st["scales"].double()
        got, at = {}, 0
        turned = st["k"].double()
        if case["rope"]:
            pos = torch.cat([torch.arange(h, h + n) for n, h in zip(new, held)]).to(dev)
            got["q"] = _exact_heads(st["q"], None, st["cos"][pos], st["sin"][pos], False)
            turned = _exact_heads(st["k"], None, st["cos"][pos], st["sin"][pos], False).to(torch.bfloat16).double()
        rows = torch.stack((turned, st["v"].double()), 1)
        tables = st["tables"].cpu()
        for s, (n, h) in enumerate(zip(new, held)):
            p = h
            while p < h + n:
                size = min(PAGE - p % PAGE, h + n - p)
                page, slot = int(tables[s, p // PAGE]), p % PAGE
                x = rows[at:at + size].permute(1, 2, 0, 3)  # K and V, heads, tokens, dims
                sc = x.abs().amax((-1, -2)).div(top).float().double()
                if slot:
                    old = scales[page]
                    sc = torch.maximum(sc, old)
                    again = _exact_codes(value[page, :, :, :slot] * old[..., None, None], sc[..., None, None], case["codes"])
                    value[page, :, :, :slot] = torch.where((sc > old)[..., None, None], again, value[page, :, :, :slot])
                value[page, :, :, slot:slot + size] = _exact_codes(x, sc[..., None, None], case["codes"])
                scales[page] = sc
                p, at = p + size, at + size
        pages = st["pages"].long()
        got["scales"], got["read"] = scales, value[pages] * scales[pages][..., None, None]
        return got
    if case["op"] == "decode":
        out = torch.zeros((case["seqs"], HQ, D), dtype=torch.float64, device=dev)
        for s, n in enumerate(st["lens"].tolist()):
            if n == 0:
                continue
            pages = st["tables"][s, :-(-n // PAGE)].long()
            raw = st["pool"].view(torch.int8)[pages].view(st["pool"].dtype).to(torch.float64)
            kv = (raw * st["scales"][pages].double()[..., None, None]).permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :n]
            q = st["q"][s].double().unflatten(0, (HKV, HQ // HKV))
            w = torch.softmax(torch.einsum("hgd,hnd->hgn", q, kv[0]) / 8, -1)
            out[s] = torch.einsum("hgn,hnd->hgd", w, kv[1]).flatten(0, 1)
        return out
    if not case["write"]:
        return None  # ids alone: whole numbers
    x = st["logits"].double()
    r, v = x.shape
    for i in range(r):
        if case["penalties"]:
            n, m = int(st["hist_lens"][i]), int(st["prompt_lens"][i])
            past = st["history"][i, :n].long()
            every, made = torch.bincount(past, minlength=v), torch.bincount(past[m:], minlength=v)
            rep = st["rep"][i].double()
            x[i] = torch.where(every > 0, torch.where(x[i] > 0, x[i] / rep, x[i] * rep), x[i])
            x[i] -= made * st["freq"][i].double() + (made > 0) * st["pres"][i].double()
        if case["bias"]:
            ids, val = st["bias_ids"][i].tolist(), st["bias"][i].tolist()
            last = {k: b for k, b in zip(ids, val) if k >= 0}
            if last:
                at = torch.tensor(list(last), device=dev)
                x[i, at] += torch.tensor(list(last.values()), dtype=torch.float64, device=dev)
        if case["mask"]:
            shift = torch.arange(32, device=dev)
            allowed = ((st["mask"][i][:, None].long() >> shift) & 1).flatten()[:v] != 0
            x[i, ~allowed] = -math.inf
    return {"ids": None, "logits": x}
