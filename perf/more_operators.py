"""Cases and plain forms of the 4-bit cache, the page tables and the sampler.

Operators of a decode loop over 16-token pages (32 query heads, 8 KV heads of
dimension 64) that stays on the GPU from one step to the next:

  tables  pages for every request's new tokens taken from the stack of free
          ones, with the rows' offsets, positions and slots ("grow"), and the
          pages of finished requests put back ("release")
  append  k, v written into pages of 4-bit codes with a scale and a minimum
          for each token and head; the written pages read back as bf16 pages
  decode  attention of one query token per sequence over such pages
  sample  the next token by temperature, top-k, top-p and min-p from given
          exponential variates, and its log-probability

Where `own` is false, run() computes them from elementary torch operations;
where it is true, by the package's calls.  exact() computes them in 64 bits
from the definitions.
"""
import math
import random

import torch

own = False

HQ, HKV, D, PAGE = 32, 8, 64, 16
BLOCK = 1152  # bytes of a page's head: 512 of K, 512 of V, 128 of scales and minima
VOCAB = 128256


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # a decode step of 32 requests: a sixteenth of them begin a page, in each of 16 layers
        dict(name="tables step", op="tables", kind="grow", rows=32, layers=16, new=1, held=2047),
        # the prompts of 64 requests of a continuous batch
        dict(name="tables prompts", op="tables", kind="grow", rows=64, layers=16, new=1920, held=0),
        # about half of a batch of 256 requests finished
        dict(name="tables release", op="tables", kind="release", rows=256, layers=16, new=0, held=2048),
        # the new token of each of 32 sequences, inside pages that are partly filled
        dict(name="append step", op="append", seqs=32, new=1, held=2047, ragged=True, rope=True),
        # eight ragged prompts, the longest 4095 tokens, behind a few held tokens each
        dict(name="append prompts", op="append", seqs=8, new=4095, held=9, ragged=True, rope=True),
        # a single short request
        dict(name="decode single", op="decode", seqs=1, tokens=37, ragged=False),
        # the batch of the decode benchmark
        dict(name="decode batch", op="decode", seqs=32, tokens=2048, ragged=False),
        # mixed lengths, an empty sequence among them
        dict(name="decode mixed", op="decode", seqs=97, tokens=8191, ragged=True),
        # one long document
        dict(name="decode long", op="decode", seqs=1, tokens=131071, ragged=False),
        # one request with top-k and top-p
        dict(name="sample one row", op="sample", rows=1, vocab=VOCAB, dtype="float32", top_k=50, top_p=0.9, min_p=0.0,
             greedy=0),
        # a batch of half-precision logits with top-p and min-p, a few rows greedy
        dict(name="sample batch", op="sample", rows=32, vocab=VOCAB, dtype="bfloat16", top_k=0, top_p=0.8, min_p=0.05,
             greedy=8),
        # a large batch in 32 bits, every row with its own limits
        dict(name="sample large", op="sample", rows=256, vocab=VOCAB, dtype="float32", top_k=200, top_p=0.7, min_p=0.02,
             greedy=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "decode", "sample"])
    if op == "tables":
        kind = rng.choice(["grow", "grow", "release"])
        rows, layers = _log(rng, 1, 1024), rng.choice([1, 2, 7, 16, 28])
        most = max(1, min(4096, 900000 // (rows * layers)))
        return dict(op=op, kind=kind, rows=rows, layers=layers, new=_log(rng, 1, most) if kind == "grow" else 0,
                    held=rng.randint(0, min(2048, 16 * most)))
    if op == "append":
        s = _log(rng, 1, 128)
        return dict(op=op, seqs=s, new=_log(rng, 1, max(1, min(4096, 32768 // s))), held=rng.randint(0, 3000),
                    ragged=rng.random() < 0.7, rope=rng.random() < 0.7)
    if op == "decode":
        s = _log(rng, 1, 256)
        return dict(op=op, seqs=s, tokens=_log(rng, 1, max(16, min(131072, 390000 // s))), ragged=rng.random() < 0.6)
    return dict(op=op, rows=_log(rng, 1, 200), vocab=_log(rng, 1000, 160000),
                dtype=rng.choice(["float32", "bfloat16", "float16"]), top_k=rng.choice([0, 0, 1, 40, 1000]),
                top_p=rng.choice([1.0, 0.95, 0.6]), min_p=rng.choice([0.0, 0.0, 0.1]), greedy=rng.choice([0, 3]))


def _spread(ragged, count, most):
    """`count` whole numbers of 0..most, the largest of them `most`, the same for the same case."""
    if not ragged:
        return [most] * count
    r = random.Random("%d %d" % (count, most))
    got = [r.randint(0, most) for _ in range(count)]
    got[r.randrange(count)] = most
    if count > 4:
        got[(got.index(most) + 1) % count] = 0
    return got


def _held(case, count):
    r = random.Random("held %d %d" % (count, case["held"]))
    return [r.randint(0, case["held"]) if case.get("ragged", True) else case["held"] for _ in range(count)]


def _append_lens(case):
    """New tokens and tokens held before, for each sequence."""
    new = [1] * case["seqs"] if case["new"] == 1 else _spread(case["ragged"], case["seqs"], case["new"])
    return new, _held(case, case["seqs"])


def _table_lens(case):
    """New tokens and tokens held, for each request, and whether it has finished."""
    n = case["rows"]
    new = [1] * n if case["new"] == 1 else _spread(True, n, case["new"])
    r = random.Random("done %d" % n)
    return new, _held(case, n), [r.random() < 0.5 or n == 1 for _ in range(n)]


def _blocks(n):
    return -(-n // PAGE)


def work(case):
    if case["op"] == "tables":
        new, held, done = _table_lens(case)
        layers, n = case["layers"], case["rows"]
        if case["kind"] == "release":
            pages = layers * sum(_blocks(h) for h, d in zip(held, done) if d)
            return {"bytes": pages * 8 + n * (4 + 1 + 4) + 8, "flops": pages}
        pages = layers * sum(_blocks(h + m) - _blocks(h) for m, h in zip(new, held))
        # the table entry of a page that new tokens continue is read too
        old = layers * sum(1 for m, h in zip(new, held) if m and h % PAGE)
        return {"bytes": pages * 8 + old * 4 + n * 16 + 12 + sum(new) * (8 + 4 * layers), "flops": sum(new) * layers}
    if case["op"] == "append":
        new, held = _append_lens(case)
        t, pages = sum(new), sum(_blocks(n + h) - h // PAGE for n, h in zip(new, held) if n)
        return {"bytes": t * HKV * (2 * D * 2 + 2 * (D // 2 + 4)) +           # rows read, codes written
                (t * (HQ * D * 2 * 2 + 8 * 32) if case["rope"] else 0) +      # q and the tables' rows
                pages * HKV * (BLOCK + 2 * PAGE * D * 2),                     # pages read back
                "flops": t * HKV * D * 2 * 4}
    if case["op"] == "decode":
        lens = _spread(case["ragged"], case["seqs"], case["tokens"])
        return {"bytes": sum(lens) * HKV * 2 * (D // 2 + 4) + sum(_blocks(n) for n in lens) * 4 +
                len(lens) * (HQ * D * 2 * 2 + 4), "flops": 4 * HQ * D * sum(lens)}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * ((4 if case["dtype"] == "float32" else 2) + 4) + case["rows"] * 24, "flops": n * 6}


# ------------------------------------------------------------------ inputs --

def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _int(values, dev):
    return torch.tensor(values, dtype=torch.int32).to(dev)


def _tables(ctx, dev):
    """cos and sin [ctx][32]."""
    f = 500000.0 ** (-torch.arange(32, dtype=torch.float64, device=dev) / 32)
    a = torch.arange(ctx, dtype=torch.float64, device=dev)[:, None] * f
    return a.cos().float(), a.sin().float()


def _block_tables(lens, spare, gen, dev):
    """Shuffled pages for sequences of these lengths, -1 behind them, and the number of pages."""
    need = [_blocks(n) for n in lens]
    width = max(1, max(need))
    total = sum(need) + spare
    perm = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    n = _int(need, dev).long()
    start = torch.cumsum(n, 0) - n
    col = torch.arange(width, device=dev)
    at = (start[:, None] + col).clamp(max=total - 1)
    return torch.where(col < n[:, None], perm[at], torch.full_like(perm[at], -1)), total


def _places(dev):
    """Where a block keeps the bytes of K and V [2, token, pair of dims] and the 32-bit words (scale, minimum) [2, token]."""
    kv, r, b = torch.meshgrid(torch.arange(2), torch.arange(PAGE), torch.arange(D // 2), indexing="ij")
    k_at = (4 * (r % 8) + b // 8) * 16 + r // 8 * 8 + b % 8
    v_at = 512 + (4 * (b // 4) + r % 8 // 2) * 16 + r // 8 * 8 + b % 4 // 2 * 4 + r % 2 * 2 + b % 2
    kv2, r2 = torch.meshgrid(torch.arange(2), torch.arange(PAGE), indexing="ij")
    words = 256 + r2 % 8 * 4 + kv2 * 2 + r2 // 8
    return torch.where(kv == 0, k_at, v_at).to(dev), words.to(dev)


def _random_pool(pages, gen, dev):
    """Pages as normal K and V rows of different sizes leave them."""
    pool = torch.empty((pages, HKV, BLOCK), dtype=torch.uint8, device=dev)
    at = _places(dev)
    for i in range(0, pages, 2048):
        n = min(2048, pages - i)
        x = torch.randn((n, HKV, 2, PAGE, D), generator=gen, device=dev)
        x *= torch.exp(0.3 * torch.randn((n, HKV, 2, PAGE, 1), generator=gen, device=dev))
        codes, scale, low = _quantise(x.to(torch.bfloat16).float())
        pool[i:i + n] = _pack(codes, scale, low, at)
    return pool


def prepare(case, seed):
    dev = _dev()
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    bf, i32 = torch.bfloat16, torch.int32

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev).to(bf)

    st = {"case": case, "err": torch.zeros(1, dtype=i32, device=dev)}
    if case["op"] == "tables":
        new, held, done = _table_lens(case)
        rows, layers = case["rows"], case["layers"]
        need = [_blocks(h) for h in held]
        more = [_blocks(h + n) - b for h, n, b in zip(held, new, need)]
        width = max(1, max(b + m for b, m in zip(need, more)))
        taken = layers * sum(need)
        pages = taken + layers * sum(more) + 100
        perm = torch.randperm(pages, generator=g, device=dev).to(i32)
        col = torch.arange(width, device=dev)
        n = _int(need, dev).long()
        start = torch.cumsum(n, 0) - n
        at = layers * start + n * torch.arange(layers, device=dev)[:, None]
        tb = perm[(at[..., None] + col).clamp(max=pages - 1)]
        st["tables"] = torch.where(col < n[:, None], tb, torch.full_like(tb, -1)).contiguous()
        # the stack: free pages below, room for the others above
        st["free"] = torch.cat((perm[taken:], torch.full((taken,), -1, dtype=i32, device=dev)))
        st["count"] = _int([pages - taken], dev)
        st["lens"] = _int(held, dev)
        st["lens_out"], st["count_out"] = torch.zeros_like(st["lens"]), torch.zeros_like(st["count"])
        if case["kind"] == "release":
            st["done"] = torch.tensor(done).to(dev)
            st["total"] = layers * sum(b for b, d in zip(need, done) if d)
        else:
            t = sum(new)
            st["new"] = _int(new, dev)
            st["total"] = layers * sum(more)
            st["cu"] = torch.zeros(rows + 1, dtype=i32, device=dev)
            st["positions"], st["token_seq"] = (torch.zeros(t, dtype=i32, device=dev) for _ in range(2))
            st["slots"] = torch.zeros((layers, t), dtype=i32, device=dev)
    elif case["op"] == "append":
        new, held = _append_lens(case)
        total = [n + h for n, h in zip(new, held)]
        t = sum(new)
        st["k"], st["v"] = normal(t, HKV, D), normal(t, HKV, D)
        st["cu"] = _int([0] + [sum(new[:i + 1]) for i in range(len(new))], dev)
        st["lens"] = _int(total, dev)
        if case["rope"]:
            st["q"], st["q_out"] = normal(t, HQ, D), torch.zeros((t, HQ, D), dtype=bf, device=dev)
            st["cos"], st["sin"] = _tables(max(16, max(total)), dev)
        # pages before the first one that is written stay unread: the sequences' tables start there with any page
        first = [h // PAGE for h in held]
        need = [max(0, _blocks(n) - f) if m else 0 for n, f, m in zip(total, first, new)]
        tb, pages = _block_tables([n * PAGE for n in need], 3, g, dev)
        width = max(1, max(f + n for f, n in zip(first, need)))
        full = torch.zeros((len(new), width + 1), dtype=i32, device=dev)
        col = torch.arange(tb.shape[1], device=dev)[None]
        at = torch.where(tb >= 0, col + _int(first, dev).long()[:, None], torch.full_like(col, width))
        full.scatter_(1, at, tb.clamp(min=0))
        st["tables"] = full[:, :width].contiguous()
        st["pages"] = tb[tb >= 0].contiguous()  # the pages written
        st["pool"] = _random_pool(pages, g, dev)
        st["read"] = torch.zeros((st["pages"].numel(), 2, HKV, PAGE, D), dtype=bf, device=dev)
    elif case["op"] == "decode":
        lens = _spread(case["ragged"], case["seqs"], case["tokens"])
        st["tables"], pages = _block_tables(lens, 3, g, dev)
        st["pool"] = _random_pool(pages, g, dev)
        st["lens"] = _int(lens, dev)
        st["q"] = normal(case["seqs"], HQ, D)
        st["out"] = torch.zeros((case["seqs"], HQ, D), dtype=bf, device=dev)
        st["longest"] = max(lens)
    else:
        r, v = case["rows"], case["vocab"]
        x = 2.5 * torch.randn((r, v), generator=g, device=dev)
        # a few tokens of each row stand out, as a model's continuations do
        near = torch.randint(0, v // 24, (r, 24), generator=g, device=dev) + torch.arange(24, device=dev) * (v // 24)
        x.scatter_(1, near, 8 + 2.5 * torch.randn((r, 24), generator=g, device=dev))
        st["logits"] = x.to(getattr(torch, case["dtype"]))
        st["noise"] = torch.empty((r, v), device=dev).exponential_(generator=g)
        st["temperature"] = 0.5 + torch.rand(r, generator=g, device=dev)
        if case["greedy"]:
            st["temperature"][::case["greedy"]] = 0
        if case["top_k"]:
            st["top_k"] = torch.randint(1, case["top_k"] + 1, (r,), generator=g, device=dev).to(i32)
        if case["top_p"] < 1:
            st["top_p"] = case["top_p"] + (1 - case["top_p"]) * torch.rand(r, generator=g, device=dev)
        if case["min_p"]:
            st["min_p"] = case["min_p"] * torch.rand(r, generator=g, device=dev)
        st["ids"] = torch.zeros(r, dtype=i32, device=dev)
        st["logprobs"] = torch.zeros(r, device=dev)
    return st


# -------------------------------------------------------------- plain forms --

def _plain_grow(st):
    lens, new, count = st["lens"].long(), st["new"].long(), st["count"].long()
    tables, dev = st["tables"], lens.device
    layers, rows, _ = tables.shape
    after = lens + new
    old = (lens + PAGE - 1) // PAGE
    more = (after + PAGE - 1) // PAGE - old
    cu = torch.cat((torch.zeros(1, dtype=torch.long, device=dev), torch.cumsum(new, 0)))
    # the i-th page taken: request by request, layer by layer, in order
    need = layers * more
    ends = torch.cumsum(need, 0)
    i = torch.arange(st["total"], device=dev)
    row = torch.searchsorted(ends, i, right=True)
    rest = i - (ends - need)[row]
    layer, block = rest // more[row], old[row] + rest % more[row]
    tables[layer, row, block] = st["free"][count - 1 - i]
    t = torch.arange(st["positions"].numel(), device=dev)
    seq = torch.searchsorted(cu[1:], t, right=True)
    pos = lens[seq] + t - cu[seq]
    slots = tables[:, seq, pos // PAGE] * PAGE + (pos % PAGE).to(torch.int32)
    i32 = torch.int32
    return {"tables": tables, "lens": after.to(i32), "count": (count - ends[-1:]).to(i32), "cu": cu.to(i32),
            "positions": pos.to(i32), "token_seq": seq.to(i32), "slots": slots}


def _plain_release(st):
    lens, done, count = st["lens"].long(), st["done"], st["count"].long()
    tables, free, dev = st["tables"], st["free"], lens.device
    layers = tables.shape[0]
    held = torch.where(done, (lens + PAGE - 1) // PAGE, torch.zeros_like(lens))
    need = layers * held
    ends = torch.cumsum(need, 0)
    i = torch.arange(st["total"], device=dev)
    row = torch.searchsorted(ends, i, right=True)
    rest = i - (ends - need)[row]
    free[count + i] = tables[rest // held[row], row, rest % held[row]]
    return {"free": free, "count": (count + ends[-1:]).to(torch.int32),
            "lens": torch.where(done, torch.zeros_like(lens), lens).to(torch.int32)}


def _rotate(x, c, s):
    """x [T, heads, 64]; c, s [T, 32]."""
    c, s = c[:, None], s[:, None]
    a, b = x[..., :32], x[..., 32:]
    return torch.cat((a * c - b * s, a * s + b * c), -1)


def _quantise(x):
    """Codes of rows x [..., 64] of bf16 values in 32 bits, and their scales and minima as bf16 values."""
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = ((high * 0.5 - low * 0.5) / 7.5).to(torch.bfloat16).float()
    scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
    inv = torch.where(scale > 0, 2.0 / scale, torch.zeros_like(scale))
    codes = ((x * 0.5 - low * 0.5) * inv).round().clamp(0, 15)
    return codes, scale, low


def _pack(codes, scale, low, at):
    """Blocks [..., 1152] of codes [..., 2, 16, 64], scales and minima [..., 2, 16, 1]."""
    bytes_at, words_at = at
    lead = codes.shape[:-3]
    c = codes.to(torch.uint8)
    block = torch.empty((*lead, BLOCK), dtype=torch.uint8, device=codes.device)
    block[..., bytes_at.flatten()] = (c[..., 0::2] | c[..., 1::2] << 4).flatten(-3)
    pair = torch.cat((scale, low), -1).to(torch.bfloat16).contiguous().view(torch.int32).flatten(-3)
    block.view(torch.int32)[..., words_at.flatten()] = pair
    return block


def _unpack(block, at):
    """Codes [..., 2, 16, 64], scales and minima [..., 2, 16, 1] of blocks, in 32 bits."""
    bytes_at, words_at = at
    b = block[..., bytes_at]
    codes = torch.stack((b & 15, b >> 4), -1).flatten(-2).float()
    pair = block.view(torch.int32)[..., words_at].contiguous().view(torch.bfloat16).unflatten(-1, (PAGE, 2)).float()
    return codes, pair[..., 0:1], pair[..., 1:2]


def _values(block, at):
    """[..., heads, 1152] -> [..., 2, heads, 16, 64]."""
    codes, scale, low = _unpack(block, at)
    return (low + codes * scale).transpose(-3, -4)


def _plain_append(st):
    case, pool = st["case"], st["pool"]
    cu, lens = st["cu"].long(), st["lens"].long()
    t, dev = st["k"].shape[0], st["k"].device
    tok = torch.arange(t, device=dev)
    row = torch.searchsorted(cu, tok, right=True) - 1
    pos = lens[row] - (cu[row + 1] - cu[row]) + tok - cu[row]
    k, got = st["k"].float(), {}
    if case["rope"]:
        c, s = st["cos"][pos], st["sin"][pos]
        got["q"] = _rotate(st["q"].float(), c, s).to(torch.bfloat16)
        k = _rotate(k, c, s).to(torch.bfloat16).float()
    codes, scale, low = _quantise(torch.stack((k, st["v"].float()), 1))  # [T, 2, heads, D]
    page, slot = st["tables"][row, pos // PAGE].long(), pos % PAGE
    at = _places(dev)
    c = codes.to(torch.uint8)
    both = (c[..., 0::2] | c[..., 1::2] << 4).transpose(1, 2)  # [T, heads, 2, 32]
    here, head = page[:, None, None, None], torch.arange(HKV, device=dev)[:, None, None]
    pool[here, head, at[0][:, slot].transpose(0, 1)[:, None]] = both
    pair = torch.cat((scale, low), -1).to(torch.bfloat16).view(torch.int32)[..., 0].transpose(1, 2)
    pool.view(torch.int32)[here[..., 0], head[..., 0], at[1][:, slot].transpose(0, 1)[:, None]] = pair
    got["read"] = _values(pool[st["pages"].long()], at).to(torch.bfloat16)
    return got


def _plain_decode(st):
    tb, lens = st["tables"].long(), st["lens"].long()
    s, m = tb.shape
    n = m * PAGE
    x = _values(st["pool"][tb.clamp(min=0)], _places(tb.device))  # [S, pages, 2, heads, 16, 64]
    x = x.permute(2, 0, 3, 1, 4, 5).reshape(2, s, HKV, n, D)
    q = st["q"].float().view(s, HKV, HQ // HKV, D)
    live = (torch.arange(n, device=tb.device) < lens[:, None])[:, None, None]
    score = (q @ x[0].transpose(-1, -2)) * 0.125
    score = torch.where(live, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top.isinf(), torch.zeros_like(top), top))
    v = torch.where(live[:, :, 0, :, None], x[1], torch.zeros_like(x[1]))
    out = (p @ v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return out.reshape(s, HQ, D).to(torch.bfloat16)


def _plain_sample(st):
    # in 64 bits: sums over the whole vocabulary decide which tokens stay
    x = st["logits"].double()
    r, v = x.shape
    temp = st["temperature"].double()[:, None]
    greedy = temp == 0
    y = (x - x.amax(1, keepdim=True)) / torch.where(greedy, torch.ones_like(temp), temp)
    w = torch.exp(y)
    z = w.sum(1, keepdim=True)
    _, order = torch.sort(st["logits"].float(), dim=1, descending=True, stable=True)
    by_rank = w.gather(1, order)
    before = torch.cumsum(by_rank, 1) - by_rank
    rank = torch.arange(v, device=x.device)
    stays = ~greedy | (rank == 0)
    if "top_k" in st:
        k = st["top_k"][:, None]
        stays = stays & ((rank < k) | (k <= 0))
    if "top_p" in st:
        stays = stays & ((before < st["top_p"].double()[:, None] * z) | (rank == 0))
    if "min_p" in st:
        stays = stays & (by_rank >= st["min_p"].double()[:, None])
    keep = torch.zeros_like(stays).scatter_(1, order, stays)
    race = torch.where(keep, w / st["noise"].double().clamp(min=2.0 ** -126), torch.full_like(w, -1.0))
    ids = torch.where(race == race.amax(1, keepdim=True), rank, v).amin(1, keepdim=True)
    return {"ids": ids[:, 0].to(torch.int32), "logprobs": (y.gather(1, ids) - torch.log(z))[:, 0].float()}


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    if op == "tables":
        return _plain_grow(state) if state["case"]["kind"] == "grow" else _plain_release(state)
    if op == "append":
        return _plain_append(state)
    if op == "decode":
        return _plain_decode(state)
    return _plain_sample(state)


# ---------------------------------------------------- the package's own calls --

def _own(op, st):
    import paged_kv_gqa_append_gb300 as pkv
    case = st["case"]
    if op == "tables":
        if case["kind"] == "release":
            pkv.release_pages(st["lens"], st["done"], st["tables"], st["free"], st["count"], seq_lens_out=st["lens_out"],
                              free_count_out=st["count_out"], d_err=st["err"])
            return {"free": st["free"], "count": st["count_out"], "lens": st["lens_out"]}
        pkv.grow_block_tables(st["lens"], st["new"], st["tables"], st["free"], st["count"], seq_lens_out=st["lens_out"],
                              free_count_out=st["count_out"], cu_new=st["cu"], positions=st["positions"],
                              token_seq=st["token_seq"], slots=st["slots"], d_err=st["err"])
        return {"tables": st["tables"], "lens": st["lens_out"], "count": st["count_out"], "cu": st["cu"],
                "positions": st["positions"], "token_seq": st["token_seq"], "slots": st["slots"]}
    if op == "append":
        turn = dict(rope_cos=st["cos"], rope_sin=st["sin"], q_in=st["q"], q_out=st["q_out"]) if case["rope"] else {}
        pkv.kv_append_rope_int4(st["k"], st["v"], st["cu"], st["lens"], st["tables"], st["pool"], d_err=st["err"], **turn)
        pkv.kv_read_int4(st["pool"], st["pages"], st["read"], d_err=st["err"])
        return {"q": st["q_out"], "read": st["read"]} if case["rope"] else {"read": st["read"]}
    if op == "decode":
        if "workspace" not in st:
            st["workspace"] = pkv.alloc_int4_workspace(case["seqs"], st["q"].device)
        pkv.paged_gqa_decode_int4(st["q"], st["pool"], st["tables"], st["lens"], st["out"], 0.125,
                                  workspace=st["workspace"], max_seq_len=st["longest"], d_err=st["err"])
        return st["out"]
    pkv.sample_logits(st["logits"], st["noise"], temperature=st["temperature"], top_k=st.get("top_k"),
                      top_p=st.get("top_p"), min_p=st.get("min_p"), ids=st["ids"], logprobs=st["logprobs"])
    return {"ids": st["ids"], "logprobs": st["logprobs"]}


# ------------------------------------------------------------ in 64 bits --

def _exact_turn(x, cos, sin):
    """Heads rotated, as complex products."""
    x = x.double()
    z = torch.complex(x[..., :32].contiguous(), x[..., 32:].contiguous()) * torch.complex(cos.double(), sin.double())[:, None]
    return torch.cat((z.real, z.imag), -1)


def _exact_rows(raw):
    """Values of blocks [n, heads, 1152], nibble by nibble: [n, 2, heads, 16, 64]."""
    word = raw.contiguous().view(torch.int32).to(torch.int64) & 0xFFFFFFFF  # [n, heads, 288]
    out = torch.zeros((raw.shape[0], 2, HKV, PAGE, D), dtype=torch.float64, device=raw.device)
    for slot in range(PAGE):
        g, upper = slot % 8, slot // 8
        for kv in range(2):
            both = word[:, :, 256 + 4 * g + 2 * kv + upper]
            scale, low = (((h << 16).to(torch.int32)).view(torch.float32).double() for h in (both & 0xFFFF, both >> 16))
            for d in range(D):
                if kv == 0:    # words of eight dims of one token
                    got = word[:, :, (4 * g + d // 16) * 4 + 2 * upper + d % 16 // 8] >> 4 * (d % 8)
                else:          # words of four dims of two tokens
                    got = word[:, :, 128 + (4 * (d // 8) + g // 2) * 4 + 2 * upper + d % 8 // 4] >> 16 * (g % 2) + 4 * (d % 4)
                out[:, kv, :, slot, d] = low + (got & 15).double() * scale
    return out


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    st = prepare(case, seed)
    dev = _dev()
    if case["op"] == "append":
        new, held = _append_lens(case)
        got, bf = {}, torch.bfloat16
        k = st["k"].double()
        pos = torch.cat([torch.arange(h, h + n) for n, h in zip(new, held)]).to(dev)
        if case["rope"]:
            got["q"] = _exact_turn(st["q"], st["cos"][pos], st["sin"][pos])
            k = _exact_turn(st["k"], st["cos"][pos], st["sin"][pos]).to(bf).double()
        x = torch.stack((k, st["v"].double()), 1)
        low, high = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
        # the definition's scales and quotients are 32-bit ones: a tie between two codes is decided by them
        scale = ((high - low) / 15).float().to(bf).double()
        inv = torch.where(scale > 0, 1 / scale, 0.0).float().double()
        code = torch.round(((x - low).float().double() * inv).float().double()).clamp(0, 15)
        pages = st["pages"].long()
        value = _exact_rows(st["pool"][pages])
        where = torch.full((st["pool"].shape[0],), -1, dtype=torch.long, device=dev)
        where[pages] = torch.arange(len(pages), device=dev)
        seq = torch.cat([torch.full((n,), i) for i, n in enumerate(new)]).to(dev)
        value[where[st["tables"][seq, pos // PAGE].long()], :, :, pos % PAGE] = low + code * scale
        got["read"] = value
        return got
    if case["op"] == "decode":
        out = torch.zeros((case["seqs"], HQ, D), dtype=torch.float64, device=dev)
        for s, n in enumerate(st["lens"].tolist()):
            if n == 0:
                continue
            kv = _exact_rows(st["pool"][st["tables"][s, :_blocks(n)].long()]).permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :n]
            q = st["q"][s].double().unflatten(0, (HKV, HQ // HKV))
            w = torch.softmax(torch.einsum("hgd,hnd->hgn", q, kv[0]) / 8, -1)
            out[s] = torch.einsum("hgn,hnd->hgd", w, kv[1]).flatten(0, 1)
        return out
    logprobs = []
    for i in range(case["rows"]):
        x, temp = st["logits"][i].double(), float(st["temperature"][i])
        if temp == 0:
            logprobs.append(torch.log_softmax(x, 0).amax())
            continue
        lp = torch.log_softmax(x / temp, 0)
        down, order = torch.sort(lp, descending=True, stable=True)
        last = case["vocab"]
        if "top_k" in st:
            last = min(last, int(st["top_k"][i]))
        if "top_p" in st:
            mass = torch.cumsum(down.exp(), 0)
            last = min(last, 1 + int((mass < float(st["top_p"][i])).sum()))
        kept = order[:last]
        if "min_p" in st:
            kept = kept[lp[kept] - down[0] >= math.log(max(float(st["min_p"][i]), 1e-300))]
        best = torch.argmax(lp[kept] - torch.log(st["noise"][i].double()[kept]))
        logprobs.append(lp[kept[best]])
    return {"ids": None, "logprobs": torch.stack(logprobs)}
