"""process_logits with lists that hold every token of the vocabulary, bit for bit
against the oracle (every operation of the definition is one rounded fp32
operation on both sides)."""
import numpy as np
import pytest
import torch

from oracle import logits as OL

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib(cuda_device):
    from paged_kv_gqa_append_gb300 import build
    build.build()
    import paged_kv_gqa_append_gb300 as m
    return m


def lists(seed, rows, vocab, hist):
    g = np.random.default_rng(seed)
    c = dict(x=(4 * g.standard_normal((rows, vocab))).astype(np.float32))
    c["bias_ids"] = np.stack([g.permutation(vocab) for _ in range(rows)]).astype(np.int32)
    c["bias_values"] = g.standard_normal((rows, vocab)).astype(np.float32)
    c["history"] = g.integers(0, vocab, (rows, hist)).astype(np.int32)
    c["history"][:, -hist // 4:] = c["bias_ids"][:, -1:]        # the last of the biases again and again
    c["history_lens"] = np.full(rows, hist, np.int32)
    c["prompt_lens"] = g.integers(0, hist, rows).astype(np.int32)
    c["repetition"] = g.uniform(0.8, 1.6, rows).astype(np.float32)
    c["presence"] = g.uniform(-1, 1, rows).astype(np.float32)
    c["frequency"] = g.uniform(-1, 1, rows).astype(np.float32)
    return c


@pytest.mark.parametrize("rows,vocab,hist,calls", [(3, 8192, 700, 40), (3, 8192, 60000, 10), (40, 8192, 700, 10),
                                                   (2, 1024, 90, 40), (2, 20011, 2048, 10), (2, 128256, 2048, 4)])
def test_every_token_listed(lib, cuda_device, rows, vocab, hist, calls):
    """Ranges of exactly 1024 tokens, all of which are in the table, from many lists."""
    c = lists(vocab + hist, rows, vocab, hist)
    want, want_ids = OL.process(c["x"], **{n: a for n, a in c.items() if n != "x"})
    d = {n: torch.from_numpy(a).to(cuda_device) for n, a in c.items()}
    x = d.pop("x")
    want = torch.from_numpy(want).to(cuda_device)
    for _ in range(calls):
        out = torch.full_like(x, 7.0)
        ids = lib.process_logits(x, out=out, **d)
        assert torch.equal(out, want)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
