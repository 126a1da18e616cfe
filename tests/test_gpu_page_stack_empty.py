"""grow_block_tables with outputs for no token at all: they count as given, so that new
tokens are more than there is room for, and nothing is taken."""
import numpy as np
import pytest
import torch

from tests._util import to_dev_i32
from tests.test_gpu_page_stack import equal, lib, start  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("own_stream", [False, True])
@pytest.mark.parametrize("rows", [3, 3000])
@pytest.mark.parametrize("given", [["positions"], ["token_seq"], ["slots"], ["positions", "token_seq", "slots"]])
def test_outputs_without_room(lib, cuda_device, given, rows, own_stream):  # noqa: F811
    dev, lens = cuda_device, np.full(rows, 20)
    tables, stack, count = start(5, 2, lens, 3, 2 * rows)
    empty = dict(positions=(0,), token_seq=(0,), slots=(2, 0))
    kw = {k: torch.empty(empty[k], dtype=torch.int32, device=dev) for k in given}
    if own_stream:  # the other way that a call is marshalled
        kw["stream"] = torch.cuda.current_stream(dev)
    for new, code in ((np.full(rows, 13), lib.ERR_DEVICE_INDEX), (np.zeros(rows, int), 0)):
        d_lens, d_count, d_tables = to_dev_i32(lens, dev), to_dev_i32([count], dev), to_dev_i32(tables, dev)
        d_stack, err = to_dev_i32(stack, dev), torch.zeros(1, dtype=torch.int32, device=dev)
        cu = lib.grow_block_tables(d_lens, to_dev_i32(new, dev), d_tables, d_stack, d_count, d_err=err, **kw)
        equal(err, [code])
        equal(cu, np.zeros(rows + 1))
        equal(d_lens, lens)
        equal(d_count, [count])
        equal(d_tables, tables)
        equal(d_stack, stack)
