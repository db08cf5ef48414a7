"""GPU: the read reports output ranges that are out of range or out of order, and
does not follow what is out of range."""
import pytest
import torch

import transform_codec_b200 as kvc
from serving_ref import HostCache
from test_gpu_attend import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out_start,kept", [
    ((-3, 5), slice(0, 10)),             # a negative start: its sequence is not read
    ((-3, 5, 8), slice(0, 5)),
    ((0, 1000000, 5), slice(10, 10)),    # far past the end, then back
    ((0, 4, 2, 6), slice(6, 10)),        # descending
    ((0, 2, 11), slice(10, 10)),
    ((4, -1, 6), slice(6, 10)),
    ((12, 14), slice(0, 10)),            # all of it past the end
])
def test_read_reports_bad_out_starts(out_start, kept):
    n = len(out_start) - 1
    host = HostCache(kvc.CACHE_E4M3, 2, 64, 16, [60] * n, seed=1)
    c = host.gpu()
    out = torch.full((2, 2, 10, 64), 9.0, device="cuda")
    kvc.cache_read(c, host.table.cuda(), i32([0] * n), i32(out_start), out)
    assert kvc.read_result(c.res)[0] == kvc.ERR_INVALID
    assert (out[:, :, kept] == 9.0).all()


@pytest.mark.parametrize("seqs", [1, 300, 70000])
def test_read_reports_one_bad_out_start_among_many(seqs):
    """Good ranges set nothing; one pair out of order, wherever it stands, does."""
    c = kvc.QuantCache(kvc.CACHE_INT8, 1, 32, 16, 1)
    table = torch.zeros(seqs, 1, dtype=torch.int32, device="cuda")
    start = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    out = torch.zeros(2, 1, 8, 32, device="cuda")
    at = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
    at[seqs // 2 + 1:] = 7
    kvc.cache_read(c, table, start, at, out)
    assert kvc.read_result(c.res)[0] == kvc.OK
    for where in {0, seqs // 2, seqs}:
        for bad in (-1, 9):
            wrong = at.clone()
            wrong[where] = bad
            c.res.zero_()
            kvc.cache_read(c, table, start, wrong, out)
            assert kvc.read_result(c.res)[0] == kvc.ERR_INVALID, (where, bad)
