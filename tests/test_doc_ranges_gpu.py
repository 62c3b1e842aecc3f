"""Document ranges of rows longer than a block's chunk by far (a block then takes several
chunks), against the definition."""
import numpy as np
import pytest
import torch

from exact_io_aware_64_b200 import binding

pytestmark = pytest.mark.gpu

CHUNK, ROW = 2048, 512 * 2048  # tokens of a chunk, of a row at one chunk a block


def expected(row):
    row = np.maximum(row, -1)
    edge = np.flatnonzero(np.concatenate([[True], row[1:] != row[:-1]]))
    n = np.diff(np.concatenate([edge, [row.size]]))
    j = np.arange(row.size)
    return (np.where(row < 0, j, np.repeat(edge, n)),
            np.where(row < 0, j, np.repeat(edge + n, n)))


def runs(N, mean, seed):
    rng = np.random.default_rng(seed)
    return np.cumsum(rng.random(N) < 1 / mean)


@pytest.mark.parametrize("N", [ROW - 1, ROW, ROW + 1, 2 * ROW + 5, 5 * ROW + 2047])
def test_long_rows(N):
    """One run, runs of every length, runs that begin and end at chunk and span bounds, and
    padding between them."""
    bounds = (np.arange(N) + 1) // (3 * CHUNK)
    mixed = runs(N, 9000, 2)
    mixed[runs(N, 3000, 3) % 5 == 0] = -1
    rows = [np.zeros(N), runs(N, 20, 1), mixed, bounds, np.arange(N) // CHUNK,
            np.where(np.arange(N) % (2 * CHUNK) < CHUNK, 7, -3)]
    ids = torch.from_numpy(np.stack(rows).astype(np.int32)).cuda()
    starts, ends = binding.doc_ranges(ids)
    binding.check_device_error()
    for row, s, e in zip(ids.cpu().numpy(), starts.cpu().numpy(), ends.cpu().numpy()):
        rs, re = expected(row)
        assert np.array_equal(s, rs) and np.array_equal(e, re)


def test_time_of_one_run_is_linear():
    """A run 16 times as long takes some 16 times as long (the square would be 256)."""
    def ms(N):
        ids = torch.zeros(1, N, dtype=torch.int32, device="cuda")
        out = binding.doc_ranges(ids)
        best = float("inf")
        for _ in range(3):
            a, b = torch.cuda.Event(True), torch.cuda.Event(True)
            a.record()
            binding.doc_ranges(ids, *out)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        assert (out[0] == 0).all() and (out[1] == N).all()
        return best

    short, long_ = ms(1 << 20), ms(1 << 24)
    assert long_ < 64 * short, (short, long_)
