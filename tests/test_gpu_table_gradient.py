"""The table's gradient at every end of a row inside a 16-byte word, and for runs of one
token over many units, with whole numbers: sums are exact in any order."""

import numpy as np
import pytest

from gpu_util import say
from test_gpu_params import _dtype, _tokens, thd, torch  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def _check(torch, thd, rows, vocab, width, dtype, out, kind, seed, accumulate=False, lead=0):
    rng = np.random.default_rng([seed, rows, vocab, width])
    # up to 2 and few non-zeros, so that 16-bit results hold the sums: 11 or 8 bits; the tensor ends with its last row
    x = rng.integers(-2, 3, (rows, width + lead)) * (rng.random((rows, width + lead)) < 0.02)
    ids, mask = _tokens(rng, rows, vocab, kind), (rng.random(rows) < 0.9).astype(np.uint8)
    drows = torch.from_numpy(x.astype(np.float32)).to(_dtype(torch, dtype)).cuda()[:, lead:]
    old = rng.integers(-3, 4, (vocab, width))
    to = torch.from_numpy(old.astype(np.float32)).to(_dtype(torch, out)).cuda()
    got, status = thd.embedding_backward(drows, torch.from_numpy(ids).cuda(), vocab, mask=torch.from_numpy(mask).cuda(),
                                         out=to, accumulate=accumulate)
    want = np.zeros((vocab, width))
    np.add.at(want, ids[mask != 0], x[mask != 0][:, lead:])
    want += old if accumulate else 0
    assert int(status) == 0 and (out == "fp32" or np.abs(want).max(initial=0) <= 256)
    assert np.array_equal(got.double().cpu().numpy(), want), (rows, vocab, width, dtype, out, kind)


@pytest.mark.parametrize("width", [*range(1, 18), 23, 31, 33, 63, 65])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
def test_every_end_of_a_row(torch, thd, width, dtype, out):
    say("table gradient row ends", width, dtype, out)
    for rows, lead in ((1, 0), (50, 0), (300, 3), (9000, 1)):
        for accumulate in (False, True):
            _check(torch, thd, rows, 211, width, dtype, out, "text", 20, accumulate, lead)


@pytest.mark.parametrize("rows", [16, 17, 129, 1000, 8192, 8193, 20000, 40000, 70000, 140000])
@pytest.mark.parametrize("width", [3, 20, 64])
def test_runs_over_many_units(torch, thd, rows, width):
    say("table gradient runs", rows, width)
    for kind, vocab in (("one", 5), ("text", 7), ("all", 3), ("text", 3000)):
        _check(torch, thd, rows, vocab, width, "fp32", "fp32", kind, 21)


# tables of more than 256 MB without gaps, at places within a line; and the same with gaps
@pytest.mark.parametrize("vocab,width,dtype", [(140_000_001, 1, "bf16"), (30_000_001, 5, "fp16"), (4_500_000, 17, "fp32"),
                                               (70_003, 1001, "fp32"), (9_001, 16411, "bf16"), (70, 1_000_003, "fp32")])
@pytest.mark.parametrize("rows", [37, 3001, 20001])
def test_large_tables(torch, thd, vocab, width, dtype, rows):
    dt, rng = _dtype(torch, dtype), np.random.default_rng([22, vocab, rows])
    rows = min(rows, (1 << 26) // width + 1)
    ids = np.concatenate([rng.integers(0, vocab, rows), [0, vocab - 1, 1, vocab // 2, vocab // 2 + 1]])
    drows = torch.from_numpy(rng.integers(-2, 3, (len(ids), 1)).astype(np.float32)).to(dt).cuda().expand(-1, width).contiguous()
    ids = torch.from_numpy(ids).cuda()
    used = torch.unique(ids)
    sums = torch.zeros((vocab, 1), device="cuda").index_add_(0, ids, drows[:, :1].float())
    for lead, gap in ((0, 0), (1, 0), (37, 0), (3, 5)):
        if gap and width * vocab > 1 << 28:
            continue
        say("table gradient large table", vocab, width, dtype, rows, lead, gap)
        room = torch.full((lead + vocab * (width + gap) + 64,), 9.0, device="cuda", dtype=dt)
        to = room[lead:].as_strided((vocab, width), (width + gap, 1), room.storage_offset() + lead)
        _, status = thd.embedding_backward(drows, ids, vocab, out=to)
        assert int(status) == 0
        assert bool((room[:lead] == 9).all()) and bool((room[lead + vocab * (width + gap):] == 9).all())
        assert torch.equal(to[used].float(), sums[used].expand(-1, width))
        assert int(torch.count_nonzero(to)) == int(torch.count_nonzero(sums)) * width
        if gap:
            assert bool((room[lead:lead + vocab * (width + gap)].view(vocab, -1)[:, width:] == 9).all())
        del room, to
