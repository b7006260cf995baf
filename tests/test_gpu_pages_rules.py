"""Rules of the cache's pages by worked examples, apart from the list model: what the header says of each case."""
import random

import pytest
import torch

from test_gpu_pages import Device, ints
from gateddeltanet_linear_attention_gb300 import gdn

pytestmark = pytest.mark.gpu


def test_fork_lanes_that_name_one_another():
    """A lane whose source is another lane's destination is skipped, and that other is carried out; a destination named twice, or
    a row forked onto itself, is skipped; a refused lane's destination is no source either."""
    d = Device(10, 8, 4)
    d.resize([0, 7], [20, 5])
    rows = d.table.clone()

    def fork(src, dst):
        gdn.gdn_page_fork(d.cfg, d.table, d.lens, d.refs, ints(src), ints(dst))
        return gdn.gdn_device_error()
    assert fork([0, 2], [2, 3]) == gdn.DEVERR_SLOT
    rows[2] = rows[0]
    assert d.lens.tolist() == [20, 0, 20, 0, 0, 0, 0, 5] and d.table.equal(rows) and d.refs.tolist()[:3] == [2, 2, 1]
    assert fork([0, 7, 1], [4, 4, 1]) == gdn.DEVERR_SLOT
    assert fork([0, 7], [7, 5]) == gdn.DEVERR_SLOT                   # row 7 is not empty: neither lane
    assert d.lens.tolist() == [20, 0, 20, 0, 0, 0, 0, 5] and d.table.equal(rows) and d.refs.tolist()[:3] == [2, 2, 1]
    assert fork([0, -1, 5, 2], [5, 6, -1, 6]) == 0                   # inactive lanes name nothing
    rows[5] = rows[6] = rows[0]
    assert d.lens.tolist() == [20, 0, 20, 0, 0, 20, 20, 5] and d.table.equal(rows) and d.refs.tolist()[:3] == [4, 4, 1]


def test_copies_before_a_compaction():
    """A shared last page that all its holders leave is free before its copies are carried out: copies first, then the
    compaction, which closes it up."""
    d = Device(10, 4, 4)
    d.resize([3], [40])                                              # pages 0 to 2, which end: holes in front
    d.resize([0], [20])                                              # pages 3, 4
    d.fork([0], [1])
    d.resize([3], [0])
    pools = [torch.zeros(10, 1, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for f, pool in enumerate(pools):
        pool[3], pool[4] = 3 + 10 * f, 4 + 10 * f
    src, dst = d.resize([0, 1], [21, 22])
    assert src.tolist() == [4, 4] and dst.tolist() == [0, 1] and d.refs[4] == 0
    gdn.gdn_page_copy(d.cfg, *pools, *pools, src, dst)
    src, dst = d.compact(10, True)
    assert src.tolist()[:2] == [3, -1] and dst.tolist()[:2] == [2, -1]
    gdn.gdn_page_copy(d.cfg, *pools, *pools, src, dst)
    for row in (0, 1):
        first, last = d.table[row, :2].tolist()
        for f, pool in enumerate(pools):
            assert (pool[first] == 3 + 10 * f).all() and (pool[last] == 4 + 10 * f).all()
    assert gdn.gdn_device_error() == 0
    d.m.check()


def test_pool_that_runs_out_behind_the_first_thousand_lanes():
    """Places of lanes that a block's threads do not hold, granted and refused."""
    d = Device(60_000, 4000, 40, 16, lanes=4000)
    rng = random.Random(5)
    rows = list(range(4000))
    rng.shuffle(rows)
    new = [rng.randint(1, 640) for _ in rows]
    d.resize(rows, new)
    refused = [i for i, (r, v) in enumerate(zip(rows, new)) if d.m.lens[r] != v]
    assert 1100 < refused[0] < 3900 and refused == list(range(refused[0], 4000)) and all(d.m.lens[rows[i]] == 0 for i in refused)
    # Some end, others shrink: nothing is granted to who asks in the same call (pages are taken from those free when it starts), and
    # in the next one a part is.
    new = [0 if i % 5 == 0 else v if i >= refused[0] else rng.choice([v, v // 2]) for i, v in enumerate(new)]
    d.resize(rows, new)
    assert all(d.m.lens[rows[i]] == 0 for i in refused)
    d.resize(rows, new)
    assert 0 < sum(d.m.lens[rows[i]] == new[i] > 0 for i in refused)
    d.m.check()


def test_copies_behind_the_first_thousand_lanes():
    """Samples of one prompt that all grow in its last page: pages for 1,500 of 1,600 copies."""
    d = Device(1502, 1700, 4, 16, lanes=1600)
    d.resize([0], [20])
    rows = list(range(1, 1601))
    d.fork([0] * 1600, rows)
    src, dst = d.resize(rows, [21] * 1600)
    assert src.tolist() == [1] * 1500 + [-1] * 100 and dst.tolist() == list(range(2, 1502)) + [-1] * 100
    assert d.lens.tolist()[1:1601] == [21] * 1500 + [20] * 100
    d.m.check()
