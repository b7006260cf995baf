"""Rules of the cache's pages by worked examples, apart from the list model: what the header says of each case."""
import pytest

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
