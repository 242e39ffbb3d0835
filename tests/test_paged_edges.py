"""The paged-cache calls where a first version went wrong: indices outside their
tables, rows that a mask hides, weights far below the largest, queries that are
not finite, padding.  Helpers and tolerances: test_paged.py."""

import pytest
import torch

from rotated_int4_kv_kvq_b200 import workloads as W
from test_paged import gen, kvq, rows  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:invalid value:RuntimeWarning")]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,group", [(64, 64), (128, 32), (256, 128)])
def test_append_many_rows_far_positions(kvq, d, group, inter):
    """Positions far outside the table among many rows: those tokens are skipped
    whole and reported, the others come out as without them."""
    t, h, page = 2601, 4, 32
    signs = torch.from_numpy(W.make_signs(d)).cuda()
    x = rows(gen(6), t, h, d, torch.float16)
    slots = torch.arange(t, device="cuda")
    table = kvq.rope_table(3000, d // 2)
    pos = torch.arange(t, device="cuda", dtype=torch.int32)
    bad = [0, 31, 500, 1999, 2600]
    far = pos.clone()
    far[bad] = torch.tensor([2 ** 31 - 1, -2 ** 31, 3000, -1, 2 ** 30], device="cuda",
                            dtype=torch.int32)
    out = []
    for p, status in ((pos, 0), (far, 11)):
        cache = kvq.PagedCache.empty(t // page + 1, h, page, d, group, signs)
        for c in cache.tensors()[:4]:
            c.zero_()
        hat = torch.full_like(x, 9.0)
        kvq.kvq_paged_append(x, x, slots, cache, positions=p, cos_sin=table, interleaved=inter,
                             k_hat=hat)
        assert kvq.kvq_device_status() == status
        out.append([c.transpose(1, 2).flatten(0, 1)[:t] for c in cache.tensors()[:4]] + [hat])
    good = torch.ones(t, dtype=torch.bool, device="cuda")
    good[bad] = False
    for a, b in zip(*out):
        assert torch.equal(a[good], b[good])
    for b in out[1][:4]:
        assert (b[bad] == 0).all()
    assert (out[1][4][bad] == 9).all()
