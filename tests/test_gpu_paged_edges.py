"""Calls around pages and attention that a user may make and that the ordinary cases leave out."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from kv_cache_token_bf16_gb300 import paged  # noqa: E402
from tests.paged_util import D, gather  # noqa: E402
from tests.test_gpu_attend import _built, attend, check, make, randn  # noqa: E402,F401


def test_a_table_shared_by_all_sequences_has_to_be_repeated():
    kp, vp = randn(40, 6, 2, 16, D), randn(41, 6, 2, 16, D)
    row, lens = torch.tensor([[3, 1]], dtype=torch.int32).cuda(), torch.tensor([20, 31, 5], dtype=torch.int32).cuda()
    for bad in (dict(table=row.expand(3, 2)),
                dict(table=row.repeat(3, 1), k_pages=kp[:1].expand_as(kp), v_pages=vp[:1].expand_as(vp))):
        with pytest.raises(ValueError, match="table|pages"):
            paged.PagedCache(**dict(dict(k_pages=kp, v_pages=vp, lens=lens), **bad))
    # repeated, the sequences read the same pages; a single sequence's row may come with any stride
    s = {"q": randn(42, 3, 4, 1, D), "prefix": None, "new": None}
    table = row.repeat(3, 1)
    s["own"] = list(zip(gather(kp, table, lens.tolist()), gather(vp, table, lens.tolist())))
    s["cache"] = paged.PagedCache(k_pages=kp, v_pages=vp, table=table, lens=lens)
    check(s, *attend(s))
    for b in range(3):
        one = dict(s, q=s["q"][b:b + 1], own=s["own"][b:b + 1])
        one["cache"] = paged.PagedCache(k_pages=kp, v_pages=vp, table=row.as_strided((1, 2), (0, 1)), lens=lens[b:b + 1])
        check(one, *attend(one))
