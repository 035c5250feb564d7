"""Pools that run out, and tables that name pages which are not theirs any more: what the page calls
leave and say then does not depend on the order in which the GPU's threads run."""
import pytest
import torch

pytestmark = pytest.mark.gpu

sd = pytest.importorskip("speculative_decoding_verification_logits_gb300")

I32 = torch.int32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _sharing(rows, full, M, page, free):
    """Rows of `full` pages of their own and, in pairs, a shared and partly filled last one; a pool
    with `free` pages left: (table, kv_len, refs)."""
    ids = torch.arange(rows * full + rows, dtype=I32)
    t = torch.full((rows, M), -1, dtype=I32)
    t[:, :full] = ids[:rows * full].view(rows, full)
    t[:, full] = ids[rows * full:][torch.arange(rows) // 2]
    refs = torch.bincount(t[t >= 0].long(), minlength=len(ids)).to(I32)
    refs = torch.cat([refs[refs > 0], torch.zeros(free, dtype=I32)])
    return t, torch.full((rows,), full * page + 1, dtype=I32), refs


@pytest.mark.parametrize("rows,full", [(2, 0), (6, 3), (6, 600), (300, 5), (60, 700)])
@pytest.mark.parametrize("free", [0, 1, 3])
def test_extend_without_pages_says_so_alone(dev, rows, full, free):
    # the copies of shared last pages find no page: the tables are sound, so the status says no more
    M, page = full + 2, 4
    t, n, refs = _sharing(rows, full, M, page, free)
    for _ in range(10):
        td, rd, st = t.to(dev), refs.to(dev), torch.zeros(1, dtype=I32, device=dev)
        m = sd.kv_extend(td, n.to(dev), rd, page, 1, status=st)
        assert int(st) == (sd.SD_STATUS_NO_PAGE if free < rows else 0)
        assert torch.equal(td[:, :full].cpu(), t[:, :full])
        assert int(m.count) == rows and int((m.src >= 0).sum()) == min(free, rows)
        got = td[:min(free, rows), full].cpu()
        assert got.tolist() == list(range(len(refs) - free, len(refs)))[:rows]
