"""Page calls refuse arguments that they write and that share memory with others (the counts above
all: they change while tables and lengths are read)."""
import pytest
import torch

import speculative_decoding_verification_logits_gb300 as sd
from speculative_decoding_verification_logits_gb300 import kv


def test_which_addresses_overlap():
    for at, n, other, size in ((100, 4, 96, 5), (100, 4, 115, 1), (100, 4, 104, 4), (100, 4, 0, 1000)):
        with pytest.raises(ValueError, match="refs overlaps"):
            kv._apart("refs", at, n, (None, 50), (other, size))
    for at, n, other, size in ((100, 4, 96, 4), (100, 4, 116, 1), (100, 4, 108, 0), (100, 0, 96, 8),
                               (None, 4, 0, 1000), (100, 4, None, 8)):
        kv._apart("refs", at, n, (other, size))


@pytest.mark.gpu
def test_refusals():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    buf = torch.zeros(200, dtype=torch.int32, device="cuda:0")
    t, n, p, r, st = buf[:12].view(4, 3), buf[12:16], buf[16:20], buf[20:60], buf[60:61]
    flags = buf[100:101].view(torch.uint8)
    pool = lambda x: torch.as_strided(buf, (40,), (1,), x)   # counts that begin at place x
    for call in (lambda r=r, st=st, n=n, p=p: sd.kv_fork(t, n, p, r, 4, append=1, status=st),
                 lambda r=r, st=st, n=n: sd.kv_extend(t, n, r, 4, 1, status=st),
                 lambda r=r, st=st, n=n: sd.kv_free(t, r, which=flags, count=n[:1], clear=True, status=st),
                 lambda r=r, st=st: sd.kv_compact(r, t, status=st)):
        names = call.__code__.co_varnames[:call.__code__.co_argcount]
        bad = [dict(r=pool(11)), dict(r=pool(60)), dict(st=r[3:4]),
               dict(st=t[1, 1:2])]
        if "n" in names:
            bad += [dict(r=pool(12)), dict(st=n[:1]), dict(n=r[:4])]
        if "p" in names:
            bad += [dict(r=pool(19)), dict(st=p[1:2]), dict(p=r[:4])]
        elif "n" in names:   # the table is written
            bad += [dict(n=t.view(-1)[2:6])]
        for change in bad:
            with pytest.raises(ValueError, match="overlaps"):
                call(**change)
        call()               # apart, though of one block
    with pytest.raises(ValueError, match="overlaps"):
        sd.kv_free(t, pool(80), which=flags)
    assert sd.kv_free(t, r, count=r.new_zeros(1)) is r
