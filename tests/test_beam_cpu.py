"""Refusals of beam search's step and of the page operators, at the C ABI and in the binding, and
their definitions against hand-worked values (no GPU: every call is refused before any launch)."""
import ctypes
import math

import pytest
import torch

import speculative_decoding_verification_logits_gb300 as sd
from speculative_decoding_verification_logits_gb300.beam import SelectArgs, StateArgs
from speculative_decoding_verification_logits_gb300.kv import CopyArgs, ForkArgs
from tests import beam_ref as ref

BAD, OK = sd.SD_ERR_INVALID_ARG, sd.SD_OK
FAKE = 1 << 20   # a non-null address that is never dereferenced: the checks fail first
i32 = lambda v: torch.tensor(v, dtype=torch.int32)


def test_struct_layouts():
    L = sd.lib()
    for fn, mirror in ((L.sd_beam_select_args_size, SelectArgs), (L.sd_beam_state_size, StateArgs),
                       (L.sd_kv_fork_args_size, ForkArgs), (L.sd_kv_copy_args_size, CopyArgs)):
        assert fn() == ctypes.sizeof(mirror)


def test_select_refuses_bad_requests():
    L = sd.lib()
    size = L.sd_beam_select_workspace_size(2, 3, 100, sd.SD_F32)
    assert size > 0
    ok = dict(B=2, W=3, V=100, k=4, dtype=sd.SD_F32, logits=FAKE, logits_sb=300, logits_sw=100,
              scores=FAKE, eos=-1, T=1.0, out_scores=FAKE, parents=FAKE, tokens=FAKE,
              workspace=FAKE, workspace_bytes=size)
    assert L.sd_beam_select(None, None) == BAD
    for bad in (dict(B=-1), dict(W=0), dict(W=sd.SD_MAX_BEAMS + 1), dict(V=0),
                dict(V=sd.SD_MAX_V + 1), dict(k=0), dict(k=sd.SD_MAX_TOP + 1), dict(dtype=2),
                dict(T=0.0), dict(T=-1.0), dict(T=math.inf), dict(T=math.nan), dict(T=1e-39), dict(eos=-2),
                dict(eos=100), dict(finished=FAKE), dict(logits=None), dict(scores=None),
                dict(out_scores=None), dict(parents=None), dict(tokens=None),
                dict(workspace=None), dict(workspace=FAKE + 8), dict(workspace_bytes=size - 1),
                dict(logits=FAKE + 2)):
        assert L.sd_beam_select(SelectArgs(**{**ok, **bad}), None) == BAD, bad
    assert L.sd_beam_select(SelectArgs(**{**ok, "B": 0, "logits": None}), None) == OK
    for bad in ((-1, 3, 100, 0), (2, 0, 100, 0), (2, 33, 100, 0), (2, 3, 0, 0), (2, 3, 100, 7)):
        assert L.sd_beam_select_workspace_size(*bad) == 0


def test_reorder_refuses_bad_requests():
    L = sd.lib()

    def call(B=2, W=3, k=3, parents=FAKE, n=1, states=True, **more):
        s = dict(in_=FAKE, in_sb=300, in_sw=100, out=2 * FAKE, out_sb=300, out_sw=100,
                 row_bytes=100)
        a = (StateArgs * 1)(StateArgs(**{**s, **more}))
        return L.sd_beam_reorder(B, W, k, parents, n, ctypes.addressof(a) if states else None,
                                 None, None)

    for bad in (dict(B=-1), dict(W=0), dict(W=sd.SD_MAX_BEAMS + 1), dict(k=-1),
                dict(k=sd.SD_MAX_TOP + 1), dict(n=-1), dict(n=sd.SD_MAX_STATES + 1),
                dict(states=False), dict(parents=None), dict(in_=None), dict(out=None),
                dict(row_bytes=-1), dict(out=FAKE, k=2), dict(out=FAKE, out_sw=101),
                dict(out=FAKE, out_sb=301)):
        assert call(**bad) == BAD, bad
    assert call(B=0, in_=None) == OK and call(k=0, in_=None) == OK
    assert call(row_bytes=0, in_=None) == OK and call(n=0, states=False) == OK


def test_fork_refuses_bad_requests():
    L = sd.lib()
    size = L.sd_kv_fork_workspace_size(4, 6, 50)
    ok = dict(rows_in=4, R=6, groups=2, max_pages=5, page_size=16, append=1, keep=0, N=50,
              parents=FAKE, table=FAKE, kv_len=FAKE, refs=FAKE, table_out=2 * FAKE,
              len_out=FAKE, src=FAKE, dst=FAKE, fill=FAKE, count=FAKE, workspace=FAKE,
              workspace_bytes=size)
    assert L.sd_kv_fork(None, None) == BAD
    for bad in (dict(rows_in=-1), dict(rows_in=sd.SD_MAX_ROWS + 1), dict(R=-1),
                dict(R=sd.SD_MAX_ROWS + 1), dict(groups=-1), dict(groups=3), dict(max_pages=-1),
                dict(page_size=0), dict(append=-1), dict(keep=2), dict(N=0),
                dict(N=sd.SD_MAX_PAGES + 1), dict(table=None), dict(kv_len=None), dict(refs=None),
                dict(table_out=None), dict(len_out=None), dict(src=None), dict(dst=None),
                dict(fill=None), dict(count=None), dict(workspace=None),
                dict(workspace=FAKE + 4), dict(workspace_bytes=size - 1),
                dict(max_pages=2 ** 20, page_size=2 ** 12),
                dict(max_pages=2 ** 29, page_size=1), dict(parents=None),
                dict(parents=None, R=4, table_out=FAKE, len_out=FAKE),
                dict(parents=None, R=4, table_out=2 * FAKE, len_out=None),
                dict(parents=None, R=4, table_out=FAKE, len_out=None, keep=1)):
        assert L.sd_kv_fork(ForkArgs(**{**ok, **bad}), None) == BAD, bad
    for bad in ((-1, 1, 5), (1, -1, 5), (1, 1, 0), (sd.SD_MAX_ROWS + 1, 1, 5)):
        assert L.sd_kv_fork_workspace_size(*bad) == 0


def test_free_compact_and_copy_refuse_bad_requests():
    L = sd.lib()
    free = lambda rows=2, cols=3, p=FAKE, N=9, r=FAKE: L.sd_kv_free(rows, cols, p, None, None, 0, N,
                                                                   r, None, None)
    for bad in (dict(rows=-1), dict(cols=-1), dict(rows=2 ** 31), dict(N=0),
                dict(N=sd.SD_MAX_PAGES + 1), dict(p=None), dict(r=None),
                dict(rows=2 ** 31 - 1, cols=2 ** 31 - 1)):
        assert free(**bad) == BAD, bad
    assert free(rows=0, p=None) == OK and free(cols=0, p=None) == OK

    size = L.sd_kv_compact_workspace_size(50)
    ok = dict(N=50, refs=FAKE, nt=4, t=FAKE, src=FAKE, dst=FAKE, c=FAKE, live=FAKE, new=FAKE,
              st=None, ws=FAKE, size=size)
    for bad in (dict(N=0), dict(N=sd.SD_MAX_PAGES + 1), dict(refs=None), dict(nt=-1), dict(t=None),
                dict(src=None), dict(dst=None), dict(c=None), dict(live=None), dict(new=None),
                dict(ws=None), dict(ws=FAKE + 8), dict(size=size - 1)):
        assert L.sd_kv_compact(*{**ok, **bad}.values(), None) == BAD, bad
    assert L.sd_kv_compact_workspace_size(0) == 0

    ptr = (ctypes.c_void_p * 2)(FAKE, 2 * FAKE)
    none = (ctypes.c_void_p * 2)(FAKE, None)
    cast = lambda a: ctypes.cast(a, ctypes.c_void_p)
    ok = dict(n_caches=2, layers=1, N=9, parts=1, page_size=16, entry_bytes=64, layer_stride=0,
              page_stride=1024, caches=cast(ptr), pairs=3, src=FAKE, dst=FAKE)
    assert L.sd_kv_copy(None, None) == BAD
    for bad in (dict(n_caches=-1), dict(n_caches=sd.SD_MAX_CACHES + 1), dict(layers=-1), dict(N=0),
                dict(N=sd.SD_MAX_PAGES + 1), dict(parts=0), dict(page_size=0),
                dict(entry_bytes=-1), dict(entry_bytes=2 ** 62), dict(pairs=-1), dict(caches=None),
                dict(caches=cast(none)), dict(src=None), dict(dst=None)):
        assert L.sd_kv_copy(CopyArgs(**{**ok, **bad}), None) == BAD, bad
    for empty in (dict(n_caches=0), dict(layers=0), dict(entry_bytes=0), dict(pairs=0)):
        assert L.sd_kv_copy(CopyArgs(**{**ok, **empty, "caches": None}), None) == OK


def test_binding_refuses_host_tensors():
    x, s = torch.zeros(2, 3, 40), torch.zeros(2, 3)
    t, n, r = i32([[0, 1], [2, -1]]), i32([20, 3]), torch.ones(5, dtype=torch.int32)
    for call in (lambda: sd.beam_select(x, s, 3), lambda: sd.beam_reorder(x, i32([[0, 1, 2]] * 2)),
                 lambda: sd.beam_reorder([x, x], i32([[0, 1, 2]] * 2)),
                 lambda: sd.kv_fork(t, n, i32([0, 0]), r, 16), lambda: sd.kv_extend(t, n, r, 16, 1),
                 lambda: sd.kv_free(t, r), lambda: sd.kv_compact(r, t),
                 lambda: sd.kv_copy(torch.zeros(2, 5, 16, 4), i32([0]), i32([1]))):
        with pytest.raises(ValueError):
            call()


def test_which_memory_rows_share():
    from speculative_decoding_verification_logits_gb300.kv import _rows_meet as meet
    buf = torch.zeros((3, 4, 20), dtype=torch.uint8)
    assert not meet(buf[..., :10], buf[..., 10:], 2) and meet(buf[..., :11], buf[..., 10:], 2)
    assert not meet(buf[:, ::2], buf[:, 1::2], 2) and meet(buf[:, ::2], buf[:, 2:], 2)
    assert meet(buf, buf, 2) and not meet(buf[:0], buf, 2)
    assert not meet(buf[:, :3, :5], buf[:, 3:, :9], 2)
    wide = buf.view(torch.int32)          # rows of different types and lengths
    assert meet(wide[:, :2, 4:], buf[:, 1:, 16:18], 2) and not meet(wide[:, :, 4:], buf[..., :16], 2)
    flat = torch.zeros(100, dtype=torch.int32)
    assert not meet(flat[:6].view(1, 2, 3), flat[6:9].view(1, 1, 3), 2)
    assert meet(flat[:6].view(1, 2, 3), flat[5:9].view(1, 2, 2), 2)


# ------------------------------------------------------- the definitions --
def test_reference_select_by_hand():
    x = torch.log(torch.tensor([[[0.5, 0.25, 0.25, 0.0], [0.1, 0.2, 0.3, 0.4]]], dtype=torch.float64))
    s = torch.log(torch.tensor([[0.25, 0.5]], dtype=torch.float64))
    found, _, status = ref.select(x, s, 3, eos=3)
    got = [(round(math.exp(r), 9), w, v, e) for r, w, v, _, e in found[0][:3]]
    assert got == [(0.2, 1, 3, 1), (0.15, 1, 2, 0), (0.125, 0, 0, 0)] and status == 0
    # ties in the order of beams, then tokens; a token of probability zero is never offered
    found, _, _ = ref.select(x[:, :1].repeat(1, 2, 1), s * 0, 8)
    assert [(w, v) for _, w, v, _, _ in found[0]] == [(0, 0), (1, 0), (0, 1), (0, 2), (1, 1), (1, 2)]
    # a finished beam offers itself; ranks go by the score over norm
    found, _, _ = ref.select(x, s, 2, finished=torch.tensor([[1, 0]]), eos=2,
                             norm=torch.tensor([[4.0, 1.0]]))
    assert found[0][0][1:3] == (0, 2) and abs(found[0][0][0] - math.log(0.25) / 4) < 1e-12
    assert abs(found[0][0][3] - math.log(0.25)) < 1e-12 and found[0][0][4] == 1


def test_reference_fork_by_hand():
    # two rows of page size 4: 6 and 8 entries, a shared first page
    t = i32([[3, 5, -1], [3, 1, -1]])
    refs = i32([0, 1, 0, 2, 0, 1, 0])
    out, n, src, dst, fill, count, r, status = ref.fork(t, i32([6, 8]), i32([0, 0, 1]), refs, 4,
                                                        append=1)
    # row 0 inherits page 5, row 1 copies it into page 0, row 2 needs a page for one more entry
    assert out.tolist() == [[3, 5, -1], [3, 0, -1], [3, 1, 2]] and n.tolist() == [6, 6, 8]
    assert (src.tolist(), dst.tolist(), fill.tolist()) == ([5, -1, -1], [0, -1, -1], [2, 0, 0])
    assert count.tolist() == [1] and r.tolist() == [1, 1, 1, 3, 0, 1, 0] and status == 0
    # both rows go on from row 1: row 0's own page comes free
    out, n, _, _, _, count, r, status = ref.fork(t, i32([6, 8]), i32([1, 1]), refs, 4)
    assert out.tolist() == [[3, 1, -1]] * 2 and r.tolist() == [0, 2, 0, 2, 0, 0, 0] and status == 0
    # the old rows stay: every new one copies
    out, n, src, dst, fill, count, r, status = ref.fork(t, i32([6, 8]), i32([0]), refs, 4, keep=True)
    assert out.tolist() == [[3, 0, -1]] and (int(src[0]), int(dst[0])) == (5, 0)
    assert r.tolist() == [1, 1, 0, 3, 0, 1, 0]
    # no page left
    out, *_, status = ref.fork(t, i32([6, 8]), i32([0, 0]), i32([1, 1, 1, 2, 1, 1, 1]), 4)
    assert out.tolist() == [[3, 5, -1], [3, -1, -1]] and status == ref.NO_PAGE
    # in place: room for three more, and a shared last page becomes a row's own
    t = i32([[2, 3, -1], [2, 3, -1]])
    out, n, src, dst, fill, count, r, status = ref.fork(t, i32([5, 5]), None, i32([0, 0, 2, 2, 0, 0]),
                                                        4, append=4)
    assert out.tolist() == [[2, 0, 1], [2, 4, 5]] and r.tolist() == [1, 1, 2, 0, 1, 1]
    assert (src.tolist(), dst.tolist(), fill.tolist()) == ([3, 3], [0, 4], [1, 1])


def test_reference_free_compact_and_copy_by_hand():
    r, t, status = ref.free(i32([[1, -1], [1, 2]]), i32([0, 2, 1]), which=[1, 0], clear=True)
    assert r.tolist() == [0, 1, 1] and t.tolist() == [[-1, -1], [1, 2]] and status == 0
    r, _, status = ref.free(i32([0, 1, 9]), i32([0, 2, 1]), count=2)
    assert r.tolist() == [0, 1, 1] and status == ref.BAD_PAGE
    src, dst, count, new, live, r, t, status = ref.compact(i32([0, 2, 0, 0, 1, 3]), i32([[5, 1], [4, -1]]))
    assert (src.tolist(), dst.tolist()) == ([4, 5, -1], [0, 2, -1]) and int(count) == 2
    assert new.tolist() == [-1, 1, -1, -1, 0, 2] and int(live) == 3
    assert r.tolist() == [1, 2, 3, 0, 0, 0] and t.tolist() == [[2, 1], [0, -1]] and status == 0
    c = torch.arange(12).reshape(1, 3, 2, 2)
    y, _ = ref.copy(c, i32([2, -1]), i32([0, -1]), fill=i32([1, 2]))
    assert y[0, 0].tolist() == [[8, 9], [2, 3]] and torch.equal(y[:, 1:], c[:, 1:])
    y, _ = ref.copy(c, i32([2]), i32([0]), fill=i32([1]), heads_first=True)
    assert y[0, 0].tolist() == [[8, 1], [10, 3]]
