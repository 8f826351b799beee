"""CPU-side refusals of the rotary and paged entry points, beside those of
test_paged_abi.py: nothing here touches a device."""
import pytest

import exact_tiled_attention_31_b200 as fa
from exact_tiled_attention_31_b200 import api, build

E, U, OK = api.FA_ERR_INVALID_ARG, api.FA_ERR_UNSUPPORTED, api.FA_OK
A = 1 << 20  # a 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build_library()
    return fa.load_library()


def rows(data=A, batch=0, head=1280, row=128, heads=2):
    return api._ROWS.pack(data, batch, head, row, heads)


def pages(k=A, v=A + (1 << 30), stride=2 * 64 * 128, table=A, row=10, n=100, page=64, heads=2, most=10):
    return api._PAGES.pack(k, v, stride, table, row, n, page, heads, most)


def test_fill_entries_refuse_what_the_plain_ones_refuse():
    for call in (fa.fa_rope, fa.fa_rope_fill):
        def status(x=rows(), y=rows(A + (1 << 20)), n=1, f=A, rot=64, amp=1.0, cu=None, nseq=0, B=1, S=10, D=128, dt=0):
            return call(x, y, n, f, rot, 0, amp, 0, None, 0, cu, nseq, B, S, D, dt, None)
        assert status(B=0) == OK and status(S=0, cu=A, nseq=0) == OK
        for bad in (dict(n=3), dict(amp=float("nan")), dict(S=-1), dict(dt=2), dict(cu=A, nseq=-1), dict(cu=A, nseq=1, B=2),
                    dict(f=None), dict(x=rows(0)), dict(y=rows(heads=3)), dict(cu=A + 2, nseq=1)):
            assert status(**bad) == E, (call, bad)
        assert status(rot=8) == U and status(D=96) == U and status(B=1 << 16, S=1 << 16) == U
    for call in (fa.fa_append_paged, fa.fa_append_paged_fill):
        def status(k=rows(), v=rows(), q=None, qo=None, pg=pages(), lens=A, cu=None, nseq=4, total=4, f=A, rot=64, D=128):
            return call(k, v, q, qo, pg, lens, cu, nseq, total, f, rot, 0, 1.0, None, D, 0, None)
        assert status(nseq=0, total=0) == OK and status(cu=A, total=0) == OK
        for bad in (dict(total=5), dict(lens=None), dict(k=rows(heads=3)), dict(q=rows(heads=8)),
                    dict(q=rows(heads=8), qo=rows(heads=8), f=None), dict(pg=pages(n=0))):
            assert status(**bad) == E, (call, bad)
        assert status(D=96) == U and status(rot=40) == U
    # with no sequences the queries' rows are still written: their rows have to be valid
    bad = dict(pages=pages(), seq_lens=None, cu_seqlens=A, nseq=0, total=4, freqs=A, rot_dim=64, interleaved=0, amp=1.0,
               positions=None, D=128, dt=0, stream=None)
    assert fa.fa_append_paged(rows(), rows(), rows(), None, **bad) == OK
    assert fa.fa_append_paged_fill(rows(), rows(), rows(), None, **bad) == E
