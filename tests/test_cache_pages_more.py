"""Pages that requests share, where one of them goes back to a row inside one: how it goes on without writing what the
other still reads."""
import numpy as np
import pytest

import int8_quantized_amd as q8
from test_cache_pages import Both, cache_of

torch = pytest.importorskip("torch")


def rows_of(b, codes, scales, r):
    """Request r's rows, as its table finds them."""
    at = np.arange(b.p.lens[r])
    page, row = b.p.table[r, at // b.p.page], at % b.p.page
    return codes[page, :, :, row].cpu(), scales[page, :, :, row].cpu()


def append(b, codes, scales, r, n, seed):
    """n rows behind request r's own, for which there is room."""
    g = torch.Generator().manual_seed(seed)
    at = b.p.lens[r] + np.arange(n)
    page, row = b.p.table[r, at // b.p.page], at % b.p.page
    codes[page, :, :, row] = torch.randint(-128, 128, (n,) + codes.shape[1:3] + codes.shape[4:], generator=g).to(torch.int8).cuda()
    scales[page, :, :, row] = torch.rand((n,) + scales.shape[1:3], generator=g).cuda()
    b.p.lens[r] += n
    b.lens.copy_(torch.from_numpy(b.p.lens))


@pytest.mark.gpu
@pytest.mark.parametrize("page,rows,keep", [(16, 32, 20), (16, 40, 1), (64, 128, 100), (5, 23, 18), (1, 9, 4), (16, 40, 32)])
def test_a_request_cut_inside_a_shared_page_goes_on_in_a_page_of_its_own(page, rows, keep):
    """Fork, cut back, fork into a free request (whose last page is its own), release, take, append, compact."""
    b = Both(4, 30, 100, page)
    codes, scales = cache_of(100, 2, page, 64, seed=3)
    b.grow([rows, 0, 0, 0])

    def fork(src, dst):
        made = b.fork([src], [dst])
        assert made[0, 0] == 1
        q8.q8ta_pages_copy(codes, scales, *(b.ints(made[:, i]) for i in (1, 2, 3)))
    fork(0, 1)
    theirs = rows_of(b, codes, scales, 0)
    b.release([1], [keep])
    kept = rows_of(b, codes, scales, 1)
    fork(1, 2)
    b.release([1])
    assert b.p.refs[b.p.table[2, :-(-keep // page)]].tolist()[keep // page:] == [1] * (keep % page != 0)
    b.take([0, 0, 8, 0])
    append(b, codes, scales, 2, 8, seed=5)
    mine = rows_of(b, codes, scales, 2)
    assert all(torch.equal(m[:keep], k) for m, k in zip(mine, kept))
    assert all(torch.equal(a, t) for a, t in zip(rows_of(b, codes, scales, 0), theirs))
    # the drafted rows behind the cut: 0, 2 and 5 are kept
    one = [b.ints([v]) for v in (keep, 3)]
    q8.q8ta_cache_compact(codes, scales, b.table[2:3].contiguous(), one[0], b.ints([[0, 2, 5]]), one[1])
    after = rows_of(b, codes, scales, 2)
    assert all(torch.equal(a[keep:keep + 3], m[[keep, keep + 2, keep + 5]]) for a, m in zip(after, mine))
    assert all(torch.equal(a, t) for a, t in zip(rows_of(b, codes, scales, 0), theirs))
    b.release()
    assert not b.p.refs.any()
