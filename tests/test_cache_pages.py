"""The pages of the int8 cache: q8ta_pages_take, _fork, _release, _copy and q8ta_cache_compact against plain
loops (numpy): shortages, pages and entries in no order, rows of any size and alignment, paths that overlap
what they move to, captured calls, and the calls they refuse.  Everything is whole numbers and bytes: equal.
"""
import numpy as np
import pytest

import int8_quantized_amd as q8

torch = pytest.importorskip("torch")


# ---------------------------------------------------------------- tables and holders
class Pool:
    """The tables, rows and holders as plain loops keep them."""

    def __init__(self, requests, width, pages, page, seed=0):
        self.g = np.random.default_rng(seed)
        self.page = page
        self.table = np.full((requests, width), -1, np.int32)
        self.lens = np.zeros(requests, np.int32)
        self.refs = np.zeros(pages, np.int32)

    def free(self):
        return np.flatnonzero(self.refs <= 0)

    def take(self, more):
        free, spent, granted = self.free(), 0, []
        for r, m in enumerate(more):
            rows = min(max(int(self.lens[r]), 0), self.table.shape[1] * self.page)
            end = -(-(rows + int(m)) // self.page) if m > 0 else 0
            if end > self.table.shape[1]:
                granted.append(0)
                continue
            first = end
            for j in range(rows // self.page, end):
                if self.table[r, j] < 0:
                    first = j
                    break
            need = max(0, end - first) if m > 0 else 0
            fine = need == 0 or spent + need <= len(free)
            granted.append(int(fine))
            if fine:
                self.table[r, first:first + need] = free[spent:spent + need]
                self.refs[free[spent:spent + need]] = 1
            spent += need
        return granted

    def fork(self, src, dst):
        free, spent, out = self.free(), 0, []
        R, W = self.table.shape
        old = self.table.copy()
        for s, d in zip(src, dst):
            if not (0 <= s < R and 0 <= d < R) or s == d:
                out.append((0, -1, -1, 0))
                continue
            rows = min(max(int(self.lens[s]), 0), W * self.page)
            full, part = divmod(rows, self.page)
            fine = part == 0 or spent < len(free)
            copy = (-1, -1, 0)
            if fine:
                row = np.full(W, -1, np.int32)
                row[:full] = old[s, :full]
                for p in old[s, :full]:
                    if 0 <= p < len(self.refs):
                        self.refs[p] += 1
                if part:
                    row[full] = free[spent]
                    self.refs[free[spent]] = 1
                    copy = (int(old[s, full]), int(free[spent]), part)
                self.table[d] = row
                self.lens[d] = rows
            spent += part > 0
            out.append((int(fine),) + copy)
        return np.array(out, np.int32).reshape(-1, 4)

    def release(self, rows, keep):
        for i in range(len(self.lens) if rows is None else len(rows)):
            r = i if rows is None else rows[i]
            if not 0 <= r < len(self.lens):
                continue
            k = 0 if keep is None else max(0, int(keep[i]))
            for j in range(-(-k // self.page), self.table.shape[1]):
                p = self.table[r, j]
                if p >= 0:
                    self.table[r, j] = -1
                    if p < len(self.refs):
                        self.refs[p] -= 1
            self.lens[r] = min(self.lens[r], k)


class Both:
    """A plain pool and its twin on the GPU, compared after every call."""

    def __init__(self, *args, **kw):
        self.p = Pool(*args, **kw)
        self.up()

    def up(self):
        self.table, self.lens, self.refs = (torch.from_numpy(a.copy()).cuda() for a in (self.p.table, self.p.lens, self.p.refs))

    def same(self, *pairs):
        for got, want in [(self.table, self.p.table), (self.lens, self.p.lens), (self.refs, self.p.refs), *pairs]:
            assert np.array_equal(got.cpu().numpy(), np.asarray(want)), (got.cpu().numpy(), want)

    @staticmethod
    def ints(a):
        return None if a is None else torch.tensor(np.asarray(a, np.int32)).cuda()

    def take(self, more):
        granted = torch.full((len(self.p.lens),), 7, dtype=torch.int32, device="cuda")
        q8.q8ta_pages_take(self.table, self.lens, self.p.page, self.ints(more), self.refs, granted)
        want = self.p.take(more)
        self.same((granted, want))
        return want

    def fork(self, src, dst):
        n = len(src)
        out = [torch.full((n,), 7, dtype=torch.int32, device="cuda") for _ in range(4)]
        q8.q8ta_pages_fork(self.table, self.lens, self.p.page, self.ints(src), self.ints(dst), self.refs, *out)
        want = self.p.fork(src, dst)
        self.same(*((o, want[:, i]) for i, o in enumerate(out)))
        return want

    def release(self, rows=None, keep=None):
        q8.q8ta_pages_release(self.table, self.lens, self.p.page, self.ints(rows), self.ints(keep), self.refs)
        self.p.release(rows, keep)
        self.same()

    def grow(self, more):
        """Rows are there: as an append leaves it."""
        got = self.take(more)
        self.p.lens += (np.asarray(more) * got * (np.asarray(more) > 0)).astype(np.int32)
        self.lens.copy_(torch.from_numpy(self.p.lens))


# few pages and entries, many entries, many pages: one launch or three
POOLS = [(6, 9, 40, 16), (5, 4, 9, 1), (70, 40, 1500, 48), (300, 12, 20000, 64), (4100, 5, 9000, 16), (20, 30, 70000, 16),
         (1, 1, 1, 7), (3, 5000, 300000, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("requests,width,pages,page", POOLS)
def test_a_pools_life(requests, width, pages, page):
    """Requests come, grow, fork, shrink and go, until and past the last page."""
    b = Both(requests, width, pages, page, seed=pages)
    g = b.p.g
    # some pages belong to others, so that free ones lie apart
    b.p.refs[g.random(pages) < 0.3] = 1
    b.up()
    for turn in range(12):
        more = g.integers(-3, max(2, width * page // 3), requests)
        b.grow(more)
        n = max(1, requests // 3)
        order = g.permutation(requests)
        b.release(order[:n], g.integers(-2, width * page, n) if turn % 2 else None)
        if requests > 2:
            # the last third of the order takes up what the first third holds
            b.release(order[-n:])
            b.fork(g.choice(order[:n], n), order[-n:])
    b.release()
    assert (b.p.table == -1).all() and (b.p.lens == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1, 300])
def test_shortages(scale):
    """As many pages as there are, one fewer, and requests behind one that gets none."""
    R = 5 * scale
    for pages in (10 * scale, 10 * scale - 1, 3 * scale, 1):
        b = Both(R, 4, pages, 8)
        want = b.take([16] * R)              # two pages each
        assert sum(want) == min(R, pages // 2)
        b.take([0, 16, -5, 1, 40] * scale)   # (40 rows do not fit four pages of 8)
    b = Both(4, 6, 3, 8)
    assert b.take([9, 17, 0, 1]) == [1, 0, 1, 0]     # the third asks for nothing
    b = Both(6, 3, 4, 8)
    b.grow([10, 16, 0, 0, 0, 0])
    got = b.fork([0, 1, 0, 5, 9, 2], [2, 3, 4, 5, 0, 2])
    assert got[:, 0].tolist() == [0, 1, 0, 0, 0, 0]   # no page for a part; whole pages need none; no such request


@pytest.mark.gpu
def test_forks_of_forks_share_pages():
    b = Both(8, 6, 60, 4)
    b.grow([18, 0, 0, 0, 0, 0, 0, 0])
    b.fork([0, 0], [1, 2])
    b.fork([1, 2, 0], [3, 4, 5])
    assert b.p.refs.max() == 6 and len(set(b.p.table[:6, 4].tolist())) == 6
    b.release([0, 1])
    b.release([2, 2, -1, 99, 3])             # twice, and no such requests
    b.release([4, 5], [8, 7])
    assert b.p.refs.tolist().count(2) == 2 and b.p.lens.tolist() == [0, 0, 0, 0, 8, 7, 0, 0]
    b.take([0, 30, 0, 0, 30, 0, 0, 0])       # the lowest free pages, wherever they lie


@pytest.mark.gpu
def test_entries_that_are_no_pages_and_lengths_out_of_range():
    b = Both(5, 4, 12, 4)
    b.p.table[0, :2] = [3, 40]               # one outside the cache: shared, released, never counted
    b.p.table[1, :3] = [5, 6, 1 << 30]
    b.p.refs[[3, 5, 6]] = 1
    b.p.lens[:] = [8, 10, 1 << 30, -7, 0]
    b.up()
    b.fork([0, 3], [4, 2])
    b.release([0, 1])
    b.take([4, 4, 4, 4, 4])


# ---------------------------------------------------------------- rows
def cache_of(pages, hk, page, d, seed=0, offset=0):
    g = np.random.default_rng(seed)
    n = pages * 2 * hk * page * d
    codes = torch.from_numpy(g.integers(-128, 128, n + offset).astype(np.int8)).cuda()[offset:].view(pages, 2, hk, page, d)
    scales = torch.from_numpy(g.random((pages, 2, hk, page)).astype(np.float32)).cuda()
    return codes, scales


@pytest.mark.gpu
@pytest.mark.parametrize("offset", [0, 1, 4])
@pytest.mark.parametrize("hk,page,d", [(1, 1, 1), (2, 16, 64), (8, 64, 128), (3, 7, 5), (1, 48, 80), (4, 16, 256), (5, 300, 12),
                                       (2, 2, 4500), (1, 3, 65536)])
def test_pages_copy(hk, page, d, offset):
    pages = 12
    codes, scales = cache_of(pages, hk, page, d, seed=d, offset=offset)
    order = np.random.default_rng(1).permutation(pages)
    src = np.array([order[0], order[1], -1, order[0], 99, order[2], order[3], order[4]], np.int32)
    dst = np.array([order[6], order[7], order[8], order[9], order[10], -5, order[3], 1 << 30], np.int32)
    for rows in (None, np.array([page, 0, 3, page // 2 + 1, 1, 2, 3, 1], np.int32), np.array([-1, 1 << 30, 1, 1, 1, 1, 1, 1], np.int32)):
        want = [t.cpu().numpy().copy() for t in (codes, scales)]
        for i, (a, b) in enumerate(zip(src, dst)):
            if 0 <= a < pages and 0 <= b < pages:
                n = page if rows is None else min(max(int(rows[i]), 0), page)
                for w in want:
                    w[b, :, :, :n] = w[a, :, :, :n]
        q8.q8ta_pages_copy(codes, scales, *(None if a is None else torch.from_numpy(a).cuda() for a in (src, dst, rows)))
        assert np.array_equal(codes.cpu().numpy(), want[0]) and np.array_equal(scales.cpu().numpy(), want[1])


def compacted(codes, scales, table, base, path, counts):
    """Every row moved at once, from what was there before."""
    pages, _, hk, page, d = codes.shape
    old, new = (codes, scales), (codes.copy(), scales.copy())
    for b in range(len(base)):
        for i in range(min(max(int(counts[b]), 0), path.shape[1])):
            s, t = int(base[b]) + int(path[b, i]), int(base[b]) + i
            if path[b, i] <= i or base[b] < 0 or s >= table.shape[1] * page:
                continue
            ps, pt = table[b, s // page], table[b, t // page]
            if 0 <= ps < pages and 0 <= pt < pages:
                for o, n in zip(old, new):
                    n[pt, :, :, t % page] = o[ps, :, :, s % page]
    return new


def check_compact(codes, scales, table, base, path, counts):
    want = compacted(codes.cpu().numpy(), scales.cpu().numpy(), table, base, path, counts)
    q8.q8ta_cache_compact(codes, scales, *(torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda() for a in (table, base, path, counts)))
    assert np.array_equal(codes.cpu().numpy(), want[0]) and np.array_equal(scales.cpu().numpy(), want[1])


def tables(B, width, pages, seed=0):
    return np.random.default_rng(seed).permutation(pages)[:B * width].reshape(B, width).astype(np.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("offset", [0, 2, 8])
@pytest.mark.parametrize("hk,page,d", [(1, 1, 1), (2, 16, 64), (8, 64, 128), (3, 7, 5), (1, 48, 80), (4, 16, 256), (2, 5, 4500), (1, 16, 65536)])
def test_compact_trees(hk, page, d, offset):
    """Kept tokens of drafted trees behind contexts of any length."""
    g = np.random.default_rng(d + page)
    B, n = 5, 12
    width = -(-60 // page) + 1
    codes, scales = cache_of(B * width + 2, hk, page, d, seed=d, offset=offset)
    path = np.full((B, n), -1, np.int32)
    counts = np.array([0, 1, 5, 12, 7], np.int32)
    for b in range(B):
        path[b, :counts[b]] = np.sort(g.choice(n, counts[b], replace=False))
    check_compact(codes, scales, tables(B, width, B * width + 2), np.array([3, 17, 40, 0, 31]), path, counts)


@pytest.mark.gpu
@pytest.mark.parametrize("d,page", [(128, 64), (16, 16), (48, 3), (256, 32), (7, 16)])
@pytest.mark.parametrize("kind", ["every other", "one out", "window", "far window", "all", "random"])
def test_compact_long_paths(kind, d, page):
    """Rows of a whole context: sources that lie among the rows that others move to, and sources that do not."""
    g = np.random.default_rng(len(kind) + d)
    n = 2900
    all_rows = np.arange(n)
    keep = {"every other": all_rows[::2], "one out": np.delete(all_rows, 5), "window": np.concatenate((all_rows[:4], all_rows[-2000:])),
            "far window": np.concatenate((all_rows[:7], all_rows[-1300:])), "all": all_rows,
            "random": np.sort(g.choice(n, 1700, replace=False))}[kind]
    B = 2
    width = -(-(n + 40) // page)
    codes, scales = cache_of(B * width, 2, page, d, seed=1)
    path = np.tile(np.pad(keep, (0, 9), constant_values=1 << 30), (B, 1)).astype(np.int32)
    check_compact(codes, scales, tables(B, width, B * width), np.array([0, 33]), path, np.array([len(keep), len(keep) - 1]))


@pytest.mark.gpu
def test_compact_lists_and_tables_out_of_range():
    codes, scales = cache_of(9, 2, 8, 32, seed=4)
    table = np.array([[0, 1, -1], [3, 1 << 30, 5], [6, 7, 8], [6, 7, 8]], np.int32)
    path = np.array([[0, 2, 9, 18, 23], [1, 8, 9, 17, 22], [4, 5, 1 << 30, 0, 0], [1, 2, 3, 4, 5]], np.int32)
    base = np.array([0, 1, 2, -1])
    for counts in ([5, 5, 3, 5], [99, 4, 2, 1 << 30], [-1, 0, -(1 << 31), 0]):
        check_compact(codes, scales, table, base, path, np.array(counts))


@pytest.mark.gpu
def test_compact_past_32_bits():
    """Rows behind 2^32 bytes of codes."""
    pages, hk, page, d = 33000, 8, 64, 128
    codes = torch.zeros((pages, 2, hk, page, d), dtype=torch.int8, device="cuda")
    scales = torch.zeros((pages, 2, hk, page), device="cuda")
    assert codes.numel() > 1 << 32
    last = pages - 1
    g = torch.Generator(device="cuda").manual_seed(1)
    codes[last] = torch.randint(-128, 128, codes[last].shape, generator=g, device="cuda", dtype=torch.int8)
    scales[last] = torch.rand(scales[last].shape, generator=g, device="cuda")
    want = codes[last].clone()
    table = torch.tensor([[last, 5]], dtype=torch.int32, device="cuda")
    path = torch.tensor([[0, 30, 63]], dtype=torch.int32, device="cuda")
    ints = [torch.tensor([v], dtype=torch.int32, device="cuda") for v in (0, 3)]
    q8.q8ta_cache_compact(codes, scales, table, ints[0], path, ints[1])
    want[:, :, 1], want[:, :, 2] = want[:, :, 30].clone(), want[:, :, 63].clone()
    assert torch.equal(codes[last], want) and not codes[:last].any()
    q8.q8ta_pages_copy(codes, scales, torch.tensor([last], dtype=torch.int32, device="cuda"),
                       torch.tensor([7], dtype=torch.int32, device="cuda"))
    assert torch.equal(codes[7], want) and torch.equal(scales[7], scales[last])


@pytest.mark.gpu
def test_a_captured_step_takes_and_frees_pages():
    """Release, fork, copy and take in one graph: replays find what eager calls and other replays left."""
    page, R, W, pages = 16, 9, 8, 120
    b = Both(R, W, pages, page, seed=3)
    b.grow([37, 50] + [0] * 7)
    codes, scales = cache_of(pages, 2, page, 64, seed=2)
    src, dst = [0, 0, 1, 1, 0], [2, 3, 4, 5, 6]
    more = [0, 0, 20, 3, 40, 1, 9, 0, 0]
    s, t, m = Both.ints(src), Both.ints(dst), Both.ints(more)
    out = [torch.zeros(5, dtype=torch.int32, device="cuda") for _ in range(4)]
    granted = torch.zeros(R, dtype=torch.int32, device="cuda")

    def step():
        q8.q8ta_pages_release(b.table, b.lens, page, t, None, b.refs)
        q8.q8ta_pages_fork(b.table, b.lens, page, s, t, b.refs, *out)
        q8.q8ta_pages_copy(codes, scales, out[1], out[2], out[3])
        q8.q8ta_pages_take(b.table, b.lens, page, m, b.refs, granted)
    saved = [x.clone() for x in (b.table, b.lens, b.refs)]
    step()
    torch.cuda.synchronize()
    for x, y in zip((b.table, b.lens, b.refs), saved):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(4):
        before = codes.cpu().numpy()
        graph.replay()
        torch.cuda.synchronize()
        b.p.release(dst, None)
        want = b.p.fork(src, dst)
        for _, a, c, n in want:
            before[c, :, :, :n] = before[a, :, :, :n]
        served = b.p.take(more)
        b.same((granted, served), *((o, want[:, i]) for i, o in enumerate(out)))
        assert np.array_equal(codes.cpu().numpy(), before)
        b.release([7, 8] if turn % 2 else [2, 5])       # eager work between the replays
        b.take([0] * 7 + [16, 16])


# ---------------------------------------------------------------- refusals
FAKE = 4096


def status(name, args):
    rc = getattr(q8.lib(), name)(*args)
    return rc, q8.q8ta_last_error()


def test_tables_refuse():
    take = dict(t=FAKE, R=4, W=8, page=16, lens=FAKE, more=FAKE, refs=FAKE, pages=64, g=FAKE, st=None)
    fork = dict(t=FAKE, R=4, W=8, page=16, lens=FAKE, src=FAKE, dst=FAKE, n=2, refs=FAKE, pages=64, g=FAKE, a=FAKE, b=FAKE, c=FAKE, st=None)
    release = dict(t=FAKE, R=4, W=8, page=16, lens=FAKE, rows=FAKE, keep=None, n=2, refs=FAKE, pages=64, st=None)
    for name, base in (("q8ta_pages_take", take), ("q8ta_pages_fork", fork), ("q8ta_pages_release", release)):
        for kw in (dict(R=-1), dict(R=(1 << 24) + 1), dict(W=0), dict(page=0), dict(W=1 << 28, page=8), dict(pages=0), dict(pages=1 << 31),
                   dict(R=1 << 24, W=1 << 17, page=1)):
            rc, said = status(name, {**base, **kw}.values())
            assert rc == q8.Q8TA_ERR_SHAPE and name in said, (name, kw, rc, said)
        for p in [k for k in base if base[k] == FAKE and k != "rows"]:
            rc, said = status(name, {**base, p: None}.values())
            assert rc == q8.Q8TA_ERR_NULL and name in said, (name, p, rc, said)
    for base, name in ((fork, "q8ta_pages_fork"), (release, "q8ta_pages_release")):
        for n in (-1, (1 << 24) + 1):
            assert status(name, {**base, "n": n}.values())[0] == q8.Q8TA_ERR_SHAPE
        assert status(name, {**base, "n": 0}.values())[0] == q8.Q8TA_OK
    assert status("q8ta_pages_take", {**take, "R": 0}.values())[0] == q8.Q8TA_OK
    rc, said = status("q8ta_pages_release", {**release, "rows": None}.values())     # all requests, but n says two
    assert rc == q8.Q8TA_ERR_SHAPE and "rows" in said


def test_rows_refuse():
    copy = dict(c=FAKE, s=FAKE, pages=64, page=16, hk=2, d=64, src=FAKE, dst=FAKE, rows=None, n=3, st=None)
    compact = dict(c=FAKE, s=FAKE, pages=64, page=16, hk=2, d=64, t=FAKE, B=2, W=8, base=FAKE, path=FAKE, n=5, counts=FAKE, st=None)
    for name, base in (("q8ta_pages_copy", copy), ("q8ta_cache_compact", compact)):
        for kw in (dict(pages=0), dict(pages=1 << 31), dict(page=0), dict(hk=0), dict(hk=32768), dict(d=0), dict(d=65537), dict(n=-1),
                   dict(n=1 << 31), dict(pages=1 << 30, page=1 << 10)):
            rc, said = status(name, {**base, **kw}.values())
            assert rc == q8.Q8TA_ERR_SHAPE and name in said, (name, kw, rc, said)
        for p in [k for k in base if base[k] == FAKE]:
            assert status(name, {**base, p: None}.values())[0] == q8.Q8TA_ERR_NULL, (name, p)
        assert status(name, {**base, "n": 0}.values())[0] == q8.Q8TA_OK
    for kw in (dict(B=-1), dict(B=(1 << 24) + 1), dict(W=0), dict(W=1 << 28), dict(B=1 << 24, n=1 << 17), dict(B=1 << 24, W=1 << 17, page=1)):
        assert status("q8ta_cache_compact", {**compact, **kw}.values())[0] == q8.Q8TA_ERR_SHAPE, kw
    assert status("q8ta_cache_compact", {**compact, "B": 0}.values())[0] == q8.Q8TA_OK


@pytest.mark.gpu
def test_bindings_refuse_shapes():
    table = torch.zeros(4, 8, dtype=torch.int32, device="cuda")
    lens, two = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    refs = torch.zeros(10, dtype=torch.int32, device="cuda")
    codes, scales = cache_of(3, 2, 4, 8)
    for call in (lambda: q8.q8ta_pages_take(table, lens[:3], 16, lens, refs, lens), lambda: q8.q8ta_pages_take(table, lens, 16, two, refs, lens),
                 lambda: q8.q8ta_pages_take(table, lens, 16, lens, refs, two), lambda: q8.q8ta_pages_take(table[0], lens, 16, lens, refs, lens),
                 lambda: q8.q8ta_pages_fork(table, lens, 16, two, lens, refs, two, two, two, two),
                 lambda: q8.q8ta_pages_fork(table, lens, 16, table, table, refs, two, two, two, two),
                 lambda: q8.q8ta_pages_release(table, lens, 16, two, lens, refs), lambda: q8.q8ta_pages_release(table, lens, 16, None, two, refs),
                 lambda: q8.q8ta_pages_copy(codes, scales[:2], two, two), lambda: q8.q8ta_pages_copy(codes, scales, two, lens),
                 lambda: q8.q8ta_pages_copy(codes, scales, two, two, lens),
                 lambda: q8.q8ta_cache_compact(codes, scales, table, lens, two, lens),
                 lambda: q8.q8ta_cache_compact(codes, scales, table, two, table, lens),
                 lambda: q8.q8ta_cache_compact(codes[0], scales, table, lens, table, lens)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises((ValueError, TypeError)):
        q8.q8ta_pages_release(table.long(), lens, 16, None, None, refs)
