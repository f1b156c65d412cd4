"""Workspaces of q8ta_verify_drafts at their largest, and that the launches of the calls beside it hold every token,
tile, page and row (CPU: a runtime that writes calls down)."""
import re
import subprocess

from recorder import recorded
from test_host_drafts import SWEEP, sizes


def sweep(*lists):
    lists = list(lists) + [[]] * (6 - len(lists))
    out = recorded(SWEEP.replace("SIZES", repr(tuple(lists))))
    mangled = sorted({n for r in out for n in r[5]})
    names = subprocess.run(["c++filt"], input="\n".join(mangled), capture_output=True, text=True, check=True).stdout.split("\n")
    plain = {m: n.replace("q8ta::", "").replace("(anonymous namespace)::", "") for m, n in zip(mangled, names)}
    for what, size, rc, grids, mallocs, kernels in out:
        assert rc == 0, (what, size)
        yield what, size, [g[0] * g[1] * g[2] for g in grids], grids, mallocs, [plain[k] for k in kernels]


def up(a, b):
    return -(-a // b)


def test_verify_workspace_is_bounded():
    """Many requests of few tokens, whose sums and last nodes take as much as the statistics."""
    cases = [(B, T, V, 0, draft) for B in (65535, 50000, 20000, 3000) for T in (1, 2, 5, 64) for V in (1, 4096, 4097, 65536, 131072, 1 << 24)
             for draft in (0, 1)]
    for _, (B, T, V, draft), _, grids, mallocs, kernels in sweep([], [], cases):
        assert len(mallocs) == 1 and mallocs[0] <= 33 * 10 ** 6, (B, T, V, draft, mallocs)
        chunks, rows = up(V, 4096), T + (T - 1 if draft else 0)
        for name, each in (("stats", rows * chunks), ("walk", chunks), ("pick", 1)):
            assert sum(g[0] for g, k in zip(grids, kernels) if name in k) == B * each, (B, T, V, draft, name)


def tiles(name, M, N):
    """What a launch of this kernel has to hold for all of [M, N]: a number, or what its mixed tiles may add up to."""
    args = re.search(r"k_scaled_rows<([^>]*)>", name)
    if args:
        _, mats, mt, fn = [a.strip() for a in args[1].split(",")][:4]
        return {up(M, 16 * int(mt)) * up(N, 16 * int(fn) // int(mats))}
    shapes = [tuple(int(v) for v in t.split(",")) for t in re.findall(r"Tile<([^>]*)>", name)]
    mats = int(re.search(r"Tile<[^>]*>, (\d), ", name)[1])
    (wn, wm, fn, fm), (_, wm2, _, fm2) = shapes
    n, ma, mb = up(N, 32 * fn * wn // mats), up(M, 32 * fm * wm), up(M, 32 * fm2 * wm2)
    return {ma * n} if shapes[0] == shapes[1] else {ma * c + mb * (n - c) for c in range(1, n)}


def test_launches_hold_all_tokens_and_tiles():
    norm, linear = sizes(120)[:2]
    norm += [(T, N, 2, 0) for T in (511, 512, 1 << 21, (1 << 22) + 5) for N in (8, 4104, 6152, 8192, 16384, 16392)]
    linear += [(M, K, N, 2, 0) for M in (1, 40, 100, 700, 1500, 2048, 5000) for K in (64, 4096) for N in (100, 4096, 11008, 28000)]
    mixed = 0
    for what, size, blocks, grids, _, kernels in sweep(norm, linear):
        if what == "norm":
            assert sum(blocks) == size[0], (size, grids)
            continue
        M, _, N, _ = size
        kernels = [k for k in kernels if "copy_rows" not in k]
        assert len(set(kernels)) == 1, (what, size, kernels)
        want = tiles(kernels[0], M, N)
        mixed += len(want) > 1
        assert sum(blocks) in want, (what, size, kernels, grids)
    assert mixed > 2


def test_launches_hold_all_pages_and_rows():
    take, copy, compact = sizes(120)[3:]
    for what, size, blocks, grids, _, kernels in sweep([], [], [], take, copy, compact):
        if what == "release":
            assert blocks == [min(size[0], 65536)], (size, grids)
        elif what == "copy":
            n, hk = size
            assert grids[0][:3] == [min(n, 1 << 22), up(2 * hk, 4), 1], (size, grids)
        elif what == "compact":
            B, n, hk, d = size
            unit, F = re.search(r"k_cache_compact<(.*), (\d)>", kernels[0]).groups()
            unit = {"unsigned int": 4, "unsigned char": 1}.get(unit, 16)
            units = 256 * int(F)                          # of a workgroup
            width = min(d, units * unit)                  # bytes of a slice
            stretch = min(units // (width // unit), 512, n)
            assert grids[0][:3] == [min(up(n, stretch), 1 << 18) * up(d, width), 2 * hk, min(B, 65535)], (size, grids, kernels)
