"""Host code of the block with scales per token, of the verification and of the cache's pages over their
stated ranges, on the CPU: what a call launches and allocates (a runtime that writes calls down refuses what
a launch cannot hold), as built and under AddressSanitizer and UndefinedBehaviorSanitizer.
"""
import math

import numpy as np
import pytest

from recorder import recorded

SWEEP = """
def grids(name):
    lines = calls()
    out = [[int(v) for v in x[2:8]] for x in lines if x[0] == "launch" and name in x[1]]
    return out, [int(x[2]) for x in lines if x[0] == "malloc"], [x[1] for x in lines if x[0] == "launch"]
result = []
norm, linear, verify, take, copy, compact = SIZES
for T, N, dt, odd in norm:
    x = ctypes.c_void_p((1 << 20) + odd)
    rc = l.q8ta_norm_quantize(x, N, F, N, dt, T, N, F, F, 0, 1.0, F, 1e-6, F, F, F, None)
    result.append(["norm", [T, N], rc] + list(grids("k_norm")))
for M, K, N, dt, odd in linear:
    x = ctypes.c_void_p((1 << 20) + odd)
    rc = l.q8ta_linear_per_token(x, M, K, F, F, N, F, None, b"none", F, dt, None)
    result.append(["linear", [M, K, N, odd], rc] + list(grids("scaled")))
    rc = l.q8ta_gated_linear(x, M, K, F, F, F, None, F, F, None, N, b"silu", F, dt, None)
    result.append(["gated", [M, K, N, odd], rc] + list(grids("scaled")))
for B, T, V, dt, draft in verify:
    rec.recorder_capture(1)     # the call's own allocation, as large as it asks for
    rc = l.q8ta_verify_drafts(F, T * V, V, F if draft else None, T * V, V, dt, B, T, V, F, None, None, F, None, F, F, F, F, None)
    result.append(["verify", [B, T, V, draft], rc] + list(grids("k_verify")))
    rec.recorder_capture(0)
for R, W, page, pages, n in take:
    rec.recorder_capture(1)
    rc = l.q8ta_pages_take(F, R, W, page, F, F, F, pages, F, None)
    result.append(["take", [R, pages], rc] + list(grids("k_pages")))
    rc = l.q8ta_pages_fork(F, R, W, page, F, F, F, n, F, pages, F, F, F, F, None)
    result.append(["fork", [n, pages], rc] + list(grids("k_pages")))
    rec.recorder_capture(0)
    rc = l.q8ta_pages_release(F, R, W, page, F, F, None, n, F, pages, None)
    result.append(["release", [n], rc] + list(grids("k_pages_release")))
for pages, page, hk, d, n, odd in copy:
    rc = l.q8ta_pages_copy(ctypes.c_void_p((1 << 20) + odd), F, pages, page, hk, d, F, F, None, n, None)
    result.append(["copy", [n, hk], rc] + list(grids("k_pages_copy")))
for pages, page, hk, d, B, W, n, odd in compact:
    rc = l.q8ta_cache_compact(ctypes.c_void_p((1 << 20) + odd), F, pages, page, hk, d, F, B, W, F, F, n, F, None)
    result.append(["compact", [B, n, hk, d], rc] + list(grids("k_cache_compact")))
"""


def sizes(n):
    g = np.random.default_rng(99)

    def one(lo, hi):
        return int(np.clip(round(math.exp(g.uniform(math.log(lo), math.log(hi)))), lo, hi))
    norm = [(min(one(1, 2 ** 31 - 1), (1 << 40) // N), N, int(g.integers(0, 3)), int(g.integers(0, 2)) * 2)
            for N in (one(1, 1 << 30) for _ in range(n))]
    norm += [(2 ** 31 - 1, 512, 2, 0), (1, 1 << 30, 0, 0), ((1 << 21) + 1, 8, 1, 0)]
    linear = []
    for _ in range(n):
        K = one(1, 1 << 16)
        N = min(one(1, 1 << 30), (1 << 40) // K)
        M = min(one(1, 1 << 21), (1 << 40) // max(K, N))
        linear.append((M, K, N, int(g.integers(0, 3)), int(g.integers(0, 4) == 0)))
    linear += [(1 << 21, 64, 1 << 19, 2, 0), (1 << 10, 1 << 10, 1 << 30, 0, 0), (65, 1 << 30, 1 << 10, 1, 0), (16, 1 << 6, 1 << 30, 1, 0),
               (1 << 21, 16, 1, 0, 0), (64, 32, 1 << 30, 2, 0)]
    verify = [(one(1, 65535), one(1, 64), one(1, 1 << 24), int(g.integers(0, 3)), int(g.integers(0, 2))) for _ in range(n)]
    verify += [(65535, 64, 1 << 24, 0, 1), (1, 1, 1, 2, 1), (65535, 1, 1, 1, 0)]
    take = []
    for _ in range(n):
        page = one(1, 4096)
        W = one(1, (2 ** 31 - 1) // page)
        R = min(one(1, 1 << 24), (1 << 40) // W)
        take.append((R, W, page, one(1, 2 ** 31 - 1), one(1, 1 << 24)))
    take += [(4096, 8, 16, 65536, 4096), (4097, 8, 16, 65536, 4097), (1, 1, 1, 65537, 1), (1 << 24, 1 << 16, 1, 2 ** 31 - 1, 1 << 24)]
    copy, compact = [], []
    for _ in range(n):
        hk, d = one(1, 32767), one(1, 65536)
        page = min(one(1, 1 << 20), max(1, (1 << 39) // (hk * d)))
        pages = max(1, min(one(1, 2 ** 31 - 1), (1 << 39) // (hk * d * page)))
        if pages * page * hk * d * 2 > 1 << 40:
            continue
        odd = int(g.choice([0, 0, 4, 1]))
        copy.append((pages, page, hk, d, one(1, 2 ** 31 - 1), odd))
        B = one(1, 1 << 24)
        W = max(1, min(one(1, (2 ** 31 - 1) // page), (1 << 40) // B))
        compact.append((pages, page, hk, d, B, W, max(1, min(one(1, 2 ** 31 - 1), (1 << 40) // B)), odd))
    compact += [(1, 1, 1, 65536, 1, 1, 2 ** 31 - 1, 1), (1, 16, 32767, 128, 1 << 24, 1, 64, 0)]
    return norm, linear, verify, take, copy, compact


def sweep(n, **kw):
    seen = {}
    for what, size, rc, grids, mallocs, names in recorded(SWEEP.replace("SIZES", repr(sizes(n))), **kw):
        assert rc == 0, (what, size, rc, grids)
        seen[what] = seen.get(what, 0) + 1
        blocks = [g[0] * g[1] * g[2] for g in grids]
        if what == "norm":
            assert sum(blocks) == size[0] if size[1] > 16384 or size[0] <= 1 else sum(blocks) > 0, (size, grids)
        elif what in ("linear", "gated"):
            assert sum(blocks) >= 1
            M, K, N, odd = size
            if K % 16 or odd:
                kp = (K + 15) // 16 * 16
                assert len(mallocs) <= 1 and all(m >= (M + (1 + (what == "gated")) * N) * kp for m in mallocs), (size, mallocs)
            else:
                assert not mallocs, (size, mallocs)
        elif what == "verify":
            assert mallocs[0] <= 33 << 20, (size, mallocs)
            B, T, V, draft = size
            rows = T + (T - 1 if draft else 0)
            stats = [g[0] for g, k in zip(grids, names) if "stats" in k]
            picks = [g[0] for g, k in zip(grids, names) if "pick" in k]
            assert sum(stats) == B * rows * -(-V // 4096) and sum(picks) == B, (size, stats, picks)
        elif what in ("take", "fork"):
            if size[0] <= 4096 and size[1] <= 65536:
                assert not mallocs
            else:
                assert mallocs[0] <= 16 * size[0] + 8 * (-(-size[1] // 4096)) + 64, (size, mallocs)
    assert set(seen) == {"norm", "linear", "gated", "verify", "take", "fork", "release", "copy", "compact"}
    assert min(seen.values()) > n // 2, seen


def test_planning():
    sweep(120)


def test_planning_under_asan_ubsan():
    from sanitized import sanitized
    from test_host_sanitizers import SAN_ENV, _clang_asan_runtime
    asan = _clang_asan_runtime()
    if asan is None:
        pytest.skip("clang's AddressSanitizer runtime is not installed")
    with sanitized() as lib:
        sweep(60, lib=lib, preload=[asan], env=SAN_ENV)
