"""Launches, workspaces and waits of the decode-step operators, on a runtime that writes them down (CPU)."""
import math

from recorder import recorded

LORA = """
def lora(M, K, N, r=8, na=2, ad=2, out=2, x=F, w=F, a=F, s=None):
    rc = l.q8ta_linear_lora(x, M, K, 0.02, 3, w, N, F, None, a, F, ad, na, r, None, None, F, b"none", F, out, s)
    return rc, calls()
"""


def launches(lines, name):
    return [[int(v) for v in x[2:8]] for x in lines if x[0] == "launch" and name in x[1]]


def test_linear_lora_grids_hold_every_channel():
    """Up to the header's 2^30 channels: no launch passes 2^32 threads, and the launches' tiles hold
    all channels, whatever their number."""
    cases = [(M, 64, N) for M in (1, 16, 17, 33, 64) for N in
             (1, 48, 49, 4096, 11008, 402653184, 402653185, 500000000, 1 << 30)]
    got = recorded(LORA + f"result = [lora(*c) for c in {cases!r}]")
    for (M, K, N), (rc, lines) in zip(cases, got):
        assert rc == 0, (M, N, lines)
        rows = launches(lines, "k_lora_rows")
        wide = {16 * c for c in (1, 2, 3) if sum(g[0] for g in rows) == math.ceil(N / (16 * c))}
        assert rows and wide and all(g[0] * g[3] < 2 ** 32 for g in rows), (M, N, rows)


def test_linear_lora_copies_hold_every_row():
    """Rows copied for their alignment: 16 bytes a thread, as many launches as it takes."""
    cases = [(1, 3, 1 << 30), (2, 1001, 1 << 26), (70, 1001, 4096), (1, 1, 1 << 30), (3, 17, 5)]
    got = recorded(LORA + f"result = [lora(*c) for c in {cases!r}]")
    for (M, K, N), (rc, lines) in zip(cases, got):
        assert rc == 0, (M, K, N, lines)
        kp = (K + 63) // 64 * 64
        pads = launches(lines, "k_pad_rows")
        chunks = sum(math.ceil(n * kp * e / 16 / 256) for n, e in ((M, 1), (N, 1), (2 * 8, 2)))
        assert all(g[0] * g[3] < 2 ** 32 for g in pads)
        assert chunks <= sum(g[0] for g in pads) <= chunks + len(pads)
