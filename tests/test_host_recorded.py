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


# q8ta_linear_lora takes a workspace on every call: its waits are those of the workspaces.
WORK = LORA + """
A, B, C, D, E = (ctypes.c_void_p(v << 12) for v in range(1, 6))
def call(s, M=4):
    rc, lines = lora(M, 64, 64, s=s)
    assert rc == 0
    return [x for x in lines if x[0] != "launch"]
"""


def test_workspace_calls_on_the_default_stream_need_no_events():
    got = recorded(WORK + "result = [call(None) for _ in range(4)] + [call(None, M=1 << 16), call(None)]")
    assert [x[0] for x in got[0]] == ["malloc"] and got[1:4] == [[], [], []]
    assert [x[0] for x in got[4]] == ["free", "malloc"] and got[5] == []      # grown, in the stream's order


def test_workspace_of_a_side_stream_leaves_the_default_stream_alone():
    """No call on a side stream records on the default stream or waits for it as a whole."""
    got = recorded(WORK + """
rec.recorder_pending(1)     # everything queued is still running
result = [call(None), call(A), call(A), call(None), call(B), call(None)]""")
    none = "(nil)"
    assert not any(x[0] in ("record", "wait") and x[2] == none for part in (got[1], got[2], got[4]) for x in part)
    assert [x[0] for x in got[1]] == ["malloc", "record"] and got[1][1][2] == "0x1000"
    assert not any(x[0] == "malloc" for x in got[2])                  # its own buffer again
    assert [x[0] for x in got[4]] == ["malloc", "record"]
    assert got[3] == got[5] == []                                     # the default stream needs none still


def test_workspace_shared_by_more_streams_than_buffers():
    """With every buffer in some stream's name, a further stream waits for one use of one of them."""
    got = recorded(WORK + """
rec.recorder_pending(1)
result = [call(s) for s in (A, None, B, C, D, D, None, None, E, E)]""")
    assert [x[0] for x in got[4]] == ["query", "wait", "record"]
    assert got[4][1][1] == got[4][0][1] and got[4][1][2] == got[4][2][2] == "0x4000"
    assert [x[0] for x in got[5]] == ["query", "wait", "record"]
    # from then on the default stream records its uses too (without waiting for its own)
    assert [(x[0], x[2]) for x in got[6] + got[7]] == [("record", "(nil)")] * 2
    # released on a side stream, an event is waited for by whoever comes next
    got = recorded(WORK + "result = [call(s) for s in (None, A, B, C, D)]")
    assert [x[0] for x in got[4]] == ["query", "record"]               # (ready: no wait)


def test_workspace_of_the_default_stream_without_an_event_is_not_handed_on():
    """Its event (the first) is neither recorded for nor asked for by another stream."""
    got = recorded(WORK + "result = [call(s) for s in (None, A, B, C, D, E)]")
    events = [[x[1] for x in part if x[0] in ("record", "query", "wait")] for part in got]
    assert events[0] == [] and all(part and "0x1" not in part for part in events[1:])


def test_workspace_under_capture_is_the_calls_own():
    got = recorded(WORK + """
call(None)
rec.recorder_capture(1)
result = [call(A), call(None)]""")
    for part in got:
        assert [x[0] for x in part] == ["malloc", "free"] and part[0][1] == part[1][1]


def test_sample_workspace_is_what_the_header_states():
    """0.05 to 0.7 MB a row and 110 MB at most (with a cached buffer's rounding), whatever the rows,
    the vocabulary and the type; every launch group holds all its rows."""
    rows = [1, 2, 63, 64, 65, 300, 1000, 1022, 1023, 1024, 1025, 2047, 2048, 5000]
    vocabs = [1, 33, 1000, 32000, 100003, 131072, 262144, 262145, 500000, (1 << 20) - 1, 1 << 20, (1 << 20) + 1,
              1 << 21, (1 << 21) + 1, 1 << 24]
    cases = [(b, v, t) for b in rows for v in vocabs for t in (0, 2)]
    got = recorded("""
def sample(rows, vocab, dtype):
    rc = l.q8ta_sample(F, vocab, dtype, rows, vocab, F, F, F, F, F, F, F, None)
    return rc, calls()
result = []
for c in %r:
    rec.recorder_capture(1)      # the call's own allocation, as large as it asks for
    own = sample(*c)
    rec.recorder_capture(0)
    result.append((own, sample(*c)))""" % cases)
    cached = 0
    for (b, v, t), ((rc, own), (rc2, lines)) in zip(cases, got):
        assert rc == rc2 == 0
        n = 16 // (4 if t == 0 else 2)
        picks = launches(own, "k_sample_pick") + launches(own, "k_sample_long")
        assert sum(g[0] for g in picks) == b
        size = [int(x[2]) for x in own if x[0] == "malloc"]
        if v > n << 18:
            assert size == []
        else:
            batch = max(g[0] for g in picks)
            assert 0.05e6 <= size[0] / batch <= 0.7e6 and size[0] <= 110e6, (b, v, t, size)
        cached += sum(int(x[2]) for x in lines if x[0] == "malloc")
        assert all(int(x[2]) <= 110e6 for x in lines if x[0] == "malloc"), (b, v, t, lines)
    assert cached > 0
