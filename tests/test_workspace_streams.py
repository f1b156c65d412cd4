"""Workspaces on several streams: calls of a side stream run beside a long queue of the default one."""
import pytest

import int8_quantized_amd as q8

torch = pytest.importorskip("torch")


def sampler(rows, vocab, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    f = [torch.randn((rows, vocab), generator=g, device="cuda") * 3, torch.full((rows,), 0.8, device="cuda"),
         torch.full((rows,), 40, dtype=torch.int32, device="cuda"), torch.full((rows,), 0.95, device="cuda"), None,
         torch.rand(rows, generator=g, device="cuda")]
    out = torch.empty(rows, dtype=torch.int32, device="cuda")

    def call(stream=None):
        q8.q8ta_sample(*f, out, None, stream=stream)
        return out
    return call


def occupy(ms):
    """Keeps the default stream busy for about `ms` milliseconds, with one small kernel."""
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda._sleep(1000)
    a.record()
    torch.cuda._sleep(1000000)
    b.record()
    torch.cuda.synchronize()
    torch.cuda._sleep(int(1000000 * ms / a.elapsed_time(b)))
    end = torch.cuda.Event()
    end.record()
    return end


def beside_the_default_stream():
    """A stream whose kernels run beside the default one's: a process has few hardware queues, and streams
    that share one with it run after what is queued there, whoever launches."""
    x = torch.zeros(64, device="cuda")
    for _ in range(12):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            x.add_(1.0)
        torch.cuda.synchronize()
        end = occupy(30)
        with torch.cuda.stream(side):
            x.add_(1.0)
        side.synchronize()
        beside = not end.query()
        torch.cuda.synchronize()
        if beside:
            return side
    pytest.skip("no stream has a hardware queue of its own")


@pytest.mark.gpu
@pytest.mark.parametrize("before", ["default", "both"])
def test_side_stream_does_not_wait_for_the_default_stream(before):
    """The side stream's call ends while the default stream is still at what was queued there, also where
    the buffers were last used there."""
    side = beside_the_default_stream()
    calls = [sampler(4, 5000, s) for s in range(3)]
    want = []
    for c in calls:
        want.append(c().clone())
    if before == "both":
        calls[0](side)
        calls[0]()
    torch.cuda.synchronize()
    end = occupy(300)
    for _ in range(3):
        for c in calls:
            c(side)
    side.synchronize()
    assert not end.query(), "the side stream waited for the default one"
    for c, w in zip(calls, want):
        assert torch.equal(c(side), w)
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_workspaces_of_many_streams_do_not_mix():
    """More streams than buffers, all at work at once, the default stream among them."""
    streams = [None] + [torch.cuda.Stream() for _ in range(6)]
    calls = [sampler(3 + i, 3000 + 517 * i, i) for i in range(len(streams))]
    want = [c().clone() for c in calls]
    torch.cuda.synchronize()
    for turn in range(20):
        outs = [c(s) for c, s in zip(calls, streams[turn % 7:] + streams[:turn % 7])]
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w), turn
            o.fill_(-9)
        torch.cuda.synchronize()
