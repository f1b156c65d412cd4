"""examples/speculative_decode.py's main: each request goes on from the last token that it said itself."""
import pytest

from test_speculative_decode import example

torch = pytest.importorskip("torch")


@pytest.mark.gpu
def test_every_request_goes_on_from_its_own_last_token(monkeypatch):
    ex = example()
    generate, calls = ex.generate, []

    def watched(model, rows, known, *args, **kw):
        said = generate(model, rows, known, *args, **kw)
        calls.append((rows.tolist(), known.tolist(), said))
        return said
    monkeypatch.setattr(ex, "generate", watched)
    ex.main()
    assert len(calls) > 1
    for (_, _, said), (rows, known, _) in zip(calls, calls[1:]):
        assert known == [said[r][-1] for r in rows]
    assert any(said[r][-1] != said[r - 2][-1] for _, _, said in calls[:-1] for r in (2, 3))   # (it does matter)
