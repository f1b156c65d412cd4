"""examples/speculative_decode.py: that it runs, that what a step keeps is what the model over the whole text says,
that a forked request goes on as its source does, and that no page is lost.

Tolerance: as for the decode step's example, a value next to a rounding may come out one step of bf16 or one code
away where the order of the sums differs; a token taken greedily from a tree is within that of the largest logit of
the text run token by token.  (The layer's last norm divides by the sums of a row; a hundred of its 256 codes one
step off move a logit by 10 of 256^0.5 * 36 parts of its standard deviation, its largest of 400 by 4 times that.)
"""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))


def example():
    import speculative_decode
    return speculative_decode


def start(ex, n=3, length=21, requests=6):
    model = ex.Model(requests=requests)
    rows = torch.arange(n, device="cuda")
    prompt = torch.randint(0, model.vocab, (n, length), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    return model, rows, prompt, model.prompt(rows, prompt)


@pytest.mark.gpu
def test_it_runs():
    ex = example()
    ex.main()


@pytest.mark.gpu
def test_greedy_trees_say_what_the_model_says():
    ex = example()
    model, rows, prompt, known = start(ex)
    g = torch.Generator(device="cuda").manual_seed(7)
    said = ex.generate(model, rows, known, 8, g, drawn=False, temperature=0.0)
    assert all(len(t) >= 8 for t in said) and sum(len(t) for t in said) > 24     # some drafts were kept
    lens = model.lens.tolist()
    for r in range(3):
        assert lens[r] == 20 + len(said[r])            # all but the last token known
        text = torch.cat((prompt[r], torch.tensor(said[r], device="cuda"))).unsqueeze(0)
        other = ex.Model(requests=1)
        row = torch.arange(1, device="cuda")
        other.take(torch.full((1,), text.shape[1], dtype=torch.int32, device="cuda"))
        logits = other.forward(row, text[:, :60])[0]
        n = min(len(said[r]), 60 - 21)
        at = torch.arange(20, 20 + n, device="cuda")
        took = logits[at, torch.tensor(said[r][:n], device="cuda")]
        assert (took >= logits[at].amax(1) - 0.07 * 4 * logits.std()).all(), r


@pytest.mark.gpu
@pytest.mark.parametrize("drawn", [True, False])
def test_a_forked_request_goes_on_as_its_source(drawn):
    ex = example()
    model, rows, _, known = start(ex)
    model.fork(rows.int(), (rows + 3).int())
    shared = model.refs.max().item()
    assert shared == 2 and (model.table[3:, 0] == model.table[:3, 0]).all() and (model.table[3:, 1] != model.table[:3, 1]).all()
    both = torch.arange(6, device="cuda")
    known = known.repeat(2)
    for i in range(6):
        u = torch.rand((3, 16), device="cuda", generator=torch.Generator(device="cuda").manual_seed(i)).repeat(2, 1)
        new, count = model.step(both, known, u, drawn=drawn, temperature=0.9)
        assert torch.equal(new[:3], new[3:]) and torch.equal(count[:3], count[3:])
        known = new.gather(1, (count - 1).long().unsqueeze(1)).squeeze(1)
    assert torch.equal(model.lens[:3], model.lens[3:])
    held = model.table[model.table >= 0]
    assert torch.equal(torch.bincount(held, minlength=64), model.refs.clamp(min=0).long())    # every holder counted
    model.free(both.int())
    assert not model.refs.any() and (model.table == -1).all()
