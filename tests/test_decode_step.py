"""The decode-step operators together, as examples/decode_step.py runs them: a prompt at once and token
by token, and a drafted tree, have to give the same logits.

Tolerance: the orders of the sums differ, so a value next to a rounding may come out one step of
bf16, and one int8 code, away.  One code of the 512 inputs of the head moves a logit by 1 of
sqrt(512) * 36 = 815 parts of its standard deviation, and a step of the output projection as much;
a row with a hundred such codes, signs at random, moves by 1.3 %, its largest of 2000 logits by 4.5
times that.
"""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))


def near(a, b):
    return (a - b).abs().max() <= 0.06 * a.std()


@pytest.mark.gpu
def test_prompt_at_once_and_token_by_token():
    import decode_step
    whole, single = decode_step.Decoder(), decode_step.Decoder()
    prompt = torch.randint(0, whole.vocab, (whole.batch, 37), device="cuda",
                           generator=torch.Generator(device="cuda").manual_seed(2))
    logits = whole.step(prompt)
    for t in range(prompt.shape[1]):
        one = single.step(prompt[:, t:t + 1])
        single.accept(1)
        assert near(one[:, 0], logits[:, t]), t
    # different adapters, different requests
    assert not near(logits[0], logits[1])


@pytest.mark.gpu
def test_tree_of_drafts():
    import decode_step
    model, plain = decode_step.Decoder(), decode_step.Decoder()
    g = torch.Generator(device="cuda").manual_seed(3)
    prompt = torch.randint(0, model.vocab, (model.batch, 20), device="cuda", generator=g)
    for m in (model, plain):
        m.step(prompt)
        m.accept(20)
    chain = torch.randint(0, model.vocab, (model.batch, 6), device="cuda", generator=g)
    spare = torch.randint(0, model.vocab, (model.batch, 6), device="cuda", generator=g)
    tokens, depth, mask = decode_step.tree_of(chain, spare)
    tree = model.step(tokens, depth, mask)
    want = plain.step(chain)
    assert near(tree[:, 0::2], want)
    for i in range(6):               # each wrong guess after the chain before it
        branch = torch.cat((chain[:, :i], spare[:, i:i + 1]), 1)
        assert near(tree[:, 2 * i + 1], plain.step(branch)[:, -1]), i


@pytest.mark.gpu
def test_sampling_is_reproducible():
    import decode_step
    model = decode_step.Decoder()
    prompt = torch.randint(0, model.vocab, (model.batch, 9), device="cuda",
                           generator=torch.Generator(device="cuda").manual_seed(4))
    logits = model.step(prompt)[:, -1]
    u = torch.rand(model.batch, device="cuda")
    a, b = model.sample(logits, u), model.sample(logits, u)
    assert torch.equal(a, b) and (a >= 0).all() and (a < model.vocab).all()
    greedy = model.sample(logits, u, temperature=0.0)
    assert torch.equal(greedy.long(), logits.argmax(1))
