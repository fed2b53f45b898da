"""The operators of a beam search together: rotated appends, attention over the
cache, selection, reordered pages (examples/beam_search.py)."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import test_activation_aware_amd as ttq  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("tokens,beams,steps", [(100, 4, 20), (33, 1, 5), (150, 7, 12)])
def test_beams_score_what_their_tokens_score(bits, tokens, beams, steps):
    """Each beam's tokens, continued alone from the prompt that was kept, one at a time, add up to the beam's score: the
    pages that the beams were left with are those of their histories.  What may differ is the order in which the rows of
    a step are summed in the projections: some 2^-11 of logits of about 10, step after step."""
    import beam_search
    said = []
    r = beam_search.run(tokens, beams, steps, bits, show=said.append)
    model = r["model"]
    assert len(said) == beams + 2 and (r["shared"] > 0 or beams == 1)
    history, scores = r["history"], r["scores"]
    assert history.shape == (beams, steps) and bool((scores[:-1] >= scores[1:]).all())
    assert len({tuple(h) for h in history.tolist()}) == beams
    for b in range(beams):
        model.cache.fork("kept", ["alone"])
        total = 0.0
        logits = r["first"]
        for t in range(steps):
            now = history[b, t:t + 1]
            total += float(ttq.ttq_token_logprobs(logits, now)[0])
            logits = model.step(["alone"], now)
        model.cache.free("alone")
        assert abs(total - float(scores[b])) <= 0.02 * steps
