"""Infinite penalties and biases (GPU): they reach the tokens that they are
for, and leave the others as they were."""
import numpy as np
import pytest

from oracle import logit_rules as lr
from tests.test_gpu_logit_rules import check_verify, dev, device_rules, make, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    from int4_output_head_amd import binding
    return binding


@pytest.mark.parametrize("bias", [0, 5, 2100])
@pytest.mark.parametrize("name,value", [("frequency", np.inf), ("frequency", -np.inf), ("presence", np.inf),
                                        ("presence", -np.inf), ("repetition", np.inf)])
def test_infinite_penalties(b, name, value, bias):
    R, T, V = 3, 4, 3000
    logits, rules, drafts = make(R, T, V, 5, bias=bias, mask=None)
    rules["n_prompt"][:] = (10, 40, 10 ** 6)           # tokens of the prompt alone, and a request with no others
    rules[name][:] = value
    want = lr.ruled(logits, rules, drafts, R, T)
    if name != "repetition":
        assert not np.isnan(want).any()
        # what was generated, and what was not
        for i in range(R):
            seen, made = lr.counts(rules, drafts, i, T - 1, V)
            row = want[i * T + T - 1]
            assert np.all(row[made > 0] == -value) and np.isfinite(row[made == 0]).all()
            assert i == R // 2 or (seen & (made == 0)).any()       # (that request has no history)
    r, d = device_rules(b, rules), dev(drafts)
    same(b.apply_logit_rules(dev(logits), r, d, R=R), want)
    check_verify(b.verify_logits(dev(logits), r, d, R=R, top_k=6), want, drafts, None, None, R, T, 6, 1.0, False)


def test_infinite_biases(b):
    R, T, V = 2, 3, 2000
    logits, rules, drafts = make(R, T, V, 8, bias=40, mask=None)
    rules["bias_values"][::2], rules["bias_values"][1::2] = -np.inf, np.inf
    want = lr.ruled(logits, rules, drafts, R, T)
    r, d = device_rules(b, rules), dev(drafts)
    same(b.apply_logit_rules(dev(logits), r, d, R=R), want)
    check_verify(b.verify_logits(dev(logits), r, d, R=R, top_k=16), want, drafts, None, None, R, T, 16, 1.0, False)
