"""Hand cases that pin the plain forms of the norm, the linear layer and the
rules on logits (CPU)."""
import numpy as np
import pytest

from int4_output_head_amd import synth
from oracle import logit_rules as lr
from oracle import rows


def test_norm_by_hand():
    # mean square (9 + 16) / 2 = 12.5
    y = rows.norm64([[3.0, 4.0]], [1.0, 2.0], eps=0.0)
    assert np.allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]], rtol=1e-15)
    assert np.allclose(rows.norm64([[1.0, 4.0]], [1.0, 2.0], residual=[[2.0, 0.0]], eps=0.0), y, rtol=1e-15)


def test_codes_by_hand():
    # peak 2: step 2 / 127; 1 -> 63.5 -> 64 (half to even), -2 -> -127
    c = rows.codes32([[1.0, -2.0, 0.0, 1 / 254.0]])
    assert c.tolist() == [[64, -127, 0, 0]]
    assert rows.codes32([[0.0, 0.0]]).tolist() == [[0, 0]]
    assert rows.codes32([[np.nan, 1.0], [np.inf, 1.0], [1e-38, 0.0]]).tolist() == [[0, 0]] * 3


def test_unpack_inverts_pack():
    q = np.random.default_rng(0).integers(-7, 8, (5, 64)).astype(np.int8)
    assert np.array_equal(rows.unpack_int4(synth.pack_int4(q)), q)


def test_linear_by_hand():
    packed = synth.pack_int4(np.array([[1, -7] + [0] * 30, [2, 3] + [0] * 30], np.int8))
    codes = np.zeros((1, 32), np.int8)
    codes[0, :2] = (10, -3)
    z, y, s = rows.linear64(codes, [0.5], packed, out_scales=[2.0, 1.0], bias=[1.0, -8.0], activation="relu",
                            residual=[[0.25, 0.5]])
    assert s.tolist() == [[31.0, 5.5]] and y.tolist() == [[32.0, -2.5]] and z.tolist() == [[32.25, 0.5]]
    assert rows.activate64(np.array([0.0]), "gelu")[0] == 0.0
    assert abs(rows.activate64(np.array([1.0]), "gelu")[0] - 0.8413447460685429) < 1e-15
    assert abs(rows.activate64(np.array([1.0]), "silu")[0] - 0.7310585786300049) < 1e-15


def test_rules_by_hand():
    logits = np.array([[2.0, -2.0, 1.0, 4.0, 0.5], [2.0, -2.0, 1.0, 4.0, 0.5]], np.float32)
    rules = dict(history=np.array([0, 1, 1, 7, -3]), history_offsets=np.array([0, 5]), n_prompt=np.array([2]),
                 repetition=np.array([2.0]), frequency=np.array([0.25]), presence=np.array([0.5]),
                 bias_ids=np.array([2, 3, 2, 9]), bias_values=np.array([100.0, 1.0, 8.0, 1.0]),
                 bias_offsets=np.array([0, 4]), mask=np.array([[0b01111], [0b11111]], np.uint32))
    x = lr.ruled(logits, rules, [[2]], 1, 2)
    # row 0: token 0 only in the prompt; 1 in the prompt and once generated
    assert x[0].tolist() == [1.0, -4.0 - 0.25 - 0.5, 1.0 + 8.0, 5.0, -np.inf]
    # row 1 also counts draft 2 as generated
    assert x[1].tolist() == [1.0, -4.75, 0.5 - 0.25 - 0.5 + 8.0, 5.0, 0.5]


def test_top_and_probability_by_hand():
    row = np.array([1.0, np.nan, 3.0, 3.0, -np.inf], np.float32)
    assert lr.top(row, 4)[0].tolist() == [2, 3, 0, -1]
    assert lr.top(row, 4)[1].tolist() == [3.0, 3.0, 1.0, -np.inf]
    e = np.exp(-2.0)
    assert lr.probability64(row, 0, 1.0, 0) == pytest.approx(e / (2 + e), rel=1e-15)
    assert lr.probability64(row, 0, 1.0, 2) == 0.0
    assert lr.probability64(row, 3, 1.0, 2) == 0.5
    assert lr.probability64(row, 4, 1.0, 0) == 0.0
    assert lr.lse64(row, 2.0) == pytest.approx(np.log(2 * np.exp(1.5) + np.exp(0.5)), rel=1e-15)
    assert lr.lse64(np.full(3, -np.inf), 1.0) == -np.inf
