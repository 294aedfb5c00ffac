"""The example's block-scaled layer against the same layer over whole sequences, part by part and
request by request: bounds that a part which is missing or wrong cannot meet."""
import pytest

from tests.test_gqa_block_layer_gpu import example  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,steps", [((37, 400, 1, 129), 20), ((1, 1, 30), 6), ((37, 300), 2)])
def test_layer_part_by_part(example, lens, steps):  # noqa: F811
    # An e4m3 value is off by 2^-3 / sqrt(12) = 0.036 of its binade (root mean square); a row's values
    # add as much of the row's size, and its weights, whose scores are off by 0.036 (unit queries and
    # keys), as much again: 0.051, twice that allowed.  (Nothing at all would be 1.)  A first prompt's
    # rows come from bf16 keys and values.
    errors = example.block_errors(lens, steps)
    assert {part for part, _ in errors} == {"prompt", "prefix", "decode"}
    assert {b for _, b in errors} == set(range(len(lens)))
    for key, (_, error) in errors.items():
        assert error <= (2.0 ** -6 if key[0] == "prompt" else 0.1), key
