"""The bounds of the attention tests with coded values are narrow enough: any
key that is left out exceeds them."""
import pytest
import torch

from attention_values import CASES, coded, reference


@pytest.mark.parametrize("name", CASES)
def test_a_lost_key_shows(name):
    lens, heads, page, window, sinks = CASES[name]
    p = coded(lens, *heads, page=page, seed=50)
    _, _, margin = reference(p, heads[2] ** -0.5, window, sinks, 2.0 ** -8, torch.bfloat16)
    assert margin > 1.25, margin
