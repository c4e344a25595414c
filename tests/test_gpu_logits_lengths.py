"""History and prompt lengths of the logits processing at and beyond their ends."""
import numpy as np
import pytest

from speculative_tree_verify_mla_b200 import kdv
from tests.test_gpu_logits import Problem, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompt,err,means", [(50, 0, 50), (51, kdv.KDV_DERR_BAD_LENGTH, 50), (2 ** 31 - 1, kdv.KDV_DERR_BAD_LENGTH, 50),
                                              (-1, kdv.KDV_DERR_BAD_LENGTH, 0), (0, 0, 0)])
def test_prompt_lengths_outside_the_history(prompt, err, means):
    """A prompt length outside [0, hist_ld] is reported and taken as the end next to it."""
    p = Problem(30, [4, 3], 2000, [50, 50])
    kdv.kdv_logits_process(p.params(prompt_len=i32([prompt, 20])))
    assert p.err.item() == err
    p.prompt_len = np.array([means, 20])
    p.check()


def test_a_prompt_beyond_the_tokens_that_are_there():
    """hist_len < prompt_len <= hist_ld: the whole history is prompt, and nothing is reported."""
    p = Problem(31, [4], 2000, [50])
    p.hist_len = np.array([30])
    kdv.kdv_logits_process(p.params(prompt_len=i32([45])))
    assert p.err.item() == 0
    p.prompt_len = np.array([30])
    p.check()
