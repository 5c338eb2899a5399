"""The rows of the sampling and verification tests lie clear of their borders: a test that compares decided rows alone says
how many it did compare."""
import pytest

import test_sample
import test_verify

pytestmark = pytest.mark.gpu


class Counted:
    """check() of a module of tests, with the rows that it got and those that it left out."""

    def __init__(self, module, monkeypatch):
        self.check, self.rows, self.left_out = module.check, 0, 0
        monkeypatch.setattr(module, "check", self)

    def __call__(self, x, *args, **kwargs):
        n = self.check(x, *args, **kwargs)
        self.rows += len(x)
        self.left_out += n
        return n


@pytest.mark.parametrize("test,cases", [
    ("test_larger_rows", [()]),
    ("test_candidate_lists", [(n, d) for n in (1, 2, 31, 32, 33, 63, 64) for d in ("bf16", "fp32")]),
    ("test_long_lists_with_ids", [()]),
    ("test_rows_of_a_wider_matrix", [(*c, d) for c in ((2050, 2051, 1), (64, 67, 3), (30000, 30001, 1), (151, 500, 7))
                                     for d in ("bf16", "fp32")]),
    ("test_a_group_full_of_the_best", [()]),
    ("test_another_stream_and_a_captured_call", [()]),
])
def test_sampling(test, cases, monkeypatch):
    counted = Counted(test_sample, monkeypatch)
    for case in cases:
        getattr(test_sample, test)(*case)
    assert counted.rows >= 10 and counted.left_out <= counted.rows // 20


def test_verification_of_a_wider_tensor(monkeypatch):
    counted = Counted(test_verify, monkeypatch)
    test_verify.test_rows_of_a_wider_tensor_another_stream_and_replays()
    assert counted.rows >= 20 and counted.left_out <= counted.rows // 10
