"""Host side of the audited loss (no GPU): which backward pass may be compared
with which stored row."""
import pytest
import torch

from silent_corruption_detection_amd import recompute
from silent_corruption_detection_amd.recompute import RecomputeAudit


@pytest.fixture
def audit(monkeypatch):
    """An audit on the CPU whose losses are the backward pass' question for its rows."""
    monkeypatch.setattr(recompute, "linear_cross_entropy",
                        lambda x, w, target, reduction, row, checked: checked)
    return RecomputeAudit(2, device="cpu", outputs=2)


def test_a_backward_pass_of_its_own_step(audit):
    audit.begin_step()
    a, b = (audit.cross_entropy(k, None, None, None) for k in range(2))
    for k, backward in ((1, b), (0, a)):
        args = backward()
        assert args["row"].data_ptr() == audit.recomputed[2 * k].data_ptr()
        assert args["ref"].data_ptr() == audit.original[2 * k].data_ptr()
        assert args["mismatch"].data_ptr() == audit.mismatch[k].data_ptr()
    with pytest.raises(RuntimeError, match="ran again"):
        a()
    assert audit.calls == [2, 2]


def test_a_backward_pass_of_an_earlier_step_is_refused(audit):
    """Two steps in flight: the earlier one's row is gone, and comparing its logits with
    the later one's would report a corruption that is none."""
    audit.begin_step()
    first = audit.cross_entropy(0, None, None, None)
    audit.begin_step()
    with pytest.raises(RuntimeError, match="an earlier step"):
        first()
    second = audit.cross_entropy(0, None, None, None)
    with pytest.raises(RuntimeError, match="an earlier step"):
        first()
    assert audit.calls == [1, 0]
    second()
    with pytest.raises(RuntimeError, match="an earlier step"):
        first()
    assert audit.calls == [2, 0]


def test_a_segment_runs_once_in_a_step(audit):
    audit.begin_step()
    audit.cross_entropy(1, None, None, None)
    with pytest.raises(RuntimeError, match="begin_step"):
        audit.cross_entropy(1, None, None, None)
    for k in (-1, 2):
        with pytest.raises(IndexError):
            audit.cross_entropy(k, None, None, None)
