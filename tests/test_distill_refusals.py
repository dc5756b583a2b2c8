"""nn.distill_loss has a gradient for the student's logits alone: a weight or a
teacher that wants one is refused rather than detached (no GPU: refused before
anything is computed)."""
import pytest
import torch

from block_planner_amd import nn as htnn


def args():
    return torch.randn(3, 50), torch.zeros(3, 4, dtype=torch.int32), torch.randn(3, 4), torch.ones(3)


@pytest.mark.parametrize("student", [True, False])
@pytest.mark.parametrize("which", ["teacher", "weight"])
def test_gradients_of_weight_and_teacher_are_refused(student, which):
    x, ids, teacher, weight = args()
    x.requires_grad_(student)
    (teacher if which == "teacher" else weight).requires_grad_()
    with pytest.raises(RuntimeError, match=f"no gradient for {which}"):
        htnn.distill_loss(x, ids, teacher, weight)
    with pytest.raises(RuntimeError, match=f"no gradient for {which}"):        # of something computed from a leaf
        htnn.distill_loss(x, ids, teacher * 2, weight * 2)


@pytest.mark.gpu
def test_detached_and_without_gradients():
    x, ids, teacher, weight = (t.cuda() for t in args())
    teacher.requires_grad_(), weight.requires_grad_()
    with torch.no_grad():
        want = htnn.distill_loss(x, ids, teacher, weight)
    x.requires_grad_()
    loss = htnn.distill_loss(x, ids, teacher.detach(), weight.detach())
    loss.backward()
    assert loss.item() == pytest.approx(want.item(), rel=1e-5) and torch.isfinite(x.grad).all()
