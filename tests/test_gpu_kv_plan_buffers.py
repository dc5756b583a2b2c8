"""kv_plan with buffers that its caller keeps."""
import pytest
import torch

from block_planner_amd import api
from block_planner_amd import binding as B

pytestmark = pytest.mark.gpu


def test_two_sets_of_buffers_in_turn():
    """Steps planned into two sets in turn equal steps with buffers of their own;
    one set alone is refused, with nothing changed."""
    R, T, pages = 3, 40, 30
    ints = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    q_len, free = ints(30, 1, 9), torch.arange(pages, dtype=torch.int32, device="cuda")
    state = [[ints(0, 0, 0), ints(0, 0, 0), ints(pages), torch.full((R, 12), -1, dtype=torch.int32, device="cuda")]
             for _ in range(2)]
    sets = [api.kv_step(R, T, "cuda") for _ in range(2)]
    for i in range(20):
        steps = []
        for s, out in zip(state, (None, sets[i % 2])):
            steps.append(api.kv_plan(q_len, s[0], s[1], s[3], free, s[2], T, out=out))
            s[:3] = [steps[-1].kv_len, steps[-1].owned, steps[-1].status[:1]]
        assert all(torch.equal(a, b) for a, b in zip(*steps)) and torch.equal(state[0][3], state[1][3]), i
    assert state[0][0].tolist() == [600, 20, 180] and int(steps[0].status[0]) == pages - 10 - 1 - 3
    before = [t.clone() for t in (*steps[1], state[1][3])]
    with pytest.raises(B.HTError) as e:
        api.kv_plan(q_len, state[1][0], state[1][1], state[1][3], free, state[1][2], T, out=steps[1])
    assert e.value.code == 1
    assert all(torch.equal(a, b) for a, b in zip(before, (*steps[1], state[1][3])))
