"""The routing oracle's order of values that fp64 cannot tell apart."""
import numpy as np

from oracle.routing import Rule, route_by


def test_equal_biases_leave_the_order_of_the_logits():
    x = np.array([[40.0, 45.0, 41.0, 39.0]])  # sigmoids of 1
    for bias in (0.0, 1e9):
        assert route_by(Rule("sigmoid", np.full(4, bias)), x, 3)[0].tolist() == [[1, 2, 0]]
        assert route_by(Rule("sigmoid", np.full(4, bias), groups=2, top_groups=1), x, 2)[0].tolist() == [[1, 0]]
    x = np.array([[40.0, 39.0, 41.0, 45.0]])
    assert route_by(Rule("sigmoid", np.zeros(4), groups=2, top_groups=1), x, 2)[0].tolist() == [[3, 2]]
    assert route_by(Rule("sigmoid", np.zeros(4), groups=2, top_groups=1, group_top=2), x, 2)[0].tolist() == [[0, 1]]  # 2 and 2


def test_values_without_a_number_go_by_the_expert():
    x = np.array([[1.0, 2.0, 3.0, np.nan, 0.5]])
    bias = np.array([-np.inf, -np.inf, np.nan, 0.0, -1.0])
    assert route_by(Rule("sigmoid", bias), x, 4)[0].tolist() == [[3, 4, 0, 1]]
    assert route_by(Rule(), x, 5)[0].tolist() == [[2, 1, 0, 4, 3]]
