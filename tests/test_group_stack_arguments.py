"""What model.GCNStack accepts as a batch of graphs, on the host: nothing is
launched."""
import pytest
import torch

N = 50


@pytest.fixture
def make():
    import quantized_gnn_message_gb300 as q
    from quantized_gnn_message_gb300 import build, model
    build.build()
    c = q.Graph_t()
    c.n = N
    empty = torch.empty(0, dtype=torch.int32)
    g = q.Graph(N, 0, empty, empty, empty, c)
    return q.GQError, lambda **kw: model.GCNStack(g, (8, 8, 8), None, device="cpu", **kw)


@pytest.mark.parametrize("ptr", [[0, 20, 40], [5, 50], [0, 51], [0, 30, 20, 50], [-1, 50], [0, 60, 50], [50], [0],
                                 [0, 50, 20]])
def test_nodes_outside_every_graph_are_refused(make, ptr):
    """They would not be normalized: no kernel writes their features."""
    err, stack = make
    with pytest.raises(err):
        stack(norm="group", ptr=torch.tensor(ptr))


@pytest.mark.parametrize("ptr", [[0, 50], [0, 0, 20, 20, 50, 50], None])
def test_offsets_over_all_nodes_are_taken(make, ptr):
    _, stack = make
    m = stack(norm="group", groups=4, ptr=None if ptr is None else torch.tensor(ptr))
    assert m.mean[0].shape == ((len(ptr) - 1) if ptr else 1, 4)


def test_offsets_elsewhere_are_refused(make):
    err, stack = make
    with pytest.raises(err):
        stack(norm="group", ptr=torch.zeros(2, dtype=torch.int64, device="meta"))


@pytest.mark.parametrize("kw", [dict(groups=0), dict(groups=-4), dict(groups=3), dict(max_rows=-1)])
def test_group_arguments(make, kw):
    err, stack = make
    with pytest.raises(err):
        stack(norm="group", **kw)


def test_no_normalization_may_be_none(make):
    """As it could be before there were two kinds of it."""
    _, stack = make
    assert stack(norm=None).norm is False
