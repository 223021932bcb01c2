"""Which weights' gradients are summed in pieces of the rows, by the size of the workspace: those that
were measured to gain by it, and none that lose."""
import os

import pytest

import combine_ep_get_03_amd as ep
from combine_ep_get_03_amd import _binding

# E, M, N; rows per expert with which the whole is as fast or faster, and with which pieces are
MEASURED = [(1, 112, 112, (384,), (512, 1024, 4096)), (1, 1000, 816, (), (512, 1024, 4096)),
            (32, 128, 120, (384,), (640, 1024, 4096)), (1, 2048, 1024, (384, 512), (640, 1024, 4096)),
            (1, 1536, 1792, (384,), (1024, 4096)), (96, 128, 256, (384, 1024, 2048), ()),
            (8, 544, 560, (384, 512), (1280, 4096)), (32, 192, 496, (640, 1024), (1408, 4096)),
            (1, 2048, 2048, (640, 1024), (1280, 4096)), (4, 1024, 1024, (384, 640), (1280, 4096))]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(_binding.LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()


@pytest.mark.parametrize("E,M,N,whole,pieces", MEASURED)
def test_pieces_where_they_are_faster(E, M, N, whole, pieces):
    for rows in whole:
        assert ep.ep_expert_weight_grad_workspace_bytes(E, E * rows, M, N) == 0, rows
    for rows in pieces:
        assert ep.ep_expert_weight_grad_workspace_bytes(E, E * rows, M, N) > 0, rows
