"""Matrices that the wrappers of the product refuse: rows that share memory or run
backwards have no leading dimension, and read as rows of their full length they
would end outside the memory that is there.  (No device needed.)"""
import numpy as np
import pytest

import dense_fp32_sgemm_gb300 as sg


def test_host_matrices():
    a, b, c = np.ones((4, 8), np.float32), np.ones((8, 6), np.float32), np.ones((4, 6), np.float32)
    flat = np.ones(64, np.float32)
    overlapping = np.lib.stride_tricks.as_strided(flat, (4, 8), (12, 4))
    for bad in (np.broadcast_to(a[:1], (4, 8)), a[::-1], overlapping):
        with pytest.raises(ValueError, match="A has overlapping rows"):
            sg.run_host(bad, b, c)
    with pytest.raises(ValueError, match="B has overlapping rows"):
        sg.run_host(a, np.broadcast_to(b[:1], (8, 6)), c)
    with pytest.raises(ValueError, match="C has overlapping rows"):
        sg.run_host(a, b, np.broadcast_to(c[:1], (4, 6)))
    with pytest.raises(ValueError, match="whole number of elements"):
        sg.run_host(np.lib.stride_tricks.as_strided(flat, (4, 8), (34, 4)), b, c)


def test_torch_matrices():
    torch = pytest.importorskip("torch")
    one = torch.ones(1, 8)
    for bad in (one.expand(4, 8), torch.ones(64).as_strided((4, 8), (7, 1)), torch.ones(1, 1).expand(3, 1)):
        with pytest.raises(ValueError, match="A has overlapping rows"):
            sg._matrix_args(bad, "A")
    assert sg._matrix_args(one, "A")[1] == 8
    assert sg._matrix_args(torch.ones(4, 12)[:, :8], "A")[1] == 12
    assert sg._matrix_args(one.expand(1, 8), "A")[1] == 8
    assert sg._matrix_args(torch.ones(3, 0), "A")[1] == 1
    assert sg._matrix_args(torch.ones(64).as_strided((1, 8), (3, 1)), "A")[1] == 8
    assert sg._matrix_args(torch.ones(8, 4).t()[:, :1], "A")[1] == 1
