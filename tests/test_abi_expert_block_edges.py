"""Edges of the norm, the routing with groups and the 4-bit operators that need no GPU."""
import ctypes

import pytest
import torch

import group_sparse_swiglu_amd as E

P = 64  # an aligned, never dereferenced address
NULL = None


def _caller(f, names, ok):
    return lambda **kw: f(*[kw.get(n, v) for n, v in zip(names, ok)])


def test_products_by_expert_of_no_rows():
    """Without rows in a nothing of it is read, and an empty tensor's address is NULL."""
    names = ("a", "sa", "R", "rows", "b", "sb", "E", "off", "dt", "M", "N", "K", "y", "ws", "bytes", "stream")
    call = _caller(E.lib().esg_mxfp4_grouped_matmul, names, (P, P, 9, P, P, P, 3, P, 1, 12288, 4096, 64, P, NULL, 0, NULL))
    assert call() == 3                                     # all is well but the workspace
    assert call(R=0, a=NULL, sa=NULL) == 3 and call(R=0) == 3
    assert call(a=NULL) == 1 and call(sa=NULL) == 1
    assert call(R=0, rows=NULL) == 1 and call(R=0, a=P + 8) == 1
