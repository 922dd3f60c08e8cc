"""A RouteRule is a plain value: it can be copied, sent to a worker and put into a config."""
from __future__ import annotations

import copy
import dataclasses
import pickle

import pytest

from sparse_moe_layer_row_gb300 import moe_block as mb

RULE = mb.RouteRule(score="sigmoid", n_groups=8, top_groups=4, group_score="top2", renormalize=False, scale=2.5)


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r)),
                                 lambda r: copy.deepcopy({"layers": [r]})["layers"][0],
                                 lambda r: mb.RouteRule(**dataclasses.asdict(r)), dataclasses.replace],
                         ids=["copy", "deepcopy", "pickle", "in a config", "asdict", "replace"])
def test_copies(how):
    r = how(RULE)
    assert r == RULE and hash(r) == hash(RULE) and type(r) is mb.RouteRule
    c = r._c
    assert (c.score, c.n_groups, c.top_groups, c.group_score, c.renormalize, c.scale) == (1, 8, 4, 1, 0, 2.5)
    assert r._ref._obj is r._c          # what a call passes is the copy's own


def test_copies_are_checked():
    with pytest.raises(ValueError):
        dataclasses.replace(RULE, score="argmax")
