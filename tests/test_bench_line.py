"""The benchmark's record stays a line that readers of a log's end can take whole: rounded
figures, records of one kind as columns."""
import json
import math

import bench


def test_short_keeps_five_digits_and_everything_else():
    v = {"a": 56.937904759100164, "b": [1, True, None, "x", 1e-9 / 3], "c": (2.0, {"d": 123456.7})}
    s = bench.short(v)
    assert s == {"a": 56.938, "b": [1, True, None, "x", 3.3333e-10], "c": [2.0, {"d": 123460.0}]}
    assert s["b"][1] is True and math.isinf(bench.short(math.inf))
    assert json.loads(json.dumps(s)) == s


def test_columns_hold_every_value():
    rows = [{"M": 1, "us": 2.5, "stages": 2}, {"M": 8, "us": 3.5, "splits": 4}]
    assert bench.columns(rows) == {"M": [1, 8], "us": [2.5, 3.5], "stages": [2, None],
                                   "splits": [None, 4]}
    assert bench.columns([]) == {}
