"""What the bench prints (no GPU): the headline is one short JSON line on
stdout, and the secondary shapes are not in its way."""

import json

import bench


def test_headline_is_one_short_line(capsys):
    line = {"metric": bench.METRIC, "value": 1.5, "unit": bench.UNIT, "e2e": {"value": 1.0}}
    shapes = {"groups": {"x": {"calls": [{"us": i / 3} for i in range(3000)]}}}
    bench._emit(line, shapes)
    out, err = capsys.readouterr()
    assert out.count("\n") == 1 and json.loads(out) == line
    assert json.loads(err) == {"shapes": shapes}
    bench._emit(line, None)
    out, err = capsys.readouterr()
    assert json.loads(out) == line and err == ""
