"""The benchmark's line is short enough to be kept whole; its tables go to stderr
when they would make it too long (no GPU needed)."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
import bench   # noqa: E402


def emitted(capsys, line):
    bench.emit(line)
    out, err = capsys.readouterr()
    assert out.endswith("\n") and out.count("\n") == 1 and len(out) <= bench.LINE_LIMIT + 1
    tables = {}
    for t in err.splitlines():
        tables.update(json.loads(t))
    return json.loads(out), tables


def test_long_tables_go_to_stderr(capsys):
    line = {"metric": "m", "value": 1.5, "unit": "TFLOP/s", "config": {"M": 2048}, "e2e": {"value": 1.0},
            "m1": {"value": 2.0}, "mlx4": {"x": "y" * 300}, "attention": {"x": "y" * 1300},
            "configs": {"c%d" % i: {"us": i, "note": "n" * 400} for i in range(45)}}
    got, tables = emitted(capsys, dict(line))
    assert set(tables) == {"configs"} and {**got, **tables} == line
    line["attention"]["x"] *= 3   # still too long without the first
    got, tables = emitted(capsys, dict(line))
    assert set(tables) == {"configs", "attention"} and {**got, **tables} == line


def test_short_line_is_whole(capsys):
    line = {"metric": "m", "value": 1.5, "m1": {"value": 2.0}, "configs": None}
    assert emitted(capsys, dict(line)) == (line, {})
