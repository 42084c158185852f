"""bench.py's one JSON line as it is printed by default: short enough to be kept
whole, with every key of the benchmark contract; the details go to stderr."""
import argparse
import json

import bench
import test_bench_cpu


def test_the_printed_line_is_short_and_the_details_are_on_stderr(capsys, monkeypatch):
    monkeypatch.setattr(bench, "time_oracle", lambda cfg: dict(value=53307.1, cores=64, sample="B=1 H=1 T=512, 3 runs"))
    args = argparse.Namespace(workload="layer340m_ctx2k", steps=1000, warmup=10, cpu_baseline=1)
    res = test_bench_cpu._fake_result()
    # the grid of a whole run
    res["long"]["sweep"] = [dict(B=b, T=t, chunked_ms=0.1234567890123, quadratic_ms=0.1234567890123)
                            for b in (1, 4, 16) for t in (1024, 2048, 8192, 32768, 131072)]
    bench.report(args, res, 0.116, 11.0, 1, brief=True)
    out, err = capsys.readouterr()
    assert len(out.strip().splitlines()) == 1 and len(out) < 3000
    line = json.loads(out)
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling",
                "vs_baseline", "dtype", "data", "config", "roofline", "e2e", "gpu_launches", "clocks", "paths",
                "cpu_baseline"):
        assert key in line, key
    assert line["value"] == 8 * 2048 / 0.116e-3 and 0 < line["roofline"]["frac"] < 1
    detail = json.loads(err.split("detail: ", 1)[1])
    assert {"mg", "train", "long_ctx"} <= set(detail) and detail["roofline"]["points"]
    assert all(detail[k] == line[k] for k in line if k != "roofline")


def test_the_traffic_reported_is_that_of_the_present_sources():
    """None once a source of the flash kernel has changed: the capture is then to be taken again."""
    assert bench.flash_traffic("layer340m_ctx2k") == bench.FLASH_TRAFFIC_BYTES
    assert bench.flash_traffic("another") is None
