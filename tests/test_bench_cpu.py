"""What bench.py reports for each operation, with the measurement itself replaced: the bytes of the
timed call are the operation's own."""
import json

import pytest

import bench

TIMED = {"ms": 5.0, "seg_us": [400.0], "e2e": None, "clocks": None, "launches_per_step": 2, "n_sets": 3,
         "chunk": 1, "per_set_bytes": 1 << 20}
KERNEL = {"layer": "attention_layer", "reduce": "state_reduce", "apply": "apply", "backward": "attention_backward",
          "causal": "causal_attention", "tconv": "temporal_conv"}


def _report(monkeypatch, capsys, op, **more):
    timed = dict(TIMED, kernel_names=(KERNEL.get(op, op),), **more)
    for name in ("run_la", "run_tconv", "run_block_op"):
        monkeypatch.setattr(bench, name, lambda *a: timed)
    monkeypatch.setattr("sys.argv", ["bench.py", "--op", op, "--steps", "10", "--cpu-seconds", "0"])
    monkeypatch.delenv("WORLD_SIZE", raising=False)
    monkeypatch.delenv("RANK", raising=False)
    bench.main()
    return json.loads(capsys.readouterr().out)


@pytest.mark.parametrize("op", sorted(KERNEL))
def test_bytes_of_the_layers_own_operations(monkeypatch, capsys, op):
    w = bench.wl.WORKLOADS[bench.DEFAULT_WORKLOAD]
    want = 2 << 20 if op == "tconv" else bench.layer_bytes(w)[KERNEL[op]]
    roof = _report(monkeypatch, capsys, op)["roofline"]
    assert roof["kernel"] == KERNEL[op] and roof["algorithmic_bytes"] == want > 0
    assert roof["achieved"] > 0 and roof["frac"] > 0


@pytest.mark.parametrize("op", sorted(bench.BLOCK_OPS))
def test_bytes_of_the_block_operators(monkeypatch, capsys, op):
    roof = _report(monkeypatch, capsys, op, op_bytes=123456789)["roofline"]
    assert roof["kernel"] == op and roof["algorithmic_bytes"] == 123456789
