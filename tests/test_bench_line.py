"""The benchmark's result is one line that is short enough to be read whole;
its details are another, on stderr."""
import json

import bench


def test_the_result_is_one_short_line(capsys):
    point = {"kernel": "qmm_dmma_kernel", "us": 21.2, "TOPS": 25.3, "frac_of_bf16_peak": 0.0133, "weight_GBps": 840.7, "bound": "hbm"}
    line = {"metric": bench.METRIC, "value": 3926.0, "unit": "GB/s", "n_gpus": 1, "steps": 20, "warmup": 5, "ms_per_step": 6.2,
            "config": {"workload": bench.WORKLOAD}, "e2e": {"value": 1.0}, "gpu_launches": 3840, "clocks": {"sm_mhz": 2070.0, "reasons": []},
            "sweep_GBps": {f"{t}/{m}/M{M}": 3959.1 for t in bench.TYPES for m in bench.MODES for M in bench.MS}}
    details = {"prefill_points": {f"q8_0/int8_act/M{i}/14336x4096": point for i in range(64)}, "small_configs": {str(i): point for i in range(20)},
               "next_types": {}, "oracle_configs": None, "dequantize_all": point}
    bench.emit({**line, **details})
    out, err = capsys.readouterr()
    assert out.count("\n") == 1 and len(out) < 3000 and json.loads(out) == line
    assert err.count("\n") == 1 and json.loads(err) == details
