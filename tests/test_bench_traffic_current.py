"""The committed DRAM-traffic table belongs to the committed kernels: bench.py reports its figures (CPU only).

A change of gemv.cu, mma.cu, common.cuh or internal.h needs the table's captures taken again (each entry has its
command); until then the bench's roofline objects would have no traffic."""
import importlib.util
import json
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("workload,stages", [("decode", ("gemv_gate_up", "gemv_down"))] +
                         [(w, ("mma_gate_up", "mma_down")) for w in ("zipf", "prefill", "sweep_t7234")])
def test_every_entry_is_reported(workload, stages):
    spec = importlib.util.spec_from_file_location("bench_traffic_now", os.path.join(ROOT, "bench.py"))
    bench = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(bench)
    table = json.load(open(os.path.join(ROOT, "profiles", "ncu_traffic.json")))
    for stage in stages:
        assert bench.ncu_traffic(workload, stage) == table[workload][stage]["dram_bytes_per_launch"]
