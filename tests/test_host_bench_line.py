"""The benchmark's printed line: whole and short enough for programs that keep
the last few KB of a run's output, with the metric's fields as measured.
"""
import json

import bench

NAME = "xdma16_tile_bf16_nn_256x256x64_w2x4_s2"


def record():
    x = 1.0 / 3.0
    row = dict(M=8192, N=4096, K=4096, layout="NN", winner=NAME, plan_candidates=193, avg_us=x, rotated_us=x, rotated_copies=16,
               batched_us=x, batched_reps=357, tflops=x, gbs=x, bound="mfma", roofline_frac=x, roofline_frac_resident=x,
               cold_tune_s=x, cold_tune_probes_cached_s=x, frac_of_read_floor=x)
    conf = dict(problem="25088x4096x64 NT", lda=4096, ldb=4096, winner=NAME, plan_candidates=68, candidates_measured=65,
                rotated_us=x, rotated_copies=8, batched_us=x, batched_reps=20, roofline_frac_resident=x, tflops=x, gbs=x,
                bound="mfma", roofline_frac=x, cold_tune_s=x, cold_tune_probes_cached_s=x, warm_call_s=x, out_gbs=x,
                out_frac_of_write_floor=x)
    full = dict(conf, exhaustive=dict(tune_s=x, candidates_timed=65, candidates_failed=0, winner=NAME,
                                      medians_us=[[NAME, x]] * 65))
    served = dict(value=x, unit="TFLOP/s", per_problem=[dict(problem="8192x4096x4096 NN", candidate=NAME, batched_us=x)] * 5)
    rt = dict(process="cold", process_s=x, rows=[dict(size=1024, first_call_ms=x, next20_min_ms=x, winner=NAME,
                                                      first_call=dict(tunes=1))] * 4)
    return dict(metric=bench.METRIC, value=x, unit="TFLOP/s", n_gpus=1, steps=20, warmup=5, ms_per_step=x,
                higher_is_better=True, scaling="weak", vs_baseline=None, dtype="bf16", data="synthetic",
                config=dict(workload=bench.WORKLOAD_TEXT["bf16_m_sweep"], problems=5, tune_mode="adaptive"),
                roofline={"k%d" % i: x for i in range(12)}, cpu_baseline=dict(value=x, sample="s" * 200),
                hbm_read_floor={"k%d" % i: x for i in range(6)}, hbm_write_floor={"k%d" % i: x for i in range(6)},
                cold_tune_s=x, cold_tune_probes_cached_s=x, cold_launches=dict(probe=1000, bench=1000), warm_dispatch_us=x,
                warm_dispatch=dict(method="m" * 200, added_us=x), candidates_in_set=300, per_problem=[row] * 5,
                untuned_default=served, offline=served, rt_tune=dict(sizes=[1, 2], cold=rt, warm=rt),
                configs={n: dict(workload=bench.WORKLOAD_TEXT[n], per_problem=[full] * 2 if n == "bf16_4096" else [conf] * (2 if n == "bf16_decode_nt" else 1))
                         for n in bench.WORKLOAD_TEXT if n not in ("bf16_m_sweep", "bf16_nsplit8")})


def test_the_line_is_whole_and_short():
    r = record()
    text = json.dumps(bench.line_of(r), separators=(",", ":"))
    assert len(text) < 7500 and "\n" not in text
    line = json.loads(text)
    assert line["value"] == r["value"] and line["ms_per_step"] == r["ms_per_step"]
    for k in ("metric", "unit", "n_gpus", "steps", "warmup", "higher_is_better", "scaling", "vs_baseline", "dtype", "data", "config"):
        assert line[k] == r[k]
    assert len(line["per_problem"]) == 5 and line["per_problem"][0]["winner"] == NAME
    assert set(line["configs"]) == set(r["configs"]) and line["configs"]["bf16_4096"][0]["exhaustive"]["candidates_timed"] == 65
    assert "medians_us" in r["configs"]["bf16_4096"]["per_problem"][0]["exhaustive"]  # the record itself is left as it was


def test_parts_that_were_not_run():
    r = dict(record(), configs=None, warm_dispatch=None, warm_dispatch_us=None, rt_tune=None, cpu_baseline=None)
    line = bench.line_of(r)
    assert line["configs"] is None and line["rt_tune"] is None
    r["rt_tune"] = dict(cold=dict(error="exit 1: x"))
    assert bench.line_of(r)["rt_tune"]["cold"] == dict(error="exit 1: x")
