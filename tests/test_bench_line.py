"""The benchmark's JSON line: floats to the digits a run resolves, and configs
brief enough that the whole line is kept where a run's last 8,000 characters are."""
import json

import bench

THIRD = 1 / 3


def call(*more):
    keys = ("ms", "us_graph", "us_eager", "us_graph_cold", "tokens_per_s", "GBs", "hbm_frac", "slot_frac") + more
    return dict({k: 1000 * THIRD for k in keys}, bytes=1 << 32, note="what it is, in a sentence of some length " * 6)


def inference():
    return dict({k: call() for k in ("step", "prefill", "block_step", "commit", "baseline_full_scan")}, workload="infer_262k_b16",
                batch=16, d_inner=2048, d_state=16, ctx=262144, block=16, denoising_steps=16, n_blocks=8, launch="graph",
                generation_tokens_per_s=1e6 * THIRD, worst_rel_err=THIRD,
                max_rel_err={"output %d" % i: {"rel": THIRD, "norm": THIRD, "bar": 0.02} for i in range(17)},
                cpu_baseline_sampled=call())


def training():
    r = inference()
    return dict(r, seq=4096, **{k: call() for k in (
        "train_scan", "train_scan_blocks", "train_scan_bwd", "train_scan_blocks_bwd", "all_block_step", "full_scan")})


def test_short_keeps_values():
    x = {"a": 1.2345678901234567, "b": [0.1, 3, True, None, "s"], "c": {"d": 123456789.123, "e": 1e-30}}
    y = bench.short(x)
    assert y["b"] == [0.1, 3, True, None, "s"] and y["a"] == 1.234568 and y["c"]["e"] == 1e-30
    assert abs(y["c"]["d"] / x["c"]["d"] - 1) < 1e-6


def test_configs_are_brief():
    got = {n: bench.config_brief(training() if n.startswith("train") else inference()) for n in bench.CONFIG_WORKLOADS}
    assert len(json.dumps(got)) < 3500                 # the rest of the line takes 4,700
    one = got["infer_65k_b1"]
    assert one["step"]["ms"] == 333.3 and one["worst_rel_err"] == 0.3333 and "max_rel_err" not in one
    assert got["train_87m"]["all_block_step"]["slot_frac"] == 333.3
    r = inference()
    del r["baseline_full_scan"], r["worst_rel_err"]
    assert "baseline_full_scan" not in bench.config_brief(r)


def test_details_on_demand():
    assert bench.config_summary(inference())["max_rel_err"] == inference()["max_rel_err"]
    assert bench.config_summary(training())["cpu_baseline_sampled"] == call()
