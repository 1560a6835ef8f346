"""What bench.py says bounds a step."""
import bench

PEAKS = {"bf16_tflops": 1916.2, "bf16_tflops_sustained": 1716.3, "hbm_gbs": 6789.0}


def test_a_step_of_the_forward_is_bound_by_the_tensor_cores():
    # HunyuanVideo 720p: 24 heads of 128, 119056 queries on as many keys
    n = 119056
    r = bench.roofline(4.0 * 128 * 24 * n * n, 24 * n * (4 * 128 * 2 + 4), 102.6, PEAKS, "measured")
    assert r["bound"] == "tensor" and r["unit"] == "TFLOP/s" and r["peak"] == 1916.2
    assert r["achieved"] == round(4.0 * 128 * 24 * n * n / 102.6 / 1e9, 2)
    assert r["frac"] == round(r["achieved"] / 1916.2, 4) and r["frac_of_sustained"] > r["frac"]


def test_one_token_on_a_cache_is_bound_by_memory():
    # one query of 24 heads of 128 on 119056 keys in e4m3, 0.14 ms
    n = 119056
    nbytes = 24 * (128 * (18 + 2 * n) + 4)
    r = bench.roofline(4.0 * 128 * 24 * n, nbytes, 0.14, PEAKS, "measured")
    assert r["bound"] == "hbm" and r["unit"] == "GB/s" and r["peak"] == 6789.0
    assert r["achieved"] == round(nbytes / 0.14e6, 1) and 0.7 < r["frac"] < 0.8


def test_without_measured_peaks():
    assert bench.roofline(1e12, 1.0, 1.0, {}, "fallback")["peak"] == bench.FALLBACK_BF16_TFLOPS
    assert bench.roofline(1.0, 1e9, 1.0, {}, "fallback")["peak"] == bench.FALLBACK_HBM_GBS
