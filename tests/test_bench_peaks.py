"""bench.py's peak for the inference sweeps (no GPU)."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402

P = 1600.0


def test_bf16_sweep_is_measured_against_twice_the_dense_rate():
    flops = bench.kernel_work("fwd_fused", 2048, 9216, 27648, 96)[0]
    assert bench.sweep_peak_s("fwd_fused", 2048, 9216, 27648, 96, P, False) == pytest.approx(flops / (2 * P * 1e12))


def test_int8_products_are_measured_against_the_int8_rate():
    T, inn, out, r = 2048, 9216, 27648, 96
    main, adapter = 2.0 * T * inn * out / (4 * P * 1e12), 2.0 * T * r * out / (P * 1e12)
    assert bench.sweep_peak_s("fwd_q8", T, inn, out, 0, P, True) == pytest.approx(main)
    assert bench.sweep_peak_s("fwd_q8", T, inn, out, r, P, True) == pytest.approx(main + adapter)
    assert bench.sweep_peak_s("adapter_fwd", T, inn, out, r, P, True) == pytest.approx(2.0 * T * r * inn / (P * 1e12))
    assert bench.sweep_peak_s("rmsnorm_q8", T, inn, out, r, P, True) == 0.0


def test_no_int8_call_reads_above_its_peak_at_the_recorded_times():
    """9216 -> 36864 at 2048 tokens took 314 us: below the int8 peak, above the bf16 one that it was held against."""
    frac = bench.sweep_peak_s("fwd_q8", 2048, 9216, 36864, 96, 1632.3, True) / 314e-6
    assert 0.5 < frac < 1.0
    assert bench.sweep_peak_s("fwd_q8", 2048, 9216, 36864, 96, 1632.3, False) / 314e-6 > 1.0
