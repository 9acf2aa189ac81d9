"""The scan's prompt kernels, compiled for gfx950 with the library's flags,
never chain a matrix instruction onto the accumulator of one of another shape
(tests/test_mfma_chains.py says why), and call nothing."""
import os
import re
import shutil

import pytest

from tests.test_mfma_chains import _asm, _build, shape_switches


@pytest.mark.skipif(not os.path.exists(_build.HIPCC) and shutil.which("hipcc") is None, reason="hipcc not available")
def test_scan_accumulator_chains(tmp_path):
    text = _asm("ssm_prefill.hip", str(tmp_path / "ssm_prefill.s"))
    assert "v_mfma_f32_32x32x16_bf16" in text and "v_mfma_f32_16x16x32_bf16" in text
    assert not shape_switches(text)[:4]
    assert not re.search(r"\ts_swappc", text)
