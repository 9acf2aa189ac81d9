"""The attention kernels, compiled for gfx950 with the library's flags, never
chain a matrix instruction onto the accumulator of one of another shape
(tests/test_mfma_chains.py says why), and call nothing."""
import os
import re
import shutil

import pytest

from tests.test_mfma_chains import _asm, _build, shape_switches


@pytest.mark.skipif(not os.path.exists(_build.HIPCC) and shutil.which("hipcc") is None, reason="hipcc not available")
def test_attention_accumulator_chains(tmp_path):
    text = _asm("attn_step.hip", str(tmp_path / "attn_step.s"))
    assert "v_mfma_f32_16x16x32_bf16" in text and "v_mfma_f32_16x16x4_f32" in text
    assert not shape_switches(text)[:4]
    assert not re.search(r"\ts_swappc", text)
