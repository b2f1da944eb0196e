"""bench.py --beams on the GPU: one JSON line with every kernel of the step."""

import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_beam_step():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--beams", "--steps", "3", "--warmup", "1"],
                       capture_output=True, text=True, timeout=110)
    assert r.returncode == 0, r.stderr[-2000:]
    line = json.loads(r.stdout.strip().splitlines()[-1])
    assert line["n_gpus"] == 1 and line["steps"] == 3 and line["value"] > 0 and line["unit"] == "tokens/s"
    assert {"latent_attention", "latent_join", "head_product", "beam_stats", "beam_select", "beam_reorder",
            "reserve_plan", "reserve_write", "cache_write", "cache_plan", "cache_copy"} <= set(line["kernels_us"])
    assert {"prompt_plan", "prompt_expand", "prompt_scale", "prompt_attention"} == set(line["prompts"]["kernels_us"])
