"""The package imports, and its host-only parts work, where torch was built without CUDA."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_without_torchs_cuda_bindings():
    code = ("import torch\n"
            "for name in [n for n in dir(torch._C) if n.startswith('_cuda')]: delattr(torch._C, name)\n"
            "import kimi_delta_attention_gated_gb300 as kda\n"
            "f, m = kda.rotary_inv_freq(8, device='cpu')\n"
            "assert f.numel() == 4 and m == 1.0 and kda.kv_cache(2, 1, 64, device='cpu').k.shape == (2, 1, 64, 64)\n"
            "x = torch.zeros((1, 1, 64), dtype=torch.bfloat16)\n"
            "i = torch.zeros(1, dtype=torch.int32)\n"
            "for call in (lambda: kda.attn_decode(x, kda.kv_cache(2, 1, 64, device='cpu'), i[None], i),\n"
            "             lambda: kda.kv_append(x, x, kda.kv_cache(2, 1, 64, device='cpu'), i[None], i)):\n"
            "    try: call()\n"
            "    except ValueError: pass\n"
            "    else: raise SystemExit('not refused')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]


def test_inv_freq_refuses_a_base_without_angles():
    import pytest

    from kimi_delta_attention_gated_gb300 import rotary_inv_freq
    for base in (0.0, -10000.0, float("inf"), float("nan")):
        for scaling in (None, "ntk", "yarn"):
            with pytest.raises(ValueError):
                rotary_inv_freq(64, base=base, scaling=scaling, factor=2.0, device="cpu")
    for factor in (float("inf"), float("nan")):
        with pytest.raises(ValueError):
            rotary_inv_freq(64, scaling="yarn", factor=factor, device="cpu")
