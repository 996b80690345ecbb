"""Without the marshalling module the build names every call that needs it, and
each of them raises.  CPU only."""
import os

import pytest

import fp16_tensor_core_gb300 as dg
from fp16_tensor_core_gb300 import build as dg_build

CALLS = {"dg_rope": 4, "dg_kv_append": 4, "dg_kv_read": 3, "dg_attn_decode": 6, "dg_rmsnorm": 2, "dg_rmsnorm_e4m3": 3,
         "dg_rmsnorm_e4m3_amax": 4, "dg_rmsnorm_grad": 3, "dg_activate": 2, "dg_activate_grad": 3,
         "dg_fp8_gemm_fused": 5, "dg_hgemm_fused": 3}


def test_what_the_marshalling_module_is_for(monkeypatch, tmp_path):
    native = os.path.join(tmp_path, os.path.basename(dg_build.NATIVE))
    monkeypatch.setattr(dg_build, "NATIVE", native)
    monkeypatch.setattr(dg, "_NATIVE_PATH", native)
    monkeypatch.setattr(dg, "_native", None)
    which = dg_build.shutil.which
    monkeypatch.setattr(dg_build.shutil, "which", lambda name: None if name == "gcc" else which(name))
    with pytest.warns(UserWarning) as caught:
        dg_build.build()
    message = next(str(w.message) for w in caught if "gcc" in str(w.message))
    for name, arguments in CALLS.items():
        assert f"{name}," in message or f"{name})" in message, name
        with pytest.raises(RuntimeError, match="not found; build it"):
            getattr(dg, name)(*[0] * arguments)
