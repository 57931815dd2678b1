"""Refusals and build rules of the receiver's decode calls at their edges: host only, nothing here
launches a kernel."""
import os
import types

import pytest
import torch

import cross_model_attention_block_b200 as package
from cross_model_attention_block_b200 import build
from cross_model_attention_block_b200 import mapflow as mfb
from tests.test_decode_host import BAD, NOGPU, attn, call_attn, needs_no_gpu

LOWEST = float(torch.finfo(torch.float32).min)


@needs_no_gpu
@pytest.mark.parametrize("kw,status", [
    (dict(scale=3e38), BAD), (dict(scale=-3e38), BAD), (dict(scale=2e38), NOGPU),
    (dict(band_bias=3e38, band_width=1), BAD), (dict(band_bias=-LOWEST, band_width=9), BAD),
    (dict(band_bias=3e38, band_width=0), NOGPU), (dict(band_bias=2.3e38, band_width=9), NOGPU),
    (dict(band_bias=LOWEST, band_width=9), NOGPU), (dict(band_bias=LOWEST, band_width=0), NOGPU),
])
def test_scales_and_biases_at_the_types_limits(lib, kw, status):
    assert call_attn(lib, a=attn(**kw)) == status and lib.mf_last_error().decode()


@pytest.mark.parametrize("other", ["torch", "python", "record"])
def test_marshalling_is_built_again_for_another_torch_or_python(lib, tmp_path, monkeypatch, other):
    """The library counts as built only for the torch and the Python that it was built for."""
    import sysconfig
    so, src, record = (str(tmp_path / n) for n in ("_marshal.so", "marshal.cpp", "marshal_for"))
    for f in (src, so):
        open(f, "w").close()
    later = os.path.getmtime(os.path.join(build.ROOT, "include", "mapflow.h")) + 1e6
    os.utime(so, (later, later))
    with open(record, "w") as f:
        f.write(build.marshal_key())
    for name, path in (("MARSHAL", so), ("MARSHAL_SRC", src), ("MARSHAL_FOR", record)):
        monkeypatch.setattr(build, name, path)
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build.subprocess, "run", run)
    assert build.build_marshal() == so and not ran             # as it was
    if other == "torch":
        monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    elif other == "python":
        soabi = sysconfig.get_config_var
        monkeypatch.setattr(sysconfig, "get_config_var",
                            lambda n: "cpython-00" if n == "SOABI" else soabi(n))
    else:
        os.remove(record)                                      # of an earlier build
    build.build_marshal()
    assert len(ran) == 1
    build.build_marshal()                                      # recorded: not once more
    assert len(ran) == 1


def test_marshalling_for_another_torch_is_not_loaded(lib, monkeypatch):
    mfb._load_fast()
    monkeypatch.setattr(mfb, "_fast", None)
    monkeypatch.setattr(package._marshal, "built_for", "torch 0.0.1", raising=True)
    with pytest.raises(RuntimeError, match="_marshal.so"):
        mfb.KVCache.make(1, 16, 1, 64, torch.float32, torch.zeros(1, 1, dtype=torch.int32))
    assert mfb._fast is None
