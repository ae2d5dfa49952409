"""What an Engine needs before a language operator is called: the library, and neither torch nor the operators' native
module (csrc/binding.cpp)."""
import os
import subprocess
import sys
import types

import pytest


from vla_dual_expert_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DIMS = types.SimpleNamespace(layers=1, hidden_v=128, inter_v=128, hidden_a=128, inter_a=128, n_q=4, n_kv=2, head_dim=32,
                             chunk=4, action_dim=8, rope_theta=1e6, rms_eps=1e-6)

# a library whose contexts are numbers, for a machine without a GPU
FAKE = """
import types

import pytest
import vla_dual_expert_b200 as pkg

class Lib:
    def dm0_create(self, cfg, out):
        out._obj.value = 7
        return 0
    def dm0_device(self, h):
        return 0
    def dm0_destroy(self, h):
        pass

pkg.load_library = Lib
"""


def _python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_an_engine_without_torch():
    build.build()
    r = _python("import sys\nsys.modules['torch'] = None\n" + FAKE +
                f"e = pkg.Engine(types.{DIMS!r}".replace("namespace", "SimpleNamespace") + ", 1, 16)\n"
                "assert e.device == 0\nassert e.weights_bytes\nprint('made')\n")
    assert r.returncode == 0 and r.stdout.strip() == "made", r.stderr


def test_a_native_module_that_does_not_load_is_named_by_the_first_operator():
    build.build()
    r = _python("import sys\nsys.modules['vla_dual_expert_b200._language'] = None\n" + FAKE +
                f"e = pkg.Engine(types.{DIMS!r}".replace("namespace", "SimpleNamespace") + ", 1, 16)\n"
                "for call in (lambda: e.embed(None, None), lambda: e.vocab_loss(None, None, None)):\n"
                "    try:\n        call()\n    except ImportError as x:\n        print(x)\n")
    assert r.returncode == 0, r.stderr
    lines = r.stdout.strip().splitlines()
    assert len(lines) == 2 and all("_language.so" in x and "vla_dual_expert_b200.build" in x for x in lines)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_prefill_tokens_takes_no_other_image_rows(dtype):
    """Image rows of another type are refused and not rounded in passing, host tensors as everywhere."""
    import torch
    build.build()
    from vla_dual_expert_b200.language import LanguageOps
    ids = torch.zeros(2, 3, dtype=torch.int64)
    with pytest.raises(TypeError, match="image_emb must be a CUDA torch.bfloat16 tensor"):
        LanguageOps().prefill_tokens(torch.zeros(2, 4, 64, dtype=getattr(torch, dtype)), None, ids)


def test_without_torch_the_library_alone_is_built(monkeypatch):
    build.build()
    asked = []
    monkeypatch.setattr(build, "build_library", lambda *a: asked.append("library"))
    monkeypatch.setattr(build, "build_binding", lambda *a: asked.append("binding"))
    build.build()
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    assert build.build() == build.LIB
    assert asked == ["library", "binding", "library"]


def test_device_of_no_context():
    build.build()
    from vla_dual_expert_b200 import load_library
    assert load_library().dm0_device(None) == -1


def test_another_torch_or_interpreter_rebuilds_the_binding(tmp_path, monkeypatch):
    """Without running the compiler: which builds are asked for."""
    build.build()
    assert build._binding_fresh()
    calls = []

    class Done(Exception):
        pass

    def run(cmd, **kw):
        calls.append(cmd)
        raise Done

    monkeypatch.setattr(build.subprocess, "run", run)
    assert build.build_binding() == build.BINDING and not calls
    for change in (lambda m: m.setattr(build.importlib.metadata, "version", lambda name: "2.99.0"),
                   lambda m: m.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-399-x86_64-linux-gnu"),
                   lambda m: m.setattr(build, "BINDING_STAMP", str(tmp_path / "missing")),
                   lambda m: m.setattr(build, "BINDING_FLAGS", ["-O3"])):
        with monkeypatch.context() as m:
            change(m)
            assert not build._binding_fresh()
            with pytest.raises(Done):
                build.build_binding()
    assert len(calls) == 4 and all("binding.cpp" in " ".join(c) for c in calls)
