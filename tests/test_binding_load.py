"""Loading the library and the compiled part of the binding: from two threads at once, and when a
part is missing."""
import importlib.util
import os
import subprocess
import sys
import threading
import time

import pytest
import torch

import mxfp4_expert_gemm_b200 as moe
from mxfp4_expert_gemm_b200 import build


@pytest.fixture
def unloaded(monkeypatch):
    build.build()
    monkeypatch.setattr(moe, "_lib", None)
    monkeypatch.setattr(moe, "_marshal", None)


def _refusal():
    """What a product call answers to a host tensor: only the compiled part can tell."""
    try:
        moe.moe_linear(torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16))
    except Exception as e:   # noqa: BLE001
        return e


def test_first_calls_of_two_threads(unloaded, monkeypatch):
    """The second call comes while the first one loads: both are whole."""
    real = importlib.util.spec_from_file_location

    def slow(*a, **k):
        time.sleep(0.3)
        return real(*a, **k)

    monkeypatch.setattr(importlib.util, "spec_from_file_location", slow)
    got = {}
    threads = [threading.Thread(target=lambda i=i: (time.sleep(0.1 * i), got.__setitem__(i, _refusal())))
               for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert [type(got[i]) for i in range(4)] == [TypeError] * 4, got


def test_a_failed_binding_publishes_nothing(unloaded):
    class Other:   # a library that lacks the calls
        pass

    moe._lib = Other()
    for _ in range(2):
        with pytest.raises(AttributeError):
            moe.moe_linear(None, None)
        assert moe._marshal is None


def test_the_compiled_part_unbound_refuses():
    """Before it has the library's addresses its calls raise; they follow no null pointer."""
    build.build()
    code = ("import importlib.util as u, sys, torch\n"
            "s = u.spec_from_file_location('_marshal', sys.argv[1]); m = u.module_from_spec(s); s.loader.exec_module(m)\n"
            "for f, n in ((m.norm, 8), (m.norm_backward, 12), (m.product, 12), (m.product_backward, 15)):\n"
            "    try:\n"
            "        f(*[None] * n)\n"
            "    except RuntimeError as e:\n"
            "        assert 'not bound' in str(e), e\n"
            "    else:\n"
            "        raise SystemExit('no refusal')\n"
            "for bad in ([0] * 8, [1] * 7):\n"
            "    try:\n"
            "        m.bind(*bad)\n"
            "    except (ValueError, TypeError):\n"
            "        continue\n"
            "    raise SystemExit('bound')\n")
    r = subprocess.run([sys.executable, "-c", code, build.build_marshal()], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_a_missing_compiled_part_stops_its_own_calls_only(unloaded, monkeypatch):
    real = os.path.exists
    monkeypatch.setattr(os.path, "exists", lambda p: real(p) and "_marshal" not in str(p))
    dims = moe.make_dims(64, 64, 4, 2)
    for _ in range(2):
        assert moe.moe_workspace_bytes(dims, 4) > 0           # the layer's own calls do without
        assert moe.moe_linear_workspace_bytes(moe.make_linear_dims(64, 64), 4) > 0
        with pytest.raises(RuntimeError, match="missing"):
            moe.moe_norm(torch.zeros(4, 64), torch.ones(64))
    monkeypatch.undo()


def test_a_compiled_part_for_another_torch_is_not_loaded(unloaded, monkeypatch):
    assert isinstance(_refusal(), TypeError)
    monkeypatch.setattr(moe, "_marshal", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert isinstance(_refusal(), RuntimeError) and "missing" in str(_refusal())


def test_another_library_is_bound_too(unloaded):
    """use_library before and after the first product call."""
    for _ in range(2):
        with moe.use_library(moe.LIB_PATH) as other:
            assert moe.lib() is other and isinstance(_refusal(), TypeError)
        assert moe.lib() is not other and isinstance(_refusal(), TypeError)
