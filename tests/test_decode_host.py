"""The decode operators' host side without a GPU: refusals, the cache's handle, the extension module's build."""
import ctypes

import pytest

vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def fp4():
    from moe_nvfp4_gemv_gb300 import fp4gemv
    return fp4gemv


@pytest.mark.parametrize("inv_t,status", [(0.99e-20, 1), (1e-30, 1), (1.01e-20, 3), (1e6, 3), (1.01e6, 1)])
def test_logprobs_range_of_temperatures(fp4, inv_t, status):
    """Outside the range: refused for it (1), before the misaligned logits are (3)."""
    assert fp4.lib().fp4gemv_token_logprobs(vp((1 << 20) + 1), 100, 0, 1, 100, None, inv_t, 4, None, None, None, None, None,
                                            1, None) == status


RUN = """
import sys
sys.path.insert(0, {root!r})
{setup}
from moe_nvfp4_gemv_gb300 import fp4gemv, kvcache, linear
import torch
assert fp4gemv.scale_bytes(128, 64) == 512 and fp4gemv.launch_count() == 0
x, i = torch.zeros(2, 8), torch.zeros(2, 2, dtype=torch.int32)
cache = kvcache.KvCache8.allocate(2, 1, 64, 16, device="cpu")
for call in (lambda: fp4gemv.moe_route(x, 2, ids=i, weights=x[:, :2]), lambda: fp4gemv.token_logprobs(x, i[:, 0]),
             lambda: cache.append(x, x, i, i), lambda: cache.attend(x, i, i, out=x, workspace=x)):
    try:
        call()
    except RuntimeError as e:
        assert "no module" in str(e) and not isinstance(e, fp4gemv.Fp4GemvError), e
    else:
        raise AssertionError("a call without its module went through")
print("fine")
"""


@pytest.mark.parametrize("setup", [
    "class No:\n    def find_spec(self, name, *a):\n        if name.endswith('_marshal'): raise ImportError('no module')\n"
    "sys.meta_path.insert(0, No())",
    "from moe_nvfp4_gemv_gb300 import build\nbuild._marshal_stale = lambda: True\n"
    "def failing(*a, **k): raise RuntimeError('no module: no compiler')\nbuild.build = failing"])
def test_the_package_without_its_extension_module(setup):
    """The products' calls need libfp4gemv.so alone; those of the decode operators say what is missing."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", RUN.format(root=root, setup=setup)], capture_output=True, text=True)
    assert out.returncode == 0 and "fine" in out.stdout, out.stderr


@pytest.mark.parametrize("name,other", [("__version__", "2.0.0+other"), ("__file__", "/elsewhere/torch/__init__.py")])
def test_the_extension_module_is_rebuilt_for_another_torch(monkeypatch, name, other):
    """Whatever the files' times are."""
    import torch

    from moe_nvfp4_gemv_gb300 import build
    build.build()
    assert not build._marshal_stale()
    monkeypatch.setattr(torch, name, other)
    assert build._marshal_stale()


def test_a_cache_keeps_its_tensors():
    """The calls use the memory that the cache was made with: its tensors cannot be exchanged behind their back."""
    import torch

    from moe_nvfp4_gemv_gb300.kvcache import KvCache8
    cache = KvCache8.allocate(2, 1, 64, 16, device="cpu")
    for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
        was = getattr(cache, name)
        with pytest.raises(AttributeError):
            setattr(cache, name, torch.ones_like(was))
        was.fill_(3)  # (in place: the same memory)
        assert getattr(cache, name) is was
    s = cache._struct
    assert [s.k_codes, s.v_codes, s.k_scale, s.v_scale] == [t.data_ptr() for t in (cache.k_codes, cache.v_codes,
                                                                                 cache.k_scale, cache.v_scale)]
