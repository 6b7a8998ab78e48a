"""The build's products: what makes them anew, and which Python they are for."""
import importlib.machinery
import os
import sysconfig

import pytest

from paged_kv_cache_248_gb300 import _build


def test_the_module_carries_the_abi_of_its_python():
    _build.build()
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert suffix and suffix != ".so"
    assert os.path.basename(_build.NATIVE) == "_native" + suffix and os.path.exists(_build.NATIVE)
    assert importlib.machinery.EXTENSION_SUFFIXES[0] == suffix  # found before a _native.so of an older build
    import paged_kv_cache_248_gb300 as pkv
    assert pkv._calls().__file__ == _build.NATIVE


@pytest.mark.parametrize("what", ["no record", "other flags", "other python"])
def test_the_module_is_built_anew_for_another_python_or_other_flags(what):
    """File times do not tell that the interpreter or the command has changed; the command that made it does."""
    _build.build()
    record = os.path.join(_build.OUT_DIR, "_native.cmd")
    with open(record) as f:
        made_by = f.read()
    before = os.stat(_build.NATIVE)
    _build.build()
    assert os.stat(_build.NATIVE).st_ino == before.st_ino  # nothing to do
    if what == "no record":
        os.remove(record)
    else:
        with open(record, "w") as f:
            f.write(made_by + " -O0" if what == "other flags" else made_by.replace("python3", "python4"))
    _build.build()
    assert os.stat(_build.NATIVE).st_ino != before.st_ino
    with open(record) as f:
        assert f.read() == made_by
