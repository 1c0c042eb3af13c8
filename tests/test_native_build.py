"""The marshalling module belongs to the interpreter that it was built for."""
import importlib.machinery
import os

import latent_attention_decode_absorbed_b200 as mla
from latent_attention_decode_absorbed_b200 import build as mla_build


def test_module_carries_the_interpreter_s_tag():
    untagged = os.path.join(mla_build.PKG, "_native.so")
    with open(untagged, "wb"):
        pass                                              # an older build's
    mla_build.build()
    assert not os.path.exists(untagged)
    tag = importlib.machinery.EXTENSION_SUFFIXES[0]
    assert tag != ".so"                                   # a plain .so loads into any interpreter
    assert os.path.basename(mla_build.BINDING) == "_native" + tag
    assert os.path.exists(mla_build.BINDING)
    assert os.path.samefile(mla.native().__file__, mla_build.BINDING)
