"""What build.py makes, and when."""
import os
import sysconfig

import torch

from pagedattention_kv_cache_attention_gb300 import build


def test_binding_is_named_for_its_torch_and_its_python():
    name = os.path.basename(build.BIND)
    assert torch.__version__ in name
    assert name.endswith("." + sysconfig.get_config_var("SOABI") + ".so")
