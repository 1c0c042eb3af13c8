"""Host limits of mla_step_plan (no GPU; the pointers are never dereferenced)."""
import pytest

import latent_attention_decode_absorbed_b200 as mla
from test_tree_host import PLAN, UNS, _refused, lib  # noqa: F401


@pytest.mark.parametrize("over", [dict(max_rows=2 ** 31 - 1), dict(max_rows=2 ** 31 - 4096), dict(mask_words=1 << 25),
                                  dict(mask_words=2 ** 31 - 1)])
def test_sizes_past_the_kernel_s_integers_are_refused(over):
    _refused(mla.mla_step_plan, {**PLAN, **over}, UNS)
