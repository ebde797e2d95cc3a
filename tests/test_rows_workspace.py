"""The gradient's workspace is sized in the header, for callers in C, and in the binding: the same bytes."""
import os
import re

import pytest

from causal_attention_attn_b200 import attn, build


@pytest.mark.parametrize("D", [32, 64, 128])
def test_the_bindings_workspace_is_the_headers(D):
    with open(os.path.join(build.INCLUDE, "attn.h")) as f:
        macro = re.search(r"#define ATTN_QK_NORM_ROPE_BWD_WORKSPACE\(D\) (.*)", f.read()).group(1)
    want = eval(re.sub(r"(\d+)u", r"\1", macro).replace("(unsigned)(D)", str(D)))
    assert attn._NORM_ROPE_BWD_BLOCKS * 2 * D * 4 == want
