"""CPU tests of the serving operators' limits: constants of the header and the binding,
sizes that are refused before any launch."""

import os
import re

from paged_kv_gb300 import pkv

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "pkv.h")


def test_binding_constants_match_the_header():
    text = open(HEADER).read()
    for name in ("PKV_MAX_HEAD_DIM", "PKV_ATTENTION_ZERO_BYTES"):
        m = re.search(r"#define\s+%s\s+(\d+)" % name, text)
        assert m is not None and int(m.group(1)) == getattr(pkv, name), name


def test_the_largest_attention_workspace():
    """What the default workspaces take, prompts of 128 wide heads, covers every call."""
    need = pkv.paged_attention_workspace_bytes
    most = need(1, 64, 64, 1, 1, 128)
    for b, n, longest, hq, hkv, d in ((1, 1, 1, 1, 1, 16), (256, 256, 1, 16, 8, 128),
                                      (9, 70000, 4096, 32, 4, 128), (4096, 10 ** 6, 10 ** 6, 64, 1, 96)):
        assert pkv.PKV_ATTENTION_ZERO_BYTES < need(b, n, longest, hq, hkv, d) <= most


def test_bias_lists_end_before_32_bits_do():
    """Threads look 512 entries ahead in 32 bits."""
    from test_serving_abi import adjust

    for n in ((1 << 30) + 1, (1 << 31) - 1, 1 << 31):
        assert adjust(nb=n) == pkv.PKV_EINVAL
        assert "n_bias" in pkv.last_error()
