"""How many shares paged_attention cuts a batch into: no more workgroups than are resident at once."""
import pytest

import weight_only_quantized_topk_amd as wq


def workspace(shares, D, heads):
    """Two pieces a share and head (D + 2 float32), two int32 a share, each of the three arrays rounded up to 256 bytes."""
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    return up(2 * shares * heads * D * 4) + up(2 * shares * heads * 2 * 4) + up(shares * 8)


@pytest.mark.parametrize("D", [16, 64, 80, 128, 192, 256])
@pytest.mark.parametrize("kv_heads,group", [(1, 1), (2, 4), (3, 1), (3, 16), (5, 8), (7, 1), (8, 8), (12, 1), (20, 1), (2, 20),
                                            (1, 71), (48, 1), (300, 1), (700, 1), (1100, 1), (2000, 1)])
def test_a_share_a_resident_workgroup(D, kv_heads, group):
    units = kv_heads * -(-group // 16)
    resident = 256 * (4 if D <= 64 else 3 if D <= 128 else 2)
    nbytes = wq.paged_attention_workspace_bytes(4, kv_heads * group, kv_heads, D, 16, 1 << 13)
    assert nbytes == workspace(max(1, resident // units), D, kv_heads * group)
