"""The attention's workspace may hold anything before a call: splits without
key tiles leave their parts unwritten, and the merge must not read them."""
import pytest
import torch

from long_context_compressed_hca_b200 import binding as hb
from tests.helpers import rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pos", [1048575, 300000])
def test_hca_attend_ignores_what_the_workspace_held(cuda, pos):
    B, n_h, c, rd, w, m, cap = 4, 64, 512, 64, 128, 128, 8200
    bf = torch.bfloat16
    q, kv, win = rnd((B, 1, n_h, c), 71, 1, bf), rnd((B, cap, c), 71, 2, bf), rnd((B, w, c), 71, 3, bf)
    sink = rnd((n_h,), 71, 4)
    d = hb.attn_desc(B, n_h, c, rd, w, m, dtype=hb.HCA_BF16)
    nbytes = hb.hca_attend_workspace_size(d, 1, pos)
    assert nbytes > 0                    # more than 8 splits: merged through the workspace
    out = []
    for fill in (0x00, 0xFF):            # 0xFF: NaN patterns
        ws = torch.full((nbytes,), fill, dtype=torch.uint8, device=cuda)
        o = torch.empty_like(q)
        hb.hca_attend(d, q, kv, cap, win, 1, sink, 1, pos, o, ws)
        out.append(o)
    assert not torch.isnan(out[1].float()).any()
    assert torch.equal(out[0], out[1])
