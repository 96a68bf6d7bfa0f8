"""One workspace for chunk attention and the INT4 decode calls."""
import pytest
import torch

from bit_kv_cache_13_gb300 import _lib
from test_gpu_chunk import Case

pytestmark = pytest.mark.gpu


def test_chunk_and_decode_calls_take_turns_in_one_workspace():
    """Units that several CTAs finish together (they count on tickets), of 1 to 40 sequences, after chunk calls of other shapes."""
    big = Case(1, [200, 60], [700, 300], 8, 2)
    decodes = [Case(2, [1], [5000], 4, 1), Case(3, [1] * 3, [2000, 0, 900], 8, 2), Case(4, [1] * 40, [300] * 40, 8, 2)]
    n = big.workspace().numel()
    for c in decodes:
        B, (h_q, h_kv) = len(c.new), (c.h_q, c.h_kv)
        n = max(n, _lib.kvq_int4_workspace_bytes(B, h_q, h_kv, c.bt.shape[1], 0), _lib.kvq_int4_workspace_bytes(B, h_q, h_kv, c.bt.shape[1], 3))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for c in decodes:
            q, _, *args = c.device()
            for splits, sliding in ((0, False), (3, False), (0, True)):
                big.check(big.run(ws))
                outs = []
                for w in (torch.zeros_like(ws), ws):
                    out = torch.empty_like(q)
                    if sliding:
                        _lib.kvq_decode_attn_int4_sliding(q, *args, 3000, 4, out, w, splits)
                    else:
                        _lib.kvq_decode_attn_int4(q, *args, out, w, splits)
                    outs.append(out)
                assert torch.equal(*outs)
                assert _lib.load().kvq_workspace_status(ws.data_ptr(), None) == 0
                if not sliding:
                    c.check(outs[1].cpu())
