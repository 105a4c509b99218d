"""gdn_attn_decode's waits that give up: GDN_FLAG_TEST_STALL lets the last computing warp of a CTA wait on a barrier that nothing
arrives on while the others go on to the group's end.  Nothing of the group may be written -- not by the warps that missed
nothing, not by the CTAs that hold other parts of it -- and every sequence reports bit 4."""
import pytest
import torch

import gated_deltanet_linear_decode_gb300 as gdn
from tests.test_attn_decode import BF, F32, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[40], [5, 0, 17, 300], [9000], [20] * 200])
@pytest.mark.parametrize("dtype,out_dtype,Hq,K,d", [
    (BF, BF, 8, 1, 64), (BF, F32, 8, 2, 128), (BF, BF, 8, 3, 256), (BF, BF, 8, 4, 256), (BF, F32, 8, 16, 128),
    (BF, BF, 8, 9, 64), (BF, BF, 16, 16, 256), (F32, F32, 2, 1, 64), (F32, F32, 8, 1, 128), (F32, BF, 8, 4, 64), (F32, F32, 8, 16, 64)])
def test_one_late_warp_stops_its_group(dtype, out_dtype, Hq, K, d, lens):
    c = Case(lens, K, Hq, 1, d, 16, dtype, seed=21)
    B = len(lens)
    dims = gdn.make_attn_dims(Hq, 1, d, dtype, out_dtype, test_stall=True)
    ws = torch.zeros(gdn.gdn_attn_decode_workspace_bytes(dims, B, K), dtype=torch.uint8, device="cuda")
    out = torch.full((B * K, Hq * d), 7.0, dtype=out_dtype, device="cuda")
    st = torch.zeros(B, dtype=torch.int32, device="cuda")
    gdn.gdn_attn_decode(dims, gdn.KvCache(c.k, c.v), K, c.q, c.table.cuda(), c.seq_len, out, gate=c.gate, workspace=ws, dev_status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [16] * B and (out == 7.0).all()
    ws.zero_()
    c.close(c.run(out_dtype, ws=ws))
