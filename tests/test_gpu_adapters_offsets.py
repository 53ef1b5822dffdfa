"""Low-rank adapters without a base, through the C ABI: base's pitch means
nothing then, whatever it holds, and decides nothing about offsets of y's rows.
(T times a pitch of 2^62 or so passes the range of 64 bits.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import quantized_moe_q4_b200 as m  # noqa: E402


@pytest.mark.parametrize("ldb", [0, -1, 2 ** 63 - 1, -2 ** 63, 2 ** 62 // 300 + 1, 2 ** 52])
@pytest.mark.parametrize("T", [6, 260, 1200])
def test_any_pitch_of_a_base_that_is_not_there(T, ldb):
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    kw = dict(device="cuda", generator=g)
    A = m.Adapters(torch.randn(2, 16, 512, **kw).bfloat16(), torch.randn(2, 200, 16, **kw).bfloat16())
    x, ids = torch.randn(T, 512, **kw), torch.randint(-1, 2, (T,), **kw).int()
    want = m.moe_q4_adapters_apply(A, x, ids)
    ldy = (6 << 30) // 4 // T // 4 * 4 + 8
    y = torch.empty((T - 1) * ldy + 200, device="cuda").as_strided((T, 200), (ldy, 1))   # 6 GB
    ws = m.alloc_workspace(m.moe_q4_adapters_workspace_bytes(A, T))
    rc = m.library().moe_q4_adapters_apply(A.ref, x.data_ptr(), 512, ids.data_ptr(), T, None, ldb, y.data_ptr(), ldy,
                                           ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert torch.equal(y, want)
