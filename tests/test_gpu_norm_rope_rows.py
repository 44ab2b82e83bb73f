"""kvq_norm_rope of a single row out of a wider buffer: its stride is not used, whatever it is."""
import pytest

from gpu_util import kvq_lib, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [1, 3, 7])
def test_a_single_row_of_any_stride(dtype, pad):
    torch, kvq = torch_cuda(), kvq_lib()
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    hq, hkv = 4, 2
    width = (hq + 2 * hkv) * 128
    buf = torch.randn(3, width + pad, device="cuda").to(dt)
    rope = kvq.Rope([10000.0 ** (-i / 32) for i in range(32)])
    pos = torch.tensor([[77]], dtype=torch.int32, device="cuda")
    one = torch.ones(128, device="cuda")

    def call(rows):
        out = [torch.empty(rows.shape[0], h, 128, dtype=dt, device="cuda") for h in (hq, hkv, hkv)]
        kvq.kvq_norm_rope(rows, pos[:, :rows.shape[0]], rope, one, one, 1e-6, *out)
        return out

    got, want = call(buf[:1, :width]), call(buf[:1, :width].contiguous())
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    with pytest.raises(kvq.KvqError):  # two rows: they would start off a 16-byte boundary
        kvq.kvq_norm_rope(buf[:2, :width], pos.expand(1, 2).contiguous(), rope, one, one, 1e-6,
                          *[torch.empty(2, h, 128, dtype=dt, device="cuda") for h in (hq, hkv, hkv)])
