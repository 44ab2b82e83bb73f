"""kvq_norm_rope of heads whose squares leave fp32's range, beside ordinary ones (bounds: test_gpu_norm_rope, to which a
head scaled by a power of two adds no rounding)."""
import math

import numpy as np
import pytest

from gpu_util import kvq_lib, torch_cuda

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def run(dtype, scales, eps, side=False, rotary=64, hq=6, hkv=2, seed=1):
    """Head h of token t of the size scales[(t + h) % len(scales)]."""
    torch, kvq = torch_cuda(), kvq_lib()
    rng = np.random.default_rng(seed)
    n, heads = 37, hq + 2 * hkv
    size = np.asarray(scales, np.float64)[(np.arange(n)[:, None] + np.arange(heads)) % len(scales)]
    x = np.clip(rng.normal(size=(n, heads, 128)), -3, 3) * size[..., None]
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    qkv = torch.from_numpy(x.reshape(n, -1)).to(dt).cuda()
    pos = torch.from_numpy(rng.integers(0, 5000, (1, n))).to(torch.int32).cuda()
    w = [torch.from_numpy(1 + 0.4 * rng.normal(size=128)).float().cuda() for _ in range(2)]
    freq = [10000.0 ** (-i / (rotary // 2)) for i in range(rotary // 2)]
    out = [torch.full((n, h, 128), math.nan, dtype=dt, device="cuda") for h in (hq, hkv, hkv)]
    kvq.kvq_norm_rope(qkv, pos, kvq.Rope(freq, interleaved=side), *w, eps, *out)
    x = qkv.double().cpu().numpy().reshape(n, heads, 128)
    at = 0
    for y, h, wt in zip(out, (hq, hkv), w):
        part, at = x[:, at:at + h], at + h
        ref = part / np.sqrt((part ** 2).mean(-1, keepdims=True) + float(np.float32(eps))) * wt.double().cpu().numpy()
        m = np.abs(ref)
        for i, f in enumerate(freq):
            a, b = (2 * i, 2 * i + 1) if side else (i, i + rotary // 2)
            ang = (pos[0].cpu().numpy().astype(np.float64) * f)[:, None]
            p, q = ref[..., a].copy(), ref[..., b].copy()
            ref[..., a], ref[..., b] = p * np.cos(ang) - q * np.sin(ang), p * np.sin(ang) + q * np.cos(ang)
            m[..., a] = m[..., b] = np.hypot(p, q)
        y = y.double().cpu().numpy()
        tol = 32 * U * m + (2.0 ** -8 if dtype == "bf16" else U) * np.abs(ref) + 1e-37
        assert np.isfinite(y).all() and (np.abs(y - ref) <= tol).all(), float((np.abs(y - ref) / tol).max())
    assert (out[2].cpu().reshape(n, -1) == qkv[:, -hkv * 128:].cpu()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("scales", [(1e20,), (1e18, 1.0, 1e38), (1.0, 1e30, 1e-3, 1e19, 1e5)])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_large_heads(dtype, side, scales, eps):
    run(dtype, scales, eps, side)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("scales", [(1e-20,), (1e-15, 1.0, 1e-25), (1e-36, 1e36, 1.0)])
@pytest.mark.parametrize("eps", [0.0, 1e-36, 1e-30])
def test_small_heads_without_an_eps_to_speak_of(dtype, side, scales, eps):
    run(dtype, scales, eps, side)


@pytest.mark.parametrize("rotary", [0, 16, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (40, 4), (64, 8)])
def test_other_head_counts(rotary, hq, hkv):
    if rotary:
        run("f32", (1e25, 1.0, 1e-22, 1e38, 2.0), 0.0, rotary=rotary, hq=hq, hkv=hkv)
    else:
        torch, kvq = torch_cuda(), kvq_lib()
        x = torch.full((3, (hq + 2 * hkv) * 128), 1e30, device="cuda")
        out = [torch.empty(3, h, 128, device="cuda") for h in (hq, hkv, hkv)]
        one = torch.ones(128, device="cuda")
        kvq.kvq_norm_rope(x, None, kvq.Rope([]), one, one, 1e-6, *out)
        assert all((o - 1).abs().max() <= 32 * U for o in out[:2])


def test_infinities_and_zeros_as_the_formula_has_them():
    torch, kvq = torch_cuda(), kvq_lib()
    x = torch.ones(2, 3 * 128, device="cuda")
    x[0, 5] = math.inf
    x[1] = 0.0
    out = [torch.empty(2, 1, 128, device="cuda") for _ in range(3)]
    one = torch.ones(128, device="cuda")
    kvq.kvq_norm_rope(x, None, kvq.Rope([]), one, one, 0.0, *out)
    want = torch.zeros(128)
    want[5] = math.nan  # infinity over infinity
    assert torch.equal(out[0][0, 0].cpu().nan_to_num(7.0), want.nan_to_num(7.0))
    assert torch.isnan(out[0][1]).all()  # 0 / 0
    kvq.kvq_norm_rope(x, None, kvq.Rope([]), one, one, 1e-6, *out)
    assert (out[0][1] == 0).all()
