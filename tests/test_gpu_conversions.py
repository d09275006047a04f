"""The hardware's conversions to bf16 and E4M3, and the addition that makes
int8 codes, on every fp32: the operators' bits are those of the block's integer
rules (f32_to_bf16 and quant4 in csrc), which are written out here."""
import pytest
import torch

import moe_expert_ffn_route_amd as moe

pytestmark = pytest.mark.gpu
T, H = 16386, 16384  # with a column for the largest value, more than 2^28 others
PART = 1 << 28


def values(first, n):
    """The n fp32 whose bits follow `first`."""
    return torch.arange(first, first + n, device="cuda").to(torch.int32).view(torch.float32)


def bf16_bits(x):
    """Nearest, ties to even, in integers; a NaN keeps its upper bits and is quiet."""
    u = x.view(torch.int32).long() & 0xFFFFFFFF
    near = (u + 0x7FFF + ((u >> 16) & 1)) >> 16
    return torch.where((u & 0x7FFFFFFF) > 0x7F800000, (u >> 16) | 0x40, near).to(torch.int16)


@pytest.mark.parametrize("part", range(16))
def test_bf16_of_every_fp32(part):
    """The joining norm of ones gated by x, one for each element: r = x. Rows of
    16383 end in seven elements that are converted one by one."""
    width = H - 1
    x = values(part * PART - (1 << 31), T * width).view(T, width)  # wraps behind the last part
    out = torch.empty(T, width, dtype=torch.bfloat16, device="cuda")
    d = moe.make_join_norm_dims(T, width, weight_dtype=torch.float32, gate_rows=T, quant=moe.MOE_QUANT_NONE)
    moe.moe_w8a8_join_norm(d, torch.ones_like(out), gate=x, residual_out=out)
    for rows in range(0, T, 4096):
        assert torch.equal(out[rows:rows + 4096].view(torch.int16), bf16_bits(x[rows:rows + 4096]))


def check(q, t, quant):
    if quant == moe.MOE_QUANT_INT8:
        return torch.equal(q, torch.round(t).clamp(-127, 127).to(torch.int8))
    # E4M3: steps of 2^(e - 3) from 2^-6 on, of 2^-9 below
    e = torch.clamp(((t.view(torch.int32) >> 23) & 0xFF) - 127, min=-6)
    power = lambda n: ((n + 127) << 23).view(torch.float32)  # noqa: E731
    want = torch.round(t * power(3 - e)) * power(e - 3)
    return torch.equal(q.float().view(torch.int32), want.view(torch.int32))  # the sign of zero, too


@pytest.mark.parametrize("amax", [1.0, 448.0])
@pytest.mark.parametrize("quant", [moe.MOE_QUANT_INT8, moe.MOE_QUANT_E4M3], ids=["int8", "e4m3"])
def test_codes_of_every_fp32(quant, amax):
    """Every value up to the row's largest, from the quantiser and both norms,
    whose codes come from r and max|r| alone."""
    top = torch.tensor(127.0 if quant == moe.MOE_QUANT_INT8 else 448.0, device="cuda")
    last = int(torch.tensor(amax).view(torch.int32))
    f32 = torch.float32
    q = torch.empty(T, H, dtype=torch.int8 if quant == moe.MOE_QUANT_INT8 else torch.float8_e4m3fn, device="cuda")
    s = torch.empty(T, device="cuda")
    x = torch.empty(T, H, device="cuda")
    for first in range(0, last + 1, PART):
        for sign in (1, -1):
            x[:, 0] = amax
            torch.mul(values(first, T * (H - 1)).view(T, H - 1).clamp(max=amax), sign, out=x[:, 1:])
            calls = (
                lambda: moe.moe_w8a8_quant(moe.make_quant_dims(T, H, dtype=f32, quant=quant), x, q=q, q_scale=s),
                lambda: moe.moe_w8a8_norm_quant(moe.make_norm_dims(T, H, dtype=f32, quant=quant), x, q=q, q_scale=s),
                lambda: moe.moe_w8a8_join_norm(moe.make_join_norm_dims(T, H, dtype=f32, quant=quant), x, q=q, q_scale=s))
            t = x * top * (1.0 / torch.tensor(amax, device="cuda"))
            for call in calls:
                q.view(torch.int8).fill_(-128)
                call()
                for rows in range(0, T, 4096):
                    assert check(q[rows:rows + 4096], t[rows:rows + 4096], quant), (first, sign)
