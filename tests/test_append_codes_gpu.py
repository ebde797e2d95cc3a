"""Codes of attn_append_paged_fp8 bit for bit: every finite bf16 value, as key and as value, over many
coefficients, against fp32 division and torch's e4m3 rounding. No tolerance: ties (x / coefficient halfway
between two codes) are as common as short significands are, and each has one code."""
import pytest
import torch

from causal_attention_attn_b200 import attn, build

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    if torch.cuda.get_device_capability(0) != (10, 0):
        pytest.skip("needs an sm_100 device")
    build.build()
    attn.load_library()
    yield
    torch.cuda.synchronize()


def coefficients(which):
    g = torch.Generator().manual_seed(3)
    short = 1 + torch.arange(D) / 128.0  # every significand of eight bits
    if which == "short":
        return short
    if which == "random":
        return 0.5 + torch.rand((D,), generator=g)
    if which == "long":  # significands next to 1 and 2, and next to the short ones
        bits = torch.cat((short[::2], short[::2])).view(torch.int32)
        bits[:64] += 1
        bits[64:] -= 1  # the first of these is 1 - 2^-24, all ones
        return bits.view(torch.float32)
    scaled = short.clone()  # the ends of the range that is promised
    scaled[::2] *= 2.0 ** -93
    scaled[1::2] *= 2.0 ** 125
    return scaled


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("which", ["short", "random", "long", "scaled"])
def test_every_value_takes_the_quotients_code(which, interleaved):
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = x[torch.isfinite(x.float())]
    S, page = x.numel(), 128
    rows = x[:, None].expand(S, D).contiguous().view(1, 1, S, D).cuda()
    per = -(-S // page)
    coef = coefficients(which)
    kp = torch.zeros((per, 1, page, D), dtype=torch.uint8, device="cuda")
    vp = kp.clone()
    attn.attn_append_paged_fp8(rows, rows, None, None, kp, vp, coef.view(1, D).cuda(), coef.view(1, D).cuda(),
                               torch.arange(per, dtype=torch.int32).view(1, per).cuda(),
                               torch.tensor([S], dtype=torch.int32).cuda(), interleaved=interleaved)
    want = (x.float()[:, None] / coef).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    for what, pages in (("k", kp), ("v", vp)):
        got = pages.cpu().view(-1, D)[:S]
        bad = (got != want).nonzero()
        assert len(bad) == 0, (f"{what}: {len(bad)} codes differ, first {float(x[bad[0][0]])} / {float(coef[bad[0][1]])}: "
                               f"{int(got[tuple(bad[0])])}, not {int(want[tuple(bad[0])])}")
