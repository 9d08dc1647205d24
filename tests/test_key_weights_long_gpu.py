"""Key weights of prompts that need more than one dispatch group of heads, and sums long enough
for their compensation to count."""
import math

import pytest
import torch

from paged_util import DT, default_scale

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,Hq,Hkv,d,dtype,group", [(1, 70, 70, 64, "bf16", 64),
                                                    (2, 20, 5, 128, "fp16", 32),
                                                    (5, 13, 13, 64, "fp16", 64)])
@pytest.mark.parametrize("causal", [False, True])
def test_dispatch_groups(B, Hq, Hkv, d, dtype, group, causal):
    """Heads are dispatched in groups whose Q fills 32 MiB: at N = 4096 64 heads of d = 64 or 32
    of d = 128, and a last group of fewer. Every head against float64 on the GPU."""
    import io_aware_attention_fa2_gb300 as fa
    N = 4096
    assert (32 << 20) // (2 * N * d) == group and group < B * Hq and B * Hq % group
    g = torch.Generator().manual_seed(Hq + d)
    q = torch.randn((B, N, Hq, d), generator=g).to(DT[dtype]).cuda()
    k = torch.randn((B, N, Hkv, d), generator=g).to(DT[dtype]).cuda()
    # the sums need no softmax: any LSE is one, here around ln(N) + 1/2
    lse = (8.8 + 0.3 * torch.randn((B, Hq, N), generator=g)).cuda()
    lens = torch.tensor([N, 3000, 1, N - 1, 129][:B], dtype=torch.int32, device="cuda")
    scale = default_scale(d)
    out = torch.full((B, Hkv, N), math.nan, device="cuda")
    fa.key_weights(q, k, lse, causal=causal, scale=scale, seqlens_k=lens, out=out)
    i = torch.arange(N, device="cuda")
    for b in range(B):
        n = int(lens[b])
        see = (i[:, None] < n) & (i[None] < n)
        if causal:
            see &= i[None] <= i[:, None]
        for hk in range(Hkv):
            want = torch.zeros(N, dtype=torch.float64, device="cuda")
            bound = torch.zeros_like(want)
            for h in range(hk * (Hq // Hkv), (hk + 1) * (Hq // Hkv)):
                qq, kk = q[b, :, h].double(), k[b, :, hk].double()
                s = qq @ kk.T * scale
                p = torch.where(see, torch.exp(s - lse[b, h, :, None].double()), 0.0)
                # as in key_weights_ref: the score's sum of d products, LSE * log2(e) and the
                # difference rounded in 32 bits, exp2 and sums of 64 (2^-24 a step), and the
                # compensated sum of the tiles
                e = scale * (d + 2) * 2.0 ** -23 * (qq.abs() @ kk.abs().T)
                r = e + 2.0 ** -22 * (lse[b, h, :, None].double().abs() + s.abs()) + 2.0 ** -17
                want += p.sum(0)
                bound += (p * r).sum(0)
            got = out[b, hk].double()
            assert ((got - want).abs() <= bound + 1e-30).all(), (b, hk)


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "fp16")])
def test_sums_of_long_prompts_are_compensated(d, dtype):
    """Scores of zero: every key gets e^-LSE_0 (2^24) and 65535 times 0.0073. A half tile of the
    latter adds 0.94, less than half of the last bit of 2^24, so that a plain 32-bit sum of the
    256 tiles would lose 239 of 479: 1.4e-5 of the sum.

    What the kernel may be off, relative to the sum: LSE_0 * log2(e) = -24 rounded to 32 bits
    (2^-20, numbers from 16 to 32 having steps of 2^-19) from a constant rounded to 2^-25 of itself
    (24 * 2^-25), both times ln 2: 1.2e-6; exp2 2^-22; what the first half tile adds beside the
    large term (0.94, lost at most: 6e-8); four roundings of a sum near 2^24, 2^-25 each: 1.2e-7.
    Together 1.7e-6 < 2^-19."""
    import io_aware_attention_fa2_gb300 as fa
    N = 65536
    q = torch.zeros((1, N, 1, d), dtype=DT[dtype], device="cuda")
    lse = torch.full((1, 1, N), -math.log(0.0073), device="cuda")
    lse[0, 0, 0] = -24 * math.log(2.0)
    w = fa.key_weights(q, q.clone(), lse, scale=default_scale(d)).double()
    want = torch.exp(-lse.double()).sum()
    assert float(((w - want).abs() / want).max()) < 2.0 ** -19
