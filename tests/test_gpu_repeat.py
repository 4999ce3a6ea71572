"""The FP4 products give the same bits at every call: sums have a fixed order, and
nothing depends on when copies and warps run.  Each case is launched many times, in
bursts after a pause (whose first launches find cold caches and slow warps), and each
output compared with the first, which is compared with the formula."""

import pytest
import torch

from tests.test_gpu_gated import SCALES, activations, check, matrices

pytestmark = pytest.mark.gpu

BURST = 16


def repeat(call, m, n, bursts):
    """The first output, and how many of the others differ from it."""
    first = call(torch.empty(m, n, dtype=torch.bfloat16, device="cuda"))
    outs = [torch.empty_like(first) for _ in range(BURST)]
    differ = 0
    for _ in range(bursts):
        for o in outs:
            o.fill_(7.0)
            call(o)
        differ += sum(torch.stack([(o != first).any() for o in outs]).tolist())
    return first, differ


# 16 or 17 experts whose tiles, four to a CTA, take the 256-row kernel with its two
# stages of weights
RAGGED = [0, 272, 281, 281, 312, 341, 593, 627, 628, 637, 1004, 1008, 1008, 1040, 1043, 1046, 1046, 1058]
EVEN = [0, 252, 444, 684, 936, 1128, 1368, 1620, 1812, 2052, 2304, 2496, 2736, 2988, 3180, 3420, 3672]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("off", [RAGGED, EVEN], ids=["ragged", "even"])
def test_gated_groups(cuda_lib, off, fmt):
    n, k = 2368, 384
    mats = [matrices(cuda_lib, n, k, fmt, 60 + e, SCALES[fmt]) for e in range(len(off) - 1)]
    rep = torch.cat([m[0] for m in mats])
    a = activations(off[-1], k, fmt, 17)
    ws = cuda_lib.Workspace()
    torch.cuda.synchronize()
    y, differ = repeat(lambda o: cuda_lib.moe_gated_gemm(a, rep, off, n, fmt, [SCALES[fmt]] * len(mats), "silu", ws, o),
                       off[-1], n, 400)
    for e, (_, wg, wu) in enumerate(mats):
        s = slice(off[e], off[e + 1])
        if off[e] < off[e + 1]:
            check(y[s], a[s], wg, wu, SCALES[fmt], "silu", f"expert {e}")
    assert differ == 0 and ws.status() == 0


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("m,n", [(4096, 14208), (300, 4736), (64, 4736), (1, 4736)])
def test_plain(cuda_lib, m, n, fmt):
    k, gen = 384, torch.Generator().manual_seed(18)
    group, low, high = (16, 0x20, 0x38) if fmt == "nvfp4" else (32, 124, 128)   # scales of 2^-3 .. 2^0
    rep = cuda_lib.repack(torch.randint(0, 256, (n, k // 2), generator=gen, dtype=torch.uint8).cuda(),
                          torch.randint(low, high, (n, k // group), generator=gen, dtype=torch.uint8).cuda(), fmt)
    a = activations(m, k, fmt, 18)
    ws = cuda_lib.Workspace()
    torch.cuda.synchronize()
    y, differ = repeat(lambda o: cuda_lib.gemm(a, rep, n, fmt, 1.0, ws, o), m, n, 100)
    # half a step of BF16, and the sum's 384 additions: a step of FP32 (2^-23) each, of
    # the products' sizes at most, 2^-14.4 of them
    w, x = cuda_lib.dequant(rep, n, k, fmt).double(), a[:256].double()
    want = x @ w.T
    assert ((y[:256].double() - want).abs() <= want.abs() * 2.0**-8 + (x.abs() @ w.abs().T) * 2.0**-14).all()
    assert differ == 0 and ws.status() == 0
