"""The forms of the selective kernels that calls with more blocks than the GPU has SMs take.

152 SMs: a pass over tokens has a block for 64 channels (32 for d_state = 64) of a row; the step takes four rows a block from
4 * 512 * 2 groups of four components an SM on."""
import pytest
import torch

from selectivelib import make, scan64, within
from test_selective_gpu import check, check_grad

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
NAN = float("nan")


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("ds,D", [(8, 2056), (16, 2056), (32, 1048), (64, 520)])
@pytest.mark.parametrize("gate,skip,bias,state", [(True, True, True, True), (False, False, False, False)])
def test_more_blocks_than_sms(cuda_lib, dt, ds, D, gate, skip, bias, state):
    """B rows of one segment each: outputs, states in front of chunks and the walk back."""
    d = make(10, 41, D, ds, dt, seed=ds, gate=gate, skip=skip, bias=bias, state=state)
    check(cuda_lib, d)
    check_grad(cuda_lib, d)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("ds,D", [(8, 1032), (16, 1032), (32, 1032), (64, 520)])
def test_more_blocks_than_sms_padded(cuda_lib, dt, ds, D):
    lengths = torch.tensor([0, 1, 32, 41, 33, 50, -3, 17, 40, 16], dtype=torch.int32, device="cuda")
    d = make(10, 41, D, ds, dt, seed=ds + 1, state=True)
    check(cuda_lib, d, lengths)
    check_grad(cuda_lib, d, lengths)


@pytest.mark.parametrize("ds", [8, 16, 32])
def test_more_blocks_than_sms_in_segments(cuda_lib, ds):
    lengths = torch.tensor([520, 256, 257, 519, 1], dtype=torch.int32, device="cuda")
    d = make(5, 520, 1032, ds, BF16, seed=ds + 2, state=True)
    check(cuda_lib, d, lengths)
    check_grad(cuda_lib, d, lengths)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("ds,D", [(8, 2056), (16, 1032), (32, 1032), (64, 520)])
@pytest.mark.parametrize("opts", [True, False])
def test_steps_of_many_rows(cuda_lib, dt, ds, D, opts):
    """Four rows a block: the last block has three; slots that repeat inside a block, in the next one and far apart, unused
    and bad ones beside good ones."""
    B, n = 319, 400
    assert B * D * ds // 4 >= 4 * 512 * 2 * torch.cuda.get_device_properties(0).multi_processor_count
    d = make(B, 1, D, ds, dt, seed=ds, gate=opts, skip=opts, bias=opts)
    g = torch.Generator(device="cuda").manual_seed(ds)
    pool = torch.randn(n, D, ds, generator=g, device="cuda")
    slots = torch.randperm(n, generator=g, device="cuda")[:B].int()
    for row, of in ((5, 4), (11, 8), (100, 3), (16, 15), (201, 16), (318, 0), (317, 316)):
        slots[row] = slots[of]
    for row, bad in ((20, -1), (21, n), (22, -7), (23, 2**31 - 1), (316, n + 5), (40, -1), (41, -1)):
        slots[row] = bad
    seen, good = set(), []
    for row, s in enumerate(slots.tolist()):
        if 0 <= s < n and s not in seen:
            good.append(row)
            seen.add(s)
    before, opt = pool.clone(), {k: d[k] for k in ("D", "dt_bias", "softplus")}
    one = [d["x"][:, 0], d["dt"][:, 0], d["A"], d["Bm"][:, 0], d["Cm"][:, 0]]
    z = None if d["z"] is None else d["z"][:, 0]
    out = torch.full((B, D), NAN, dtype=dt, device="cuda")
    assert cuda_lib.la_selective_scan_step(*one, pool, z=z, slots=slots, out=out, **opt) is out
    assert cuda_lib.device_status() == 1 and cuda_lib.device_status() == 0
    at = slots[good].long()
    rows = {k: d[k][good] if d[k] is not None else None for k in ("x", "dt", "Bm", "Cm", "z", "dout")}
    ref, bound, S, Sb, _ = scan64(d | rows | {"S0": before[at]})
    within(out[good], ref[:, 0], bound[:, 0], "out")
    within(pool[at], S, Sb, "S")
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(pool[rest], before[rest]), "a state outside the batch was touched"
    skipped = torch.ones(B, dtype=torch.bool, device="cuda")
    skipped[good] = False
    assert out[skipped].eq(0).all()
    # without slots: row b on state b; one row at a time gives the same bits as four a block
    pool = before.clone()
    out = cuda_lib.la_selective_scan_step(*one, pool, z=z, **opt)
    few = before[:9].clone()
    cut = [t if t is d["A"] else t[:9] for t in one]
    o = cuda_lib.la_selective_scan_step(*cut, few, z=None if z is None else z[:9], **opt)
    assert torch.equal(o, out[:9]) and torch.equal(few, pool[:9]) and torch.equal(pool[B:], before[B:])
    assert cuda_lib.device_status() == 0
