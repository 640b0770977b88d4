"""GPU parity of tl_lora_plan and tl_lora_apply against the 64-bit oracle (oracle/serving.py).

Tolerance, for u = 2^-23 (a matrix instruction may truncate its fp32 sums) and
T = scale |B| (|A| |x|):
  h      (K / 16 + 40) u, and its split into parts: 2^-16 (bf16), 2^-21 (fp16 parts),
         2^-22 (three bf16 parts)
  y      (rank / 16 + 20) u, then half a unit in the last place of its type
"""

import numpy as np
import pytest
import torch

from oracle import serving as O
from quantized_linear_layers_block_gb300 import tl

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_ULP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


def make(seed, M, K, N, rank, n, dtype="bf16", out="bf16", ids=None, mult=1.0):
    rng = np.random.default_rng(seed)
    f = lambda *s: torch.tensor(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    x = (f(M, K) * mult).to(TYPES[dtype])
    A, B = (f(n, rank, K) / K ** 0.5).to(TYPES[dtype]), (f(n, N, rank) / rank ** 0.5).to(TYPES[dtype])
    scale = torch.tensor(rng.uniform(-2, 2, n).astype(np.float32))
    base = f(M, N).to(TYPES[out])
    if ids is None:
        ids = rng.integers(-1, n, M)
    return x, A, B, scale, base, np.asarray(ids, dtype=np.int32)


def check(x, A, B, scale, base, ids, dtype="bf16", out="bf16", in_place=False, wide=0, stream=None):
    M, K = x.shape
    bank = tl.LoraBank(A.cuda(), B.cuda(), scale.cuda())
    plan = bank.plan(torch.tensor(ids).cuda(), stream=stream)
    xd, bd = x.cuda(), base.cuda()
    if wide:
        xw = torch.zeros((M, K + wide), dtype=x.dtype, device="cuda")
        bw = torch.full((M, base.shape[1] + wide), 3.0, dtype=base.dtype, device="cuda")
        xw[:, :K], bw[:, :base.shape[1]] = xd, bd
        xd, bd = xw[:, :K], bw[:, :base.shape[1]]
    y = bank.apply(xd, bd, plan, out=bd if in_place else None, stream=stream)
    assert tl.tl_get_status(stream) == tl.TL_OK
    ref, T = O.lora(x.double().numpy(), base.double().numpy(), A.double().numpy(), B.double().numpy(), scale.double().numpy(), ids)
    u = 2.0 ** -23
    split = 2.0 ** -21 if dtype == "f16" else 2.0 ** -22 if out == "f32" else 2.0 ** -16
    tol = HALF_ULP[out] * np.abs(ref) + ((K / 16 + 40 + A.shape[1] / 16 + 20) * u + split) * T + 2.0 ** -24 * (out == "f16") + u * np.abs(ref)
    got, fine = y.double().cpu().numpy(), np.isfinite(ref)
    assert np.array_equal(np.isfinite(got), fine)
    err = np.abs(got - ref)[fine]
    assert np.all(err <= tol[fine]), float((err / tol[fine]).max())
    bare = ids < 0
    assert torch.equal(y.cpu()[bare], base[bare])
    if wide and in_place:
        assert bool((bw[:, base.shape[1]:] == 3).all())
    return y


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rank", [8, 16, 24, 32, 64, 72, 128])
def test_types_and_ranks(dtype, out, rank):
    check(*make(rank, 70, 520, 264, rank, 4, dtype, out), dtype, out)


@pytest.mark.parametrize("M", [1, 2, 8, 31, 32, 33, 65, 300])
@pytest.mark.parametrize("K,N", [(8, 8), (40, 1000), (5120, 512), (1000, 136)])
def test_sizes(M, K, N):
    check(*make(M + K, M, K, N, 16, 3))


def test_few_and_many_adapters():
    check(*make(1, 50, 256, 128, 16, 1))
    check(*make(2, 200, 256, 128, 8, 500))
    check(*make(3, 40, 256, 128, 16, 2, ids=[-1] * 40))
    check(*make(4, 100, 256, 128, 16, 3, ids=[1] * 100))
    check(*make(5, 33, 256, 128, 16, 2, ids=[0] * 16 + [1] + [-1] * 16), in_place=True)


@pytest.mark.parametrize("M", [39, 45, 52, 70, 90, 140, 305])
def test_clusters_of_every_size(M):
    check(*make(100 + M, M, 2056, 1000, 24, M, ids=np.arange(M)))


@pytest.mark.parametrize("rank", [40, 64, 96, 128])
@pytest.mark.parametrize("M,n", [(1, 1), (5, 5), (20, 1), (60, 4)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16")])
def test_few_items_of_large_adapters(rank, M, n, dtype, out):
    check(*make(400 + M + rank, M, 6152, 2056, rank, n, dtype, out, ids=np.arange(M) % n), dtype, out)


@pytest.mark.parametrize("M", [1023, 1024, 1100])
@pytest.mark.parametrize("rank", [8, 32, 128])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_both_sizes_of_items(M, rank, out):
    check(*make(300 + M + rank, M, 392, 296, rank, 5, out=out), out=out)


@pytest.mark.parametrize("M", [1, 3, 7, 11])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_columns_of_an_item_over_several_clusters(M, out):
    check(*make(200 + M, M, 600, 20008, 40, M, out=out, ids=np.arange(M)), out=out)


def test_in_place_strided_and_another_stream():
    for out in ("bf16", "f32"):
        check(*make(6, 45, 264, 200, 16, 3, out=out), out=out, in_place=True)
        check(*make(7, 45, 264, 200, 16, 3, out=out), out=out, in_place=True, wide=24)
        check(*make(8, 45, 264, 200, 16, 3, out=out), out=out, wide=8)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        check(*make(9, 45, 264, 200, 16, 3), stream=st)
        st.synchronize()


@pytest.mark.filterwarnings("ignore:invalid value")
def test_first_products_beyond_f16():
    """A x above 65504 and far below f16's normal range: the second product keeps its precision. (At 3e4 some
    elements of x are infinite themselves: what they reach is not finite, in the oracle and here.)"""
    for mult in (3e4, 5e3, 1e-5):
        x, A, B, scale, base, ids = make(10, 20, 512, 64, 16, 2, "f16", "f32", mult=mult)
        A = (A.float() * 16).half()
        check(x, A, B, scale, base * 0, ids, "f16", "f32")


def test_repeats_are_equal_and_a_token_does_not_depend_on_its_batch():
    x, A, B, scale, base, ids = make(11, 64, 1024, 256, 32, 5)
    a = check(x, A, B, scale, base, ids)
    assert torch.equal(a, check(x, A, B, scale, base, ids))
    turn = np.random.default_rng(0).permutation(64)
    b = check(x[turn], A, B, scale, base[turn], ids[turn])
    assert torch.equal(a[torch.tensor(turn).cuda()], b)


def test_plan_rewrite_and_mismatch():
    x, A, B, scale, base, ids = make(12, 40, 256, 128, 16, 3)
    bank = tl.LoraBank(A.cuda(), B.cuda(), scale.cuda())
    plan = bank.plan(torch.zeros(40, dtype=torch.int32, device="cuda"))
    bank.plan(torch.tensor(ids).cuda(), plan)
    y = bank.apply(x.cuda(), base.cuda(), plan)
    assert torch.equal(y, check(x, A, B, scale, base, ids))
    with pytest.raises(ValueError):
        bank.plan(torch.zeros(41, dtype=torch.int32, device="cuda"), plan)
    with pytest.raises(ValueError):
        bank.apply(x[:39].cuda(), base[:39].cuda(), plan)
    # a plan of another batch under this one's description: refused on the device, nothing written
    other = bank.plan(torch.tensor(ids[:30]).cuda())
    forged = tl.LoraPlan(40, 3, torch.zeros((tl.tl_lora_plan_size(40, 3),), dtype=torch.uint8, device="cuda"))
    forged.data[:other.data.numel()] = other.data
    hold = torch.full_like(y, 7.0)
    bank.apply(x.cuda(), base.cuda(), forged, out=hold)
    assert tl.tl_get_status() == tl.TL_EDATA and bool((hold == 7).all())


def test_adapter_out_of_range_is_reported():
    x, A, B, scale, base, ids = make(13, 10, 64, 64, 8, 3)
    bank = tl.LoraBank(A.cuda(), B.cuda(), scale.cuda())
    ids[4] = 3
    plan = bank.plan(torch.tensor(ids).cuda())
    assert tl.tl_get_status() == tl.TL_EDATA
    y = bank.apply(x.cuda(), base.cuda(), plan)
    assert tl.tl_get_status() == tl.TL_OK and torch.equal(y[4].cpu(), base[4])


def test_infinities_stay_in_their_token():
    x, A, B, scale, base, ids = make(14, 12, 64, 64, 8, 2, ids=[0] * 12)
    x[3, 5] = float("inf")
    bank = tl.LoraBank(A.cuda(), B.cuda(), scale.cuda())
    y = bank.apply(x.cuda(), base.cuda(), bank.plan(torch.tensor(ids).cuda())).cpu()
    others = [i for i in range(12) if i != 3]
    assert bool(torch.isfinite(y[others].float()).all()) and not bool(torch.isfinite(y[3].float()).any())


def test_a_large_batch():
    check(*make(15, 3001, 512, 1024, 16, 7))
    check(*make(16, 3001, 256, 520, 64, 3, out="f32"), out="f32")


def test_no_tokens():
    x, A, B, scale, base, _ = make(17, 4, 64, 64, 8, 2)
    bank = tl.LoraBank(A.cuda(), B.cuda(), scale.cuda())
    plan = bank.plan(torch.empty((0,), dtype=torch.int32, device="cuda"))
    assert bank.apply(x[:0].cuda(), base[:0].cuda(), plan).shape == (0, 64)


def test_binding_refusals():
    x, A, B, scale, base, ids = make(18, 4, 64, 64, 8, 2)
    x, A, B, scale, base = (t.cuda() for t in (x, A, B, scale, base))
    for bad in ((A.float(), B, scale), (A, B.half(), scale), (A, B[:1], scale), (A[:, :, :4], B, scale), (A, B, scale[:1]), (A, B, scale.double())):
        with pytest.raises(ValueError):
            tl.LoraBank(*bad)
    bank = tl.LoraBank(A, B, scale)
    plan = bank.plan(torch.tensor(ids).cuda())
    for bad in ((x.half(), base), (x[:, :32], base), (x, base[:, :32]), (x, base.double()), (x.cpu(), base), (x, base[:3])):
        with pytest.raises(ValueError):
            bank.apply(*bad, plan)
    with pytest.raises(ValueError):
        bank.plan(torch.tensor(ids).cuda().long())
    with pytest.raises(ValueError):
        bank.apply(x, base, plan, out=base.float())
