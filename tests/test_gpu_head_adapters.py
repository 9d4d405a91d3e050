"""The adapters' form on the tensor cores (pairs of CTAs), each test sure that it reaches it, and the
precision that the projection's kernels state: f32 logits summed outside the accumulator, u in 24 bits."""

import pytest
import torch

import ragged_log_probs_gb300 as lp
from tests import parity
from tests.test_gpu_head_project import BF16, E4M3, F16, F32, Case

pytestmark = pytest.mark.gpu

V = 20001
# requests of 256 and of 600 rows (one tile, three): blocks of one adapter, of two, of one and none
ONE_TILE = ([0, 40, 96, 160, 168, 256], [0, 1, 2, -1, 1])
TILES = ([0, 3, 130, 200, 232, 296, 300, 420, 600], [0, 2, -1, 1, 1, 0, 2, 1])


@pytest.fixture(scope="module", autouse=True)
def _built():
    parity.ensure_built()


def on_tensor_cores(c):
    return lp.project_cut(c.T, c.x.shape[1], c.V, c.x.dtype, c.A, c.rank)[2]


@pytest.mark.parametrize("dtype,lora_dtype", [(BF16, BF16), (F16, F16), (E4M3, BF16), (E4M3, F16)])
@pytest.mark.parametrize("rank", [8, 16, 32, 40, 48, 56, 64])
def test_ranks(rank, dtype, lora_dtype):
    off, ids = ONE_TILE
    H = 512 if dtype == E4M3 else 256  # 512 bytes: pairs are not taken for less
    c = Case(256, H, V, dtype, A=3, rank=rank, ids=ids, off=off, seed=41, lora_dtype=lora_dtype)
    assert on_tensor_cores(c)
    for out_dtype in (F32, BF16):
        c.check(c.run(out_dtype))


@pytest.mark.parametrize("dtype", [BF16, F16, E4M3])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("form", [ONE_TILE, TILES])
def test_several_chunks_and_passes_in_a_ring_of_accumulators(form, out_dtype, dtype):
    off, ids = form
    c = Case(off[-1], 2304, V, dtype, A=3, rank=64, ids=ids, off=off, seed=42, lora_dtype=BF16 if dtype == E4M3 else None)
    assert on_tensor_cores(c)
    c.check(c.run(out_dtype))


@pytest.mark.parametrize("dtype,scale", [(F16, 1e-18), (F16, 1e18), (F16, 1e-30), (F16, 1e30), (BF16, 1e-18), (BF16, 1e30)])
def test_sizes_of_u_far_from_one(dtype, scale):
    # through adapter_scale: u leaves float16's range, and the whole sum with it
    off, ids = ONE_TILE
    c = Case(256, 256, V, dtype, A=3, rank=16, ids=ids, off=off, seed=43, unit=True)
    assert on_tensor_cores(c)
    w = torch.zeros_like(c.w)
    out = c.run(w=w.cuda(), adapter_scale=torch.full((3,), scale).cuda()).double().cpu()
    s = float(torch.tensor(scale))
    for b, a in enumerate(ids):
        r = slice(off[b], off[b + 1])
        if a < 0:
            assert (out[r] == 0).all()
            continue
        u, um = c.x[r].double() @ c.la[a].double().t() * s, c.x[r].double().abs() @ c.la[a].double().abs().t() * s
        # sums of 256 and of 3 x 16 products, each step losing at most 2^-23 of the magnitudes; f16 parts
        # hold u to 2^-38 of the row's largest
        bound = (um @ c.lb[a].double().abs().t()) * (256 / 16 + 2 * 16 + 8) * 2.0 ** -23
        bound += 2.0 ** -37 * u.abs().amax(1, keepdim=True) * c.lb[a].double().abs().sum(1)
        assert ((out[r] - u @ c.lb[a].double().t()).abs() <= bound).all()


def products_in_64_bits(x, w):
    return x.cuda().double() @ w.cuda().double().t()


def relative(out, want):
    return float((out.double() - want).norm() / want.norm())


@pytest.mark.parametrize("T,most", [(8, 8e-7), (64, 8e-7), (256, 1.5e-6)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_f32_logits_are_summed_outside_the_accumulator(T, most, dtype):
    """The accumulator loses up to its last place at every step of 16 products, on average half, always
    towards zero: a sum of c products that end at a part sqrt(c / H) of the whole loses about (c / 16)
    (2/3) sqrt(c / H) 2^-24 of it, and the H / c such sums lose independently of each other. With H =
    4096 and c = 768, then 512: 1.4e-6; 384, then 256 (tiles of up to 64 rows): 6.8e-7, to which the
    f32 additions of 16 sums add 2^-24 each at random (1.2e-7). All at once: 1e-5 (4.4e-6 measured)."""
    g = torch.Generator().manual_seed(T)
    x, w = torch.randn(T, 4096, generator=g).to(dtype), torch.randn(V, 4096, generator=g).to(dtype)
    out = lp.project(x.cuda(), w.cuda(), workspace=lp.new_head_workspace())
    assert relative(out, products_in_64_bits(x, w)) < most


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("rank", [16, 64])
def test_u_enters_the_tensor_cores_in_24_bits(rank, dtype):
    """Adapters whose part is all of the logits. Two 16-bit parts of 8 bits would leave u 2^-17 off on
    average (7.6e-6). u itself is a sum of H = 512 products in f32, 2^-24 off at each of 32 steps at
    most, and the three parts' 12 steps of 16 products lose 2/3 2^-24 each: below 2^-24 (32 + 8) = 2.4e-6
    where all fell one way; half of that is asked for."""
    off, ids = [0, 64, 256], [0, 1]
    c = Case(256, 512, V, dtype, A=2, rank=rank, ids=ids, off=off, seed=44, lora_dtype=BF16)
    assert on_tensor_cores(c)
    out = c.run(F32, w=torch.zeros(V, 512).to(dtype).cuda())
    for b in range(2):
        r = slice(off[b], off[b + 1])
        x = c.x[r].cuda().double()
        if c.sx is not None:
            x = x * c.sx[r].cuda().double()[:, None]
        want = float(c.scale[b]) * (x @ c.la[b].cuda().double().t()) @ c.lb[b].cuda().double().t()
        assert relative(out[r], want) < 1.2e-6


def test_pairs_give_the_same_result_each_time_and_in_a_graph():
    off, ids = TILES
    c = Case(600, 1024, V, BF16, A=3, rank=32, ids=ids, off=off, seed=45)
    assert on_tensor_cores(c)
    first = c.run()
    for _ in range(3):
        assert torch.equal(c.run(), first)
    x, w, la, lb, sc = (t.cuda() for t in (c.x, c.w, c.la, c.lb, c.scale))
    ids, off = (torch.tensor(v, dtype=torch.int32).cuda() for v in (ids, off))
    ws, out = lp.new_head_workspace(600, 32), torch.empty(600, V, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            lp.project(x, w, lora_a=la, lora_b=lb, adapter_scale=sc, adapter_ids=ids, row_offsets=off, out=out, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
