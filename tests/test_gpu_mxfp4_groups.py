"""moe_gemm_mxfp4 over padded segments, through every kernel it can take: held
to float64, its padding and the rows behind the segments left alone, and in
captured graphs."""
import numpy as np
import pytest
import torch

import fp8_grouped_gemm_amd as moe
import ops_util as ou
from parity_util import say
from test_gpu_mxfp4_ops import DT, bound, operand

pytestmark = pytest.mark.gpu

# routed rows, n, k, segments, alignment, the tile of a call that states its
# rows, whether b streams past the caches
CASES = [(14, 459, 1024, 12, 16, (16, 16), False), (3, 105, 1120, 20, 1, (16, 16), False),
         (2, 512, 7168, 2, 128, (16, 16), False), (87, 683, 1248, 3, 16, (32, 16), False),
         (183, 920, 448, 17, 16, (32, 64), False), (625, 3705, 480, 7, 16, (32, 128), False),
         (1088, 1368, 1504, 5, 64, (64, 128), False), (1662, 1784, 1600, 9, 128, (128, 128), False),
         (3030, 5065, 832, 7, 128, (256, 256), False),
         # the three kernels whose copies of b are nontemporal: 32 x 128 with two and with three
         # buffers (more than 256 tiles, and fewer), 128 x 128
         (496, 5350, 1824, 20, 16, (32, 128), True), (5, 3258, 3264, 17, 16, (32, 128), True),
         (1300, 3079, 3616, 17, 128, (128, 128), True)]
IDS = [f"{c[0]}x{c[1]}x{c[2]}-{c[3]}-{c[5][0]}x{c[5][1]}{'-nt' if c[6] else ''}" for c in CASES]


def streams(rows, n, k, E):
    """The kernels' rule for weights that stream past the caches."""
    return E * n * (k // 2) > 64 << 20 and rows <= E * 128


def segments(rng, rows, E, align):
    """Counts and aligned offsets of `rows` rows over E experts, the first without any."""
    lens = rng.multinomial(rows, rng.dirichlet(np.full(E, 2.0)))
    lens[E // 2] += lens[0]
    lens[0] = 0
    offsets = np.concatenate([[0], np.cumsum([-(-c // align) * align for c in lens])]).astype(np.int32)
    return lens, offsets


def on_gpu(codes, sf):
    """float64 values of packed codes (their scale code 255: NaN)."""
    table = torch.from_numpy(ou.E2M1).cuda()
    v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)
    s = torch.where(sf == 255, torch.nan, torch.exp2(sf.double() - 127))
    return v * s.repeat_interleave(32, -1)


@pytest.mark.parametrize("rows,n,k,E,align,tile,nt", CASES, ids=IDS)
def test_padded_segments_by_kernel(rows, n, k, E, align, tile, nt):
    say(f"{rows} rows x {n} x {k}, {E} segments aligned to {align}: tile {tile}{' nt' if nt else ''}")
    assert tuple(moe.moe_gemm_mxfp4_info(rows, n, k, E).values()) == tile and streams(rows, n, k, E) == nt
    rng = np.random.default_rng(rows + n)
    lens, offsets = segments(rng, rows, E, align)
    pool = int(offsets[-1]) + 7                              # seven rows behind the last segment
    a, asf = operand(rng, pool, k, 3)
    b, bsf = operand(rng, E * n, k, 3)
    live = np.zeros(pool, bool)
    for first, c in zip(offsets, lens):
        live[first:first + c] = True
    asf[~live] = 255                                         # what lies outside holds NaN
    a, asf, b, bsf, off, dead = (torch.from_numpy(v).cuda() for v in (a, asf, b, bsf, offsets, ~live))
    counts = torch.tensor(lens, dtype=torch.int32, device="cuda")
    va, vb = on_gpu(a, asf), on_gpu(b, bsf).view(E, n, k)
    ex, mag = torch.full((pool, n), 55.0, dtype=torch.float64, device="cuda"), torch.zeros(pool, n, dtype=torch.float64, device="cuda")
    for e, c in enumerate(lens):
        if c:
            s = slice(offsets[e], offsets[e] + c)
            ex[s], mag[s] = va[s] @ vb[e].t(), va[s].abs() @ vb[e].abs().t()
    # (no sum leaves the range of f16 here, so every difference is a number)
    assert ex.abs().max() < 65504
    for name, dtype in DT.items():
        for slots in (rows, 0, rows + 5):                    # 0: the tile and the launch of the whole pool
            big = torch.full((pool, n + 5), 55.0, dtype=dtype, device="cuda")
            y = big[:, 2:n + 2]
            moe.moe_gemm_mxfp4(a, asf, b.view(E, n, -1), bsf.view(E, n, -1), offsets=off, counts=counts, out=y,
                               slots=slots)
            assert torch.all(big[dead] == 55) and torch.all(big[:, :2] == 55) and torch.all(big[:, n + 2:] == 55)
            off_by, lim = (y.double() - ex).abs(), bound(k, mag, ex, dtype)
            assert torch.all(off_by <= lim), (name, slots, (off_by / lim).nan_to_num().max().item())


# the same sizes, and dense calls of one row, few rows and rows by streamed weights
GRAPHS = [c[:6] for c in CASES] + [(1, 700, 1184, 0, 1, (16, 16)), (29, 3000, 1056, 0, 1, (32, 16)),
                                   (31, 66010, 2080, 0, 1, (32, 128)), (511, 3000, 2144, 0, 1, (64, 128))]


@pytest.mark.parametrize("rows,n,k,E,align,tile", GRAPHS, ids=str)
def test_every_kernel_in_a_graph(rows, n, k, E, align, tile):
    say(f"captured: {rows} rows x {n} x {k}, {E} segments: tile {tile}")
    assert tuple(moe.moe_gemm_mxfp4_info(rows, n, k, E).values()) == tile
    rng = np.random.default_rng(rows)
    g = torch.Generator(device="cuda").manual_seed(rows)
    u = lambda lo, hi, *s: torch.randint(lo, hi, s, dtype=torch.uint8, device="cuda", generator=g)
    pool, kw, lead = rows, {}, ()
    if E:
        lens, offsets = segments(rng, rows, E, align)
        pool, lead = int(offsets[-1]), (E,)
        counts = torch.tensor(lens, dtype=torch.int32, device="cuda")
        kw = dict(offsets=torch.from_numpy(offsets).cuda(), counts=counts, slots=rows)
    a, a_sf = u(0, 256, pool, k // 2), u(120, 134, pool, k // 32)
    b, b_sf = u(0, 256, *lead, n, k // 2), u(120, 134, *lead, n, k // 32)
    y, z = (torch.full((pool, n), 9.0, device="cuda") for _ in range(2))
    run = lambda out: moe.moe_gemm_mxfp4(a, a_sf, b, b_sf, out=out, **kw)
    run(z)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(y)
    for turn in range(4):
        a.copy_(u(0, 256, *a.shape)), a_sf.copy_(u(120, 134, *a_sf.shape))
        if E:                                                # other segments of the same pool
            counts.copy_(torch.from_numpy(np.minimum(lens, rng.integers(0, 1 + max(lens), E))).int())
        y.fill_(turn), z.fill_(turn)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(run(z), y), turn
