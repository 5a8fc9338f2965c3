"""The training operators against plain implementations in 64 bits: grouped
products with both gradients, the gated activation with its gradient, the
orthogonalised update.

Bounds.  A product's FP32 sum truncates once per tensor-core step of 16 k; a
16-bit result takes one chain over all of k, an FP32 result short chains
that are then added.  With S = sum |a||b| that is at most S * 2^-23 per step
(and per addition); 16-bit results add half a step of the result.  The
activation's exponential and divide are good to 2^-18 here (arguments within
+-16), relative to the sum of magnitudes of the formula's terms.  The update:
F16 operands round X, A and P at 2^-12; a CPU simulation of those roundings
over the same distributions gives at most 2.3e-3 of the result's norm, the
BF16 result adds 1.7e-3 (root mean square), so 4e-3 in all.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

# half the gap between neighbours, relative to the value (8, 11, 24 significant bits)
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}


@pytest.fixture(scope="module")
def pkg():
    import group_limited_routed_gb300 as p
    p.lib()
    return p


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dt=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)


def bounds(counts, lead=0):
    off = [lead]
    for c in counts:
        off.append(off[-1] + c)
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def close(got, ref, mag, k):
    """Elementwise |got - ref| within the bound above; mag = sum |a||b|."""
    dt = got.dtype
    steps = (k + 15) // 16 + 8 if dt != torch.float32 else 16 + 8 + (k + 255) // 256
    bound = HALF_STEP[dt] * 1.01 * ref.abs() + TINY[dt] + mag * (2.0 ** -23) * steps
    off = (got.double() - ref).abs()
    assert torch.isfinite(got).all()
    assert (off <= bound).all(), f"{(off - bound).max().item():.3e} over the bound"


def plain_product(x, w, off):
    rows = x.shape[0]
    y = torch.zeros(rows, w.shape[1], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(y)
    o = off.tolist()
    for e in range(len(o) - 1):
        s = slice(o[e], o[e + 1])
        y[s] = x[s].double() @ w[e].double().t()
        mag[s] = x[s].double().abs() @ w[e].double().abs().t()
    return y, mag


def plain_dw(dy, x, off):
    o = off.tolist()
    dw = torch.stack([dy[a:b].double().t() @ x[a:b].double() for a, b in zip(o, o[1:])])
    mag = torch.stack([dy[a:b].double().abs().t() @ x[a:b].double().abs()
                       for a, b in zip(o, o[1:])])
    return dw, mag


GROUPS = [
    [1], [8, 0, 0, 3], [0, 1, 2, 15, 16, 17], [31, 33, 63, 64, 65], [127, 129, 0, 255],
    [256, 257], [0, 0, 700, 0], [513, 5], [0, 0, 0],
]
SIZES = [(64, 64), (256, 128), (1, 8), (8, 1), (136, 520), (100, 257), (255, 1000), (520, 72)]


@pytest.mark.parametrize("counts", GROUPS, ids=str)
@pytest.mark.parametrize("N,K", [(136, 520), (256, 128), (100, 257)])
@pytest.mark.parametrize("out", ["same", "f32"])
def test_products_over_group_sizes(pkg, counts, N, K, out):
    g = gen(len(counts) * 1000 + sum(counts))
    dt = torch.bfloat16
    off = bounds(counts)
    rows = sum(counts)
    E = len(counts)
    x, dy, w = randn(g, rows, K), randn(g, rows, N), randn(g, E, N, K, scale=0.1)
    odt = torch.float32 if out == "f32" else dt
    y, mag = plain_product(x, w, off)
    close(pkg.grouped_matmul(x, w, off, out_dtype=odt), y, mag, K)
    dx, mag = plain_product(dy, w.transpose(1, 2), off)
    close(pkg.grouped_matmul_dx(dy, w, off, out_dtype=odt), dx, mag, N)
    dw, mag = plain_dw(dy, x, off)
    close(pkg.grouped_matmul_dw(dy, x, off, out_dtype=odt), dw, mag, max(counts))


@pytest.mark.parametrize("N,K", SIZES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
def test_products_over_widths(pkg, N, K, dt):
    g = gen(N * 7 + K)
    counts = [5, 0, 40, 70, 300]
    off = bounds(counts)
    rows, E = sum(counts), len(counts)
    x, dy, w = randn(g, rows, K, dt=dt), randn(g, rows, N, dt=dt), randn(g, E, N, K, dt=dt)
    y, mag = plain_product(x, w, off)
    close(pkg.grouped_matmul(x, w, off), y, mag, K)
    close(pkg.grouped_matmul(x, w, off, out_dtype=torch.float32), y, mag, K)
    dx, mag = plain_product(dy, w.transpose(1, 2), off)
    close(pkg.grouped_matmul_dx(dy, w, off), dx, mag, N)
    dw, mag = plain_dw(dy, x, off)
    close(pkg.grouped_matmul_dw(dy, x, off), dw, mag, max(counts))
    close(pkg.grouped_matmul_dw(dy, x, off, out_dtype=torch.float32), dw, mag, max(counts))


@pytest.mark.parametrize("rows", [1, 3, 20, 50, 100, 400])
def test_every_row_tile_over_many_groups(pkg, rows):
    """Mean group sizes on both sides of each tile width, 24 groups, long k."""
    g = gen(rows)
    E, N, K = 24, 264, 1096
    share = torch.rand(E, generator=g, device="cuda").cpu()
    counts = torch.bincount(torch.multinomial(share, rows * E // 4 + rows, replacement=True),
                            minlength=E).tolist()
    off = bounds(counts)
    n = sum(counts)
    x, w = randn(g, n, K), randn(g, E, N, K, scale=0.05)
    y, mag = plain_product(x, w, off)
    close(pkg.grouped_matmul(x, w, off), y, mag, K)
    close(pkg.grouped_matmul(x, w, off, out_dtype=torch.float32), y, mag, K)
    dx, mag = plain_product(y.bfloat16(), w.transpose(1, 2), off)
    close(pkg.grouped_matmul_dx(y.bfloat16(), w, off), dx, mag, N)


@pytest.mark.parametrize("counts", [
    [257, 256, 320], [384, 385, 0, 257], [272], [320, 1, 383, 514, 300, 288, 255, 384],
    [340] * 7], ids=str)
@pytest.mark.parametrize("N,K", [(264, 1096), (136, 72), (129, 513)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
def test_groups_of_two_row_blocks(pkg, counts, N, K, dt):
    """Groups of 257 to 384 rows between others, mean groups of 226 to 340
    rows: one tile of two row blocks; weights read along either axis."""
    g = gen(sum(counts) + N)
    off = bounds(counts)
    E, n = len(counts), sum(counts)
    x, dy = randn(g, n, K, dt=dt), randn(g, n, N, dt=dt)
    for w in (randn(g, E, N, K, dt=dt, scale=0.1),
              randn(g, E, K, N, dt=dt, scale=0.1).transpose(1, 2)):
        y, mag = plain_product(x, w, off)
        close(pkg.grouped_matmul(x, w, off), y, mag, K)
        close(pkg.grouped_matmul(x, w, off, out_dtype=torch.float32), y, mag, K)
        dx, mag = plain_product(dy, w.transpose(1, 2), off)
        close(pkg.grouped_matmul_dx(dy, w, off), dx, mag, N)


@pytest.mark.parametrize("counts", [[257, 256, 320, 384, 385, 0, 300, 290], [340, 1, 300, 383]],
                         ids=str)
@pytest.mark.parametrize("N,K", [(136, 72), (129, 513), (256, 200)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
def test_many_groups_of_two_row_blocks(pkg, counts, N, K, dt):
    """As above with 48 groups: enough of them that the tiles of two blocks
    save a wave of the device's SM pairs."""
    counts = (counts * 12)[:48]
    g = gen(sum(counts) + K)
    off = bounds(counts)
    E, n = len(counts), sum(counts)
    x, dy = randn(g, n, K, dt=dt), randn(g, n, N, dt=dt)
    for w in (randn(g, E, N, K, dt=dt, scale=0.1),
              randn(g, E, K, N, dt=dt, scale=0.1).transpose(1, 2)):
        y, mag = plain_product(x, w, off)
        close(pkg.grouped_matmul(x, w, off), y, mag, K)
        dx, mag = plain_product(dy, w.transpose(1, 2), off)
        close(pkg.grouped_matmul_dx(dy, w, off), dx, mag, N)


@pytest.mark.parametrize("counts", [[130, 127, 1, 0, 65, 100], [257, 600, 0, 31, 513, 129],
                                    [513, 400, 700, 0, 256, 767], [17, 1, 63, 64, 0, 65]], ids=str)
@pytest.mark.parametrize("N,K", [(520, 136), (136, 700)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_products_over_many_groups(pkg, counts, N, K, out):
    """72 groups: more tiles of every height than run at once."""
    counts = counts * 12
    g = gen(sum(counts) + K)
    off = bounds(counts)
    E, n = len(counts), sum(counts)
    x, dy = randn(g, n, K), randn(g, n, N)
    for w in (randn(g, E, N, K, scale=0.1), randn(g, E, K, N, scale=0.1).transpose(1, 2)):
        y, mag = plain_product(x, w, off)
        close(pkg.grouped_matmul(x, w, off, out_dtype=out), y, mag, K)
        dx, mag = plain_product(dy, w.transpose(1, 2), off)
        close(pkg.grouped_matmul_dx(dy, w, off, out_dtype=out), dx, mag, N)


@pytest.mark.parametrize("N", [1, 7, 8, 33, 130, 1000])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_zero_rows_of_any_alignment(pkg, N, out):
    """Rows outside all groups, in outputs of every base and row stride: zeros
    there, and the neighbours of each row stay."""
    g = gen(N)
    off = bounds([3, 0, 5], lead=11)                        # rows 11 .. 19 of 60
    x, w = randn(g, 60, 40), randn(g, 3, N, 40)
    ref, mag = plain_product(x, w, off)
    for at, ld in ((0, N), (1, N + 3), (5, N + 16), (8, N + 8)):
        buf = torch.full((60, ld + at), 7.0, dtype=out, device="cuda")
        pkg.grouped_matmul(x, w, off, out=buf[:, at:at + N])
        close(buf[:, at:at + N].contiguous(), ref, mag, 40)
        assert (buf[:11, at:at + N] == 0).all() and (buf[19:, at:at + N] == 0).all()
        assert (buf[:, :at] == 7).all() and (buf[:, at + N:] == 7).all()


def test_long_sums_in_32_bits(pkg):
    """FP32 results over a long k stay at FP32 accuracy (short chains, added in FP32)."""
    g = gen(5)
    off = bounds([130, 20])
    x, w = randn(g, 150, 8192), randn(g, 2, 64, 8192)
    y, _ = plain_product(x, w, off)
    got = pkg.grouped_matmul(x, w, off, out_dtype=torch.float32).double()
    assert ((got - y).norm() / y.norm()).item() < 1e-6
    off = bounds([20000, 480])
    dy, x = randn(g, 20480, 64), randn(g, 20480, 72)
    dw, _ = plain_dw(dy, x, off)
    got = pkg.grouped_matmul_dw(dy, x, off, out_dtype=torch.float32).double()
    assert ((got - dw).norm() / dw.norm()).item() < 1e-6


def test_strides_views_and_unaligned_bases(pkg):
    g = gen(11)
    counts = [17, 0, 90, 5]
    off = bounds(counts)
    rows, E, N, K = sum(counts), 4, 72, 200
    wide = randn(g, rows, 2 * K + 16)
    wt = randn(g, E, K, N, scale=0.1)                       # stored [E, K, N]
    big = randn(g, E, N, K + 3, scale=0.1)
    dy = randn(g, rows, N + 5)
    for x in (wide[:, :K], wide[:, K:2 * K], wide[:, 3:3 + K]):
        for w in (wt.transpose(1, 2), big[:, :, :K], big[:, :, 1:1 + K], wt[:1].transpose(1, 2).expand(E, N, K)):
            y, mag = plain_product(x, w, off)
            close(pkg.grouped_matmul(x, w, off), y, mag, K)
            for d in (dy[:, :N], dy[:, 1:1 + N]):
                dx, mag = plain_product(d, w.transpose(1, 2), off)
                close(pkg.grouped_matmul_dx(d, w, off), dx, mag, N)
        for d in (dy[:, :N], dy[:, 1:1 + N]):
            dw, mag = plain_dw(d, x, off)
            close(pkg.grouped_matmul_dw(d, x, off), dw, mag, 90)
    # an output that is part of a wider buffer: its neighbours stay
    buf = torch.full((rows, N + 7), 7.0, dtype=torch.bfloat16, device="cuda")
    x, w = wide[:, :K], wt.transpose(1, 2)
    y, mag = plain_product(x, w, off)
    pkg.grouped_matmul(x, w, off, out=buf[:, 2:2 + N])
    close(buf[:, 2:2 + N].contiguous(), y, mag, K)
    assert (buf[:, :2] == 7).all() and (buf[:, 2 + N:] == 7).all()


def test_rows_outside_groups_and_foreign_rows(pkg):
    """Rows outside all groups give zeros; NaN and infinities there and in
    other groups stay where they are."""
    g = gen(13)
    off = bounds([20, 0, 37], lead=9)                       # rows 9 .. 66 of 80
    x, dy, w = randn(g, 80, 128), randn(g, 80, 72), randn(g, 3, 72, 128, scale=0.1)
    for t in (x, dy):
        t[:9] = float("nan")
        t[66:] = float("inf")
    ref = plain_product(torch.nan_to_num(x, 0, 0, 0), w, off)
    y = pkg.grouped_matmul(x, w, off)
    assert (y[:9] == 0).all() and (y[66:] == 0).all()
    close(y[9:66], ref[0][9:66], ref[1][9:66], 128)
    y32 = pkg.grouped_matmul(x, w, off, out_dtype=torch.float32)
    assert (y32[:9] == 0).all() and (y32[66:] == 0).all()
    dw, mag = plain_dw(torch.nan_to_num(dy, 0, 0, 0), torch.nan_to_num(x, 0, 0, 0), off)
    close(pkg.grouped_matmul_dw(dy, x, off), dw, mag, 37)
    # a NaN row spoils its own row and its own group's gradient, nothing else
    x[9:29] = float("nan")
    y = pkg.grouped_matmul(x, w, off)
    assert torch.isnan(y[9:29]).all() and torch.isfinite(y[29:66]).all()
    got = pkg.grouped_matmul_dw(dy, x, off)
    assert torch.isnan(got[0]).all() and (got[1] == 0).all()
    close(got[2], dw[2], mag[2], 37)


def test_weight_gradient_accumulates(pkg):
    g = gen(17)
    off = bounds([30, 0, 300])
    dy, x = randn(g, 330, 96), randn(g, 330, 264)
    dw, mag = plain_dw(dy, x, off)
    acc = torch.randn(3, 96, 264, generator=g, device="cuda")
    start = acc.double()
    pkg.grouped_matmul_dw(dy, x, off, out=acc, accumulate=True)
    assert (acc[1].double() == start[1]).all()
    close(acc, start + dw, mag + start.abs(), 300)
    none = torch.zeros(4, dtype=torch.int32, device="cuda")
    out = torch.full((3, 96, 264), 3.0, device="cuda")
    pkg.grouped_matmul_dw(dy[:0], x[:0], none, out=out)
    assert (out == 0).all()


@pytest.mark.parametrize("counts", [[5000], [3000, 0, 70, 2000, 1], [64, 9000, 63], [1024, 1025, 2111]],
                         ids=str)
@pytest.mark.parametrize("N,K", [(136, 520), (1, 257), (600, 33)])
def test_weight_gradients_over_many_rows(pkg, counts, N, K):
    """Few tiles with long sums: the rows are taken in parts, added in order."""
    g = gen(sum(counts) + N)
    off = bounds(counts)
    dy, x = randn(g, sum(counts), N), randn(g, sum(counts), K)
    ref, mag = plain_dw(dy, x, off)
    n = max(counts)
    close(pkg.grouped_matmul_dw(dy, x, off), ref, mag, n)
    got = pkg.grouped_matmul_dw(dy, x, off, out_dtype=torch.float32)
    close(got, ref, mag, n)
    assert (got[[c == 0 for c in counts]] == 0).all()
    assert torch.equal(got, pkg.grouped_matmul_dw(dy, x, off, out_dtype=torch.float32))
    base = randn(g, len(counts), N, K, dt=torch.float32)
    total = base.clone()
    pkg.grouped_matmul_dw(dy, x, off, out=total, accumulate=True)
    close(total, ref + base.double(), mag + base.double().abs(), n)


def test_weight_gradient_in_a_smaller_workspace(pkg):
    """Room for some of the parts or none: fewer are taken."""
    g = gen(71)
    off = bounds([9000])
    dy, x = randn(g, 9000, 136), randn(g, 9000, 264)
    ref, mag = plain_dw(dy, x, off)
    full = pkg.grouped_matmul_workspace_size(9000, 1, 136, 264)
    assert full > 136 * 264 * 8
    for nbytes in (4096, 136 * 264 * 8 + 8192, full):
        ws = pkg.OpWorkspace(nbytes)
        close(pkg.grouped_matmul_dw(dy, x, off, out_dtype=torch.float32, ws=ws), ref, mag, 9000)
        close(pkg.grouped_matmul_dw(dy, x, off, ws=ws), ref, mag, 9000)


@pytest.mark.parametrize("N,K", [(264, 1096), (129, 513), (1, 1), (513, 7)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_gradients_of_groups_without_rows(pkg, N, K, out):
    """Zeros over whatever the output held, next to groups with rows."""
    g = gen(N + K)
    counts = [0, 9, 0, 0, 1, 0]
    off = bounds(counts)
    dy, x = randn(g, 10, N), randn(g, 10, K)
    ref, mag = plain_dw(dy, x, off)
    buf = torch.full((6, N, K), float("nan"), dtype=out, device="cuda")
    pkg.grouped_matmul_dw(dy, x, off, out=buf)
    close(buf, ref, mag, 9)


def test_gradients_against_differences(pkg):
    """The products are linear: the gradient along a direction equals the
    central difference, up to FP32 sums."""
    g = gen(19)
    counts = [12, 0, 45, 7]
    off = bounds(counts)
    rows, E, N, K = 64, 4, 80, 136
    x, w, c = randn(g, rows, K), randn(g, E, N, K), randn(g, rows, N)
    d = (torch.randint(-2, 3, (rows, K), generator=g, device="cuda") * 0.5).bfloat16()
    f = lambda a: (pkg.grouped_matmul(a, w, off, out_dtype=torch.float32).double() * c.double()).sum()
    # integer-valued inputs, so that x + d and x - d are exact
    xi = torch.randint(-8, 9, (rows, K), generator=g, device="cuda").bfloat16()
    diff = (f(xi + d) - f(xi - d)) / 2
    dx = pkg.grouped_matmul_dx(c, w, off, out_dtype=torch.float32).double()
    scale = (dx.abs() * d.double().abs()).sum()
    assert abs((dx * d.double()).sum() - diff) <= 1e-5 * scale
    wi = torch.randint(-8, 9, (E, N, K), generator=g, device="cuda").bfloat16()
    dd = (torch.randint(-2, 3, (E, N, K), generator=g, device="cuda") * 0.5).bfloat16()
    h = lambda a: (pkg.grouped_matmul(x, a, off, out_dtype=torch.float32).double() * c.double()).sum()
    diff = (h(wi + dd) - h(wi - dd)) / 2
    dw = pkg.grouped_matmul_dw(c, x, off, out_dtype=torch.float32).double()
    scale = (dw.abs() * dd.double().abs()).sum()
    assert abs((dw * dd.double()).sum() - diff) <= 1e-5 * scale


def test_boundaries_out_of_order_are_reported(pkg):
    g = gen(23)
    x, w = randn(g, 40, 64), randn(g, 3, 64, 64)
    ws = pkg.OpWorkspace(pkg.grouped_matmul_workspace_size(40, 3, 64, 64))
    good = bounds([10, 20, 10])
    ref = pkg.grouped_matmul(x, w, good, ws=ws)
    assert pkg.check_status(ws) == 0
    for bad in ([0, 30, 10, 40], [0, 10, 30, 4000], [-5, 10, 30, 40]):
        pkg.grouped_matmul(x, w, torch.tensor(bad, dtype=torch.int32, device="cuda"), ws=ws)
        assert pkg.check_status(ws) == 6, bad
    assert torch.equal(pkg.grouped_matmul(x, w, good, ws=ws), ref)
    assert pkg.check_status(ws) == 0


def test_repeats_streams_and_graphs(pkg):
    """Bit-identical results call after call, on another stream and replayed."""
    g = gen(29)
    off = bounds([100, 3, 0, 150])
    x, w, dy = randn(g, 253, 264), randn(g, 4, 136, 264), randn(g, 253, 136)
    m = randn(g, 2, 80, 200)
    ws = pkg.OpWorkspace(pkg.grouped_matmul_workspace_size(253, 4, 136, 264))
    ows = pkg.OpWorkspace(pkg.orthogonalize_workspace_size(2, 80, 200))

    def calls():
        return [pkg.grouped_matmul(x, w, off, ws=ws), pkg.grouped_matmul_dx(dy, w, off, ws=ws),
                pkg.grouped_matmul_dw(dy, x, off, ws=ws), pkg.swiglu(dy, dy),
                pkg.orthogonalize(m, ws=ows)]
    first = calls()
    for a, b in zip(first, calls()):
        assert torch.equal(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = calls()
    s.synchronize()
    for a, b in zip(first, other):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    for t in held:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, held):
        assert torch.equal(a, b)


def test_a_stream_of_the_callers_choice(pkg):
    """Outputs and workspaces that the call itself allocates belong to the
    stream it runs on, also when that is not the current one."""
    g = gen(31)
    counts = [9, 0, 61, 130]
    off = bounds(counts)
    x, w, dy = randn(g, 200, 131), randn(g, 4, 65, 131), randn(g, 200, 65)  # copies needed
    m = randn(g, 2, 3, 40, 70).transpose(0, 1)                              # a copy needed
    want = [pkg.grouped_matmul(x, w, off), pkg.grouped_matmul_dx(dy, w, off),
            pkg.grouped_matmul_dw(dy, x, off), pkg.swiglu(dy, dy),
            pkg.swiglu_grad(dy, dy, dy)[0], pkg.orthogonalize(m)]
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        s.wait_stream(torch.cuda.current_stream())
        got = [pkg.grouped_matmul(x, w, off, stream=stream),
               pkg.grouped_matmul_dx(dy, w, off, stream=stream),
               pkg.grouped_matmul_dw(dy, x, off, stream=stream),
               pkg.swiglu(dy, dy, stream=stream),
               pkg.swiglu_grad(dy, dy, dy, stream=stream)[0],
               pkg.orthogonalize(m, stream=stream)]
        s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_no_group_has_a_row(pkg):
    g = gen(37)
    x, dy, w = randn(g, 5, 64), randn(g, 5, 32), randn(g, 3, 32, 64)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert (pkg.grouped_matmul(x, w, off) == 0).all()
    assert (pkg.grouped_matmul_dx(dy, w, off, out_dtype=torch.float32) == 0).all()
    assert (pkg.grouped_matmul_dw(dy, x, off) == 0).all()
    assert (pkg.grouped_matmul_dw(dy, x, off, out_dtype=torch.float32) == 0).all()


def test_back_to_back_calls_wait_for_one_another(pkg):
    """Calls launched early behind one another (programmatic serialization)
    read what the call before wrote: a chain equals its single steps."""
    g = gen(41)
    off = bounds([33, 0, 90, 5])
    x, w = randn(g, 128, 256), randn(g, 4, 256, 256, scale=0.05)
    m = randn(g, 3, 100, 160)

    def chain(wait):
        y = x
        out = []
        for _ in range(4):
            y = pkg.grouped_matmul(y, w, off)
            wait()
            h = pkg.swiglu(y, y)
            wait()
            y = pkg.grouped_matmul_dx(h, w, off)
            wait()
            out.append(pkg.grouped_matmul_dw(h, y, off))
            wait()
        out.append(pkg.orthogonalize(pkg.orthogonalize(m)))
        wait()
        out.append(pkg.orthogonalize(out[0][:, :200].contiguous()))
        return out + [y]
    single = chain(torch.cuda.synchronize)
    for _ in range(3):
        for a, b in zip(single, chain(lambda: None)):
            assert torch.equal(a, b)


# -------------------------------------------------------------- activation
def plain_gate(g, u, w):
    return w[:, None] * g * torch.sigmoid(g) * u


@pytest.mark.parametrize("rows,F", [(1, 1), (1, 2560), (7, 8), (3, 257), (64, 256), (33, 1001),
                                    (2500, 264), (5000, 40)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("weighted", [True, False])
def test_gated_activation_and_gradient(pkg, rows, F, dt, weighted):
    gg = gen(rows + F)
    g, u = randn(gg, rows, F, dt=dt, scale=2.0), randn(gg, rows, F, dt=dt)
    dh = randn(gg, rows, F, dt=dt)
    w = torch.rand(rows, generator=gg, device="cuda") + 0.1 if weighted else None
    G, U, D = g.double(), u.double(), dh.double()
    W = w.double() if weighted else torch.ones(rows, dtype=torch.float64, device="cuda")
    h = plain_gate(G, U, W)
    eps = 2.0 ** -18

    def near(got, ref, mag):
        off = (got.double() - ref).abs()
        assert (off <= HALF_STEP[got.dtype] * 1.01 * ref.abs() + TINY[got.dtype] + eps * mag).all()
    near(pkg.swiglu(g, u, w), h, h.abs())
    got = pkg.swiglu_grad(dh, g, u, w)
    s = torch.sigmoid(G)
    base = D * W[:, None] * U * s
    near(got[0], base * (1 + G * (1 - s)), base.abs() * (1 + G.abs()))
    du = D * W[:, None] * G * s
    near(got[1], du, du.abs())
    if weighted:
        terms = D * G * s * U
        near(got[2], terms.sum(1), terms.abs().sum(1))
    else:
        assert len(got) == 2
    # the formulas against central differences of the plain forward, in 64 bits
    t = 1e-5
    num = (plain_gate(G + t, U, W) - plain_gate(G - t, U, W)) / (2 * t) * D
    near(got[0], num, base.abs() * (1 + G.abs()) + 1e-4)


def test_gated_activation_extremes_and_strides(pkg):
    """Large arguments saturate, infinities behave as the formula's limits,
    NaN stays in its element (and its row's weight gradient)."""
    v = [0.0, -0.0, 80.0, -80.0, 1000.0, -1000.0, 3e38, -3e38, 1.5, float("inf"), float("nan")]
    g = torch.tensor([v + [0.5] * 5], device="cuda").bfloat16()
    u = torch.ones_like(g)
    h = pkg.swiglu(g, u).float()
    ref = (g.float() * (1 / (1 + torch.exp(-g.float())))).bfloat16().float()
    assert torch.equal(torch.isnan(h), torch.isnan(ref))
    ok = ~torch.isnan(ref)
    assert torch.allclose(h[ok], ref[ok], rtol=2 ** -8, atol=1e-30)
    gg = gen(3)
    both = randn(gg, 40, 2 * 48)
    dh = randn(gg, 40, 50)[:, 1:49]
    w = torch.rand(40, generator=gg, device="cuda")
    g, u = both[:, :48], both[:, 48:]
    want = pkg.swiglu_grad(dh.contiguous(), g.contiguous(), u.contiguous(), w)
    out = torch.empty(40, 96, dtype=torch.bfloat16, device="cuda")
    got = pkg.swiglu_grad(dh, g, u, w, out=(out[:, :48], out[:, 48:]))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    keep = both.clone()
    pkg.swiglu_grad(dh, g, u, w, out=(g, u))                # in place
    assert torch.equal(both, out) and not torch.equal(both, keep)
    assert pkg.swiglu(both[:0, :48], both[:0, 48:]).shape == (0, 48)


# -------------------------------------------------------------- the update
COEFFS = (3.4445, -4.7750, 2.0315)


def plain_update(m, steps=5, coeffs=COEFFS, eps=1e-7):
    a, b, c = coeffs
    x = m.double()
    x = x / (x.norm() + eps)
    for _ in range(steps):
        q = x @ x.t()
        x = a * x + (b * q + c * (q @ q)) @ x
    return x


def momentum(g, b, R, C, dt):
    k = max(1, min(R, C) // 16)
    m = torch.randn(b, R, k, generator=g, device="cuda") @ torch.randn(b, k, C, generator=g, device="cuda")
    m = m / math.sqrt(k) + 0.3 * torch.randn(b, R, C, generator=g, device="cuda")
    return (m * 1e-3).to(dt)


@pytest.mark.parametrize("b,R,C", [(1, 1, 1), (1, 1, 40), (3, 40, 1), (2, 16, 16), (1, 64, 512),
                                   (2, 33, 100), (2, 100, 33), (1, 257, 300), (3, 300, 257),
                                   (1, 512, 512), (1, 640, 1290), (1, 1290, 640), (40, 96, 40),
                                   (12, 520, 600), (12, 600, 520)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32],
                         ids=["bf16", "f16", "f32"])
def test_update_over_shapes(pkg, b, R, C, dt):
    m = momentum(gen(R * 31 + C + b), b, R, C, dt)
    got = pkg.orthogonalize(m)
    assert got.dtype == (dt if dt != torch.float32 else torch.bfloat16) and got.shape == m.shape
    for i in range(b):
        ref = plain_update(m[i])
        off = ((got[i].double() - ref).norm() / ref.norm()).item()
        assert off <= 4e-3, (i, off)


@pytest.mark.parametrize("b,R,C", [(1, 64, 384), (1, 64, 385), (1, 65, 384), (2, 64, 513),
                                   (1, 50, 1025), (1, 64, 4096), (1, 17, 8192), (1, 30, 8200),
                                   (1, 120, 5120), (17, 64, 700), (5, 2500, 60), (40, 7, 600),
                                   (20, 128, 512), (160, 64, 100)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_update_over_small_extents(pkg, b, R, C, dt):
    """Both tile heights, one CTA and clusters of every size, more clusters
    than the device runs at once, widths just past one launch's limit."""
    m = momentum(gen(R * 31 + C + b), b, R, C, dt)
    got = pkg.orthogonalize(m)
    for i in range(b):
        ref = plain_update(m[i])
        off = ((got[i].double() - ref).norm() / ref.norm()).item()
        assert off <= 4e-3, (i, off)


def test_update_steps_coefficients_and_layouts(pkg):
    g = gen(7)
    m = momentum(g, 2, 96, 160, torch.bfloat16)
    for steps, coeffs in ((1, COEFFS), (2, COEFFS), (8, (2.0, -1.5, 0.5)), (6, (1.875, -1.25, 0.375))):
        got = pkg.orthogonalize(m, steps=steps, coeffs=coeffs)
        for i in range(2):
            ref = plain_update(m[i], steps, coeffs)
            assert ((got[i].double() - ref).norm() / ref.norm()).item() <= 4e-3, (steps, coeffs)
    want = pkg.orthogonalize(m)
    big = torch.zeros(2, 100, 200, dtype=torch.bfloat16, device="cuda")
    big[:, 2:98, 5:165] = m
    assert torch.equal(pkg.orthogonalize(big[:, 2:98, 5:165]), want)
    t = m.transpose(1, 2).contiguous().transpose(1, 2)      # column-major storage
    assert torch.equal(pkg.orthogonalize(t), want)
    assert torch.equal(pkg.orthogonalize(m[0]), want[0])
    assert torch.equal(pkg.orthogonalize(m.view(2, 1, 96, 160)), want.view(2, 1, 96, 160))
    assert pkg.orthogonalize(m[:0]).shape == (0, 96, 160)
    assert pkg.orthogonalize(m, out_dtype=torch.float16).dtype == torch.float16


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1.0, 1e15, 1e30])
def test_update_over_magnitudes(pkg, scale):
    """The norm neither over- nor underflows: with eps 0 the result does not
    depend on the update's magnitude."""
    m = momentum(gen(9), 1, 48, 80, torch.float32) * scale
    got = pkg.orthogonalize(m, eps=0.0)[0].double()
    ref = plain_update(m[0], eps=0.0)
    assert ((got - ref).norm() / ref.norm()).item() <= 4e-3


def test_update_of_degenerate_matrices(pkg):
    z = torch.zeros(3, 40, 72, dtype=torch.bfloat16, device="cuda")
    z[1] = momentum(gen(1), 1, 40, 72, torch.bfloat16)[0]
    z[2, 3, 5] = 2.0                                        # rank one
    got = pkg.orthogonalize(z)
    assert (got[0] == 0).all()
    ref = plain_update(z[2])
    assert ((got[2].double() - ref).norm() / ref.norm()).item() <= 4e-3
    alone = pkg.orthogonalize(z[1:2])
    assert torch.equal(got[1], alone[0])
    for v in (float("nan"), float("inf")):
        z[0, 7, 7] = v
        got = pkg.orthogonalize(z)
        assert torch.isnan(got[0]).all() and torch.equal(got[1], alone[0])


def test_refusals(pkg):
    g = gen(2)
    x, w = randn(g, 10, 64), randn(g, 2, 32, 64)
    off = bounds([4, 6])
    dy = randn(g, 10, 32)
    with pytest.raises(TypeError):
        pkg.grouped_matmul(x.float(), w.float(), off)
    with pytest.raises(TypeError):
        pkg.grouped_matmul(x, w.half(), off)
    with pytest.raises(TypeError):
        pkg.grouped_matmul(x, w, off.long())
    with pytest.raises(TypeError):
        pkg.grouped_matmul(x, w, off, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        pkg.grouped_matmul(x.cpu(), w, off)
    with pytest.raises(ValueError):
        pkg.grouped_matmul(x[:, :32], w, off)
    with pytest.raises(ValueError):
        pkg.grouped_matmul(x, w, bounds([10]))
    with pytest.raises(ValueError):
        pkg.grouped_matmul(x.t().contiguous().t(), w, off)
    with pytest.raises(ValueError):
        pkg.grouped_matmul(x, w[:, ::2, ::2], off)
    with pytest.raises(ValueError):
        pkg.grouped_matmul(x, w, off, out=torch.empty(9, 32, dtype=x.dtype, device="cuda"))
    with pytest.raises(ValueError):
        pkg.grouped_matmul_dw(dy, x[:5], off)
    with pytest.raises(ValueError):
        pkg.grouped_matmul_dw(dy, x, off, accumulate=True)
    small = pkg.OpWorkspace(256)
    with pytest.raises(pkg.BeamError) as err:
        pkg.grouped_matmul(randn(g, 10, 65)[:, 1:], w, off, ws=small)
    assert err.value.code == 3
    with pytest.raises(TypeError):
        pkg.swiglu(x.float(), x.float())
    with pytest.raises(ValueError):
        pkg.swiglu(x, x[:5])
    with pytest.raises(ValueError):
        pkg.swiglu(x, x, torch.ones(9, device="cuda"))
    m = randn(g, 40, 40)
    with pytest.raises(TypeError):
        pkg.orthogonalize(m, out_dtype=torch.float32)
    for kw in (dict(steps=0), dict(steps=65), dict(eps=-1.0), dict(eps=float("nan")),
               dict(coeffs=(float("nan"), 0, 0)), dict(coeffs=(17.0, 0, 0))):
        with pytest.raises(pkg.BeamError) as err:
            pkg.orthogonalize(m, **kw)
        assert err.value.code == 1, kw
    with pytest.raises(pkg.BeamError) as err:
        pkg.orthogonalize(m, ws=small)
    assert err.value.code == 3
