"""moe_permute, moe_combine and moe_combine_backward on the GPU, against plain 64-bit forms (rows_ref), and the
gradients against differences.

fp32 sums of k products in order are off by at most (k + 2) 2^-24 of the sum of magnitudes; a bf16 output adds half a
step, 2^-8 of its value.
"""
import numpy as np
import pytest
import torch

import rows_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _case(T, E, k, N, seed):
    g = _gen(seed)
    logits = torch.randn(T, E, generator=g)
    return g, logits, torch.randn(T, N, generator=g)


def _close(got, want, S, k, dtype):
    err = (k + 2) * 2.0 ** -24 * S
    if dtype == BF16:
        err = err + 2.0 ** -8 * (np.abs(want) + err)
    assert np.all(np.abs(ref.f64(got) - want) <= err)


SHAPES = [(1, 8, 8, 2048), (1, 2, 1, 1), (5, 7, 3, 8), (64, 256, 8, 2048), (33, 16, 4, 1111), (9, 4, 2, 250), (3, 40, 8, 2056),
          (2, 5, 5, 4099), (7, 5, 3, 257), (6, 9, 4, 511), (4, 6, 6, 769), (40, 16, 2, 255), (20, 4, 1, 513), (11, 3, 2, 3)]


@pytest.mark.parametrize("T,E,k,N", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_there_and_back(nv, T, E, k, N, dtype):
    g, logits, x = _case(T, E, k, N, T + N)
    ids, w, offsets, lst = nv.moe_route_topk(logits.cuda(), k)
    x = x.to(dtype)
    rows, pos = nv.moe_permute(x.cuda(), lst, k)
    want_pos = np.full(T * k, -1)
    want = ref.permute(ref.f64(x), lst.cpu().numpy(), k, want_pos)
    assert np.array_equal(ref.f64(rows), want) and np.array_equal(pos.cpu().numpy(), want_pos)
    back = torch.randn(T * k, N, generator=g).to(dtype)
    add = torch.randn(T, N, generator=g).to(BF16)
    wn = ref.f64(w)
    for out in (BF16, F32):
        for use_w in (True, False):
            for use_pos in (True, False):
                for use_add in (True, False):
                    y, S = ref.combine(ref.f64(back), wn if use_w else None, want_pos if use_pos else None,
                                       ref.f64(add) if use_add else None, T, k)
                    got = nv.moe_combine(back.cuda(), k, w if use_w else None, pos if use_pos else None,
                                         add=add.cuda() if use_add else None, out_dtype=out)
                    _close(got, y, S, k, out)
    for dy_type in (BF16, F32):
        dy = torch.randn(T, N, generator=g).to(dy_type)
        want_rows = np.zeros((T * k, N))
        d_w, S = ref.combine_backward(ref.f64(dy), ref.f64(back), wn, want_pos, T, k, want_rows)
        got_rows, got_w = nv.moe_combine_backward(dy.cuda(), back.cuda(), w, pos)
        _close(got_rows, want_rows, np.abs(want_rows), 0, dtype)
        # a chain of at most N / 256 / 8 * 8 + 8 fused additions a thread, 5 over the lanes, 8 over the warps
        assert np.all(np.abs(ref.f64(got_w) - d_w) <= (N / 256 + 8 + 13) * 2.0 ** -24 * S)
    d_x, S = ref.combine(ref.f64(back), None, want_pos, None, T, k)
    _close(nv.moe_combine(back.cuda(), k, None, pos, out_dtype=F32), d_x, S, k, F32)


def test_more_entries_than_the_router_gives(nv):
    """Up to 8 entries come from moe_route_topk; other routers have more, or one."""
    for T, k, N in ((3, 17, 136), (2, 33, 77), (4, 1, 64)):
        g = _gen(k)
        lst = torch.randperm(T * k, generator=g).to(torch.int32)
        x, back = torch.randn(T, N, generator=g), torch.randn(T * k, N, generator=g)
        w, dy = torch.randn(T, k, generator=g), torch.randn(T, N, generator=g)
        rows, pos = nv.moe_permute(x.cuda(), lst.cuda(), k)
        p = np.full(T * k, -1)
        assert np.array_equal(ref.f64(rows), ref.permute(ref.f64(x), lst.numpy(), k, p))
        y, S = ref.combine(ref.f64(back), ref.f64(w), p, None, T, k)
        _close(nv.moe_combine(back.cuda(), k, w.cuda(), pos, out_dtype=F32), y, S, k, F32)
        want_rows = np.zeros((T * k, N))
        d_w, S = ref.combine_backward(ref.f64(dy), ref.f64(back), ref.f64(w), p, T, k, want_rows)
        d_rows, got = nv.moe_combine_backward(dy.cuda(), back.cuda(), w.cuda(), pos)
        _close(d_rows, want_rows, np.abs(want_rows), 0, F32)
        assert np.all(np.abs(ref.f64(got) - d_w) <= (N / 256 + 21) * 2.0 ** -24 * S)


def test_gradients_against_differences(nv):
    """L = <c, combine(rows, w)> is linear in rows and in w: differences of exactly representable values are the
    gradients, up to the roundings of two fp32 results."""
    T, k, N = 4, 3, 24
    g = _gen(11)
    ints = lambda *s: torch.randint(-4, 5, s, generator=g).float()  # noqa: E731
    lst = torch.randperm(T * k, generator=g).to(torch.int32).cuda()
    x, w, rows, c = ints(T, N), ints(T, k), ints(T * k, N), ints(T, N)
    _, pos = nv.moe_permute(x.cuda(), lst, k)
    loss = lambda r, v: float((nv.moe_combine(r.cuda(), k, v.cuda(), pos, out_dtype=F32).cpu() * c).sum())  # noqa: E731
    d_rows, d_w = nv.moe_combine_backward(c.cuda(), rows.cuda(), w.cuda(), pos)
    base = loss(rows, w)
    for r, n in ((0, 0), (5, 23), (11, 7)):
        at = rows.clone()
        at[r, n] += 1
        assert loss(at, w) - base == float(d_rows[r, n])
    for t in range(T):
        for j in range(k):
            at = w.clone()
            at[t, j] += 1
            assert loss(rows, at) - base == float(d_w[t, j])
    # permute's: L = <c2, permute(x)>
    c2 = ints(T * k, N)
    d_x = nv.moe_combine(c2.cuda(), k, None, pos, out_dtype=F32).cpu()
    first = lambda v: float((nv.moe_permute(v.cuda(), lst, k)[0].cpu() * c2).sum())  # noqa: E731
    for t, n in ((0, 0), (3, 23), (2, 9)):
        at = x.clone()
        at[t, n] += 1
        assert first(at) - first(x) == float(d_x[t, n])


def test_entries_left_out_and_bad_ones(nv):
    """A list with entries outside [0, T*k): rows of zeros, positions and rows that nothing names left as they were."""
    T, k, N = 6, 2, 40
    g = _gen(3)
    lst = torch.tensor([3, -1, 11, 0, 12, 2, 1 << 30, 7, 8, -(1 << 31), 10, 1], dtype=torch.int32)
    x = torch.randn(T, N, generator=g).to(BF16)
    rows, pos = nv.moe_permute(x.cuda(), lst.cuda(), k)
    p = np.full(T * k, -1)
    assert np.array_equal(ref.f64(rows), ref.permute(ref.f64(x), lst.numpy(), k, p)) and np.array_equal(pos.cpu().numpy(), p)
    mine = torch.full((T * k,), 77, dtype=torch.int32, device="cuda")
    nv.moe_permute(x.cuda(), lst.cuda(), k, positions=mine)
    assert np.array_equal(mine.cpu().numpy(), np.where(p < 0, 77, p))
    w, back = torch.randn(T, k, generator=g), torch.randn(T * k, N, generator=g)
    for positions in (pos, mine):
        y, S = ref.combine(ref.f64(back), ref.f64(w), positions.cpu().numpy(), None, T, k)
        _close(nv.moe_combine(back.cuda(), k, w.cuda(), positions, out_dtype=F32), y, S, k, F32)
        d_rows = torch.full((T * k, N), 5.0, device="cuda")
        want = np.full((T * k, N), 5.0)
        d_w, _ = ref.combine_backward(ref.f64(x), ref.f64(back), ref.f64(w), positions.cpu().numpy(), T, k, want)
        _, got = nv.moe_combine_backward(x.cuda(), back.cuda(), w.cuda(), positions, d_rows=d_rows)
        _close(d_rows, want, np.abs(want), 0, F32)
        left = (positions.cpu().numpy().reshape(T, k) < 0) | (positions.cpu().numpy().reshape(T, k) >= T * k)
        assert left.any() and not got.cpu().numpy()[left].any()
    fresh, _ = nv.moe_combine_backward(x.cuda(), back.cuda(), w.cuda(), pos)
    assert not fresh.cpu().numpy()[np.setdiff1d(np.arange(T * k), p)].any()


def test_in_place_nan_and_the_same_bits_every_time(nv):
    T, E, k, N = 300, 64, 8, 1000
    g, logits, x = _case(T, E, k, N, 9)
    ids, w, offsets, lst = nv.moe_route_topk(logits.cuda(), k)
    _, pos = nv.moe_permute(x.cuda(), lst, k)
    back, dy = torch.randn(T * k, N, generator=g).to(BF16).cuda(), torch.randn(T, N, generator=g).to(BF16).cuda()
    add = torch.randn(T, N, generator=g).to(BF16).cuda()
    first = nv.moe_combine(back, k, w, pos, add=add), *nv.moe_combine_backward(dy, back, w, pos)
    for _ in range(3):
        again = nv.moe_combine(back, k, w, pos, add=add), *nv.moe_combine_backward(dy, back, w, pos)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    y = add.clone()
    assert nv.moe_combine(back, k, w, pos, add=y, y=y) is y and torch.equal(y, first[0])
    rows = back.clone()
    nv.moe_combine_backward(dy, rows, w, pos, d_rows=rows)
    assert torch.equal(rows, first[1])
    # a NaN or an infinity in a row reaches its own token alone
    bad = back.clone()
    bad[int(pos[5 * k]), 3], bad[int(pos[7 * k + 1]), 4] = float("nan"), float("inf")
    y = nv.moe_combine(bad, k, w, pos, add=add)
    changed = (y != first[0]) | y.isnan()
    assert changed.nonzero().tolist() == [[5, 3], [7, 4]] and y[5, 3].isnan() and y[7, 4].isinf()


@pytest.mark.parametrize("N", [1, 63, 255, 257, 511, 513, 1025])
def test_odd_lengths_in_place_and_between_others(nv, N):
    """Rows of an odd length share 4-byte words with their neighbours: every element is written, once, none beside the
    tensor, and in place the same."""
    T, E, k = 37, 16, 3
    g, logits, x = _case(T, E, k, N, N)
    ids, w, offsets, lst = nv.moe_route_topk(logits.cuda(), k)
    x = x.to(BF16).cuda()

    def inside(rows):
        buf = torch.full((rows * N + 16,), 7.0, dtype=BF16, device="cuda")
        return buf, buf[:rows * N].view(rows, N)
    buf, rows = inside(T * k)
    _, pos = nv.moe_permute(x, lst, k, rows=rows)
    assert torch.equal(rows, x[lst.long() // k]) and (buf[-16:] == 7).all()
    back, dy = torch.randn(T * k, N, generator=g).to(BF16).cuda(), torch.randn(T, N, generator=g).to(BF16).cuda()
    buf, y = inside(T)
    y.copy_(x)
    nv.moe_combine(back, k, w, pos, add=y, y=y)
    assert torch.equal(y, nv.moe_combine(back, k, w, pos, add=x)) and (buf[-16:] == 7).all()
    d_rows, d_w = nv.moe_combine_backward(dy, back, w, pos)
    buf, here = inside(T * k)
    here.copy_(back)
    _, again = nv.moe_combine_backward(dy, here, w, pos, d_rows=here)
    assert torch.equal(here, d_rows) and torch.equal(again, d_w) and (buf[-16:] == 7).all()
    # some rows alone: the others keep what they had
    few = torch.where(torch.arange(T * k, device="cuda") % 3 == 1, pos, -1).to(torch.int32)
    buf, here = inside(T * k)
    here.fill_(5.0)
    nv.moe_combine_backward(dy, back, w, few, d_rows=here)
    named = torch.zeros(T * k, dtype=torch.bool, device="cuda")
    named[few[few >= 0].long()] = True
    assert torch.equal(here[named], d_rows[named]) and (here[~named] == 5).all() and (buf[-16:] == 7).all()


def test_streams_graphs_and_nothing_to_do(nv):
    T, E, k, N = 50, 16, 4, 264
    g, logits, x = _case(T, E, k, N, 2)
    ids, w, offsets, lst = nv.moe_route_topk(logits.cuda(), k)
    x = x.to(BF16).cuda()
    rows, pos = nv.moe_permute(x, lst, k)
    y = nv.moe_combine(rows, k, w, pos, add=x)
    d_rows, d_w = nv.moe_combine_backward(y, rows, w, pos)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    r2, p2 = nv.moe_permute(x, lst, k, stream=st)
    y2 = nv.moe_combine(r2, k, w, p2, add=x, stream=st)
    dr2, dw2 = nv.moe_combine_backward(y2, r2, w, p2, stream=st)
    st.synchronize()
    for a, b in ((rows, r2), (pos, p2), (y, y2), (d_rows, dr2), (d_w, dw2)):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    outs = [torch.zeros_like(t) for t in (rows, pos, y, d_rows, d_w)]
    with torch.cuda.graph(graph):
        nv.moe_permute(x, lst, k, rows=outs[0], positions=outs[1])
        nv.moe_combine(outs[0], k, w, outs[1], add=x, y=outs[2])
        nv.moe_combine_backward(outs[2], outs[0], w, outs[1], d_rows=outs[3], d_w=outs[4])
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((rows, pos, y, d_rows, d_w), outs):
        assert torch.equal(a, b)
    none = torch.empty(0, N, dtype=BF16, device="cuda")
    i0 = torch.empty(0, dtype=torch.int32, device="cuda")
    r0, p0 = nv.moe_permute(none, i0, k)
    assert r0.shape == (0, N) and p0.shape == (0,)
    assert nv.moe_combine(none, k).shape == (0, N)
    assert nv.moe_combine_backward(none, none, torch.empty(0, k, device="cuda"))[1].shape == (0, k)


def test_rows_past_32_bits(nv):
    """4.4e9 elements of rows: the last entries are where they should be."""
    T, k, N = 65536, 8, 8400
    x = torch.zeros(T, N, dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    x[-4:] = torch.randint(-4, 5, (4, N), generator=g, device="cuda").to(BF16)
    lst = torch.arange(T * k, dtype=torch.int32, device="cuda").roll(5)
    rows, pos = nv.moe_permute(x, lst, k)
    assert torch.equal(pos, torch.arange(T * k, dtype=torch.int32, device="cuda").roll(-5))
    assert torch.equal(rows[:5], x[-1:].expand(5, N)) and torch.equal(rows[-1], x[-1]) and torch.equal(rows[-4], x[-2])
    w = torch.full((T, k), 0.5, device="cuda")
    y = nv.moe_combine(rows, k, w, pos)
    assert torch.equal(y[-4:], x[-4:] * 4) and not y[:-4].any()
    d_rows, d_w = nv.moe_combine_backward(x, rows, w, pos)
    assert torch.equal(d_w[-4:], (x[-4:].float() ** 2).sum(1, keepdim=True).expand(4, k))
    assert torch.equal(d_rows[:5], rows[:5] * 0.5) and torch.equal(d_rows[-8:], rows[-8:] * 0.5)


@pytest.mark.parametrize("k,N", [(1, 64), (2, 250), (3, 257), (8, 2048), (11, 40)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_gradients_of_entries_that_are_not_there_beside_values_that_are_not_finite(nv, k, N, dtype, bad):
    """d_w of an entry without a row is 0 whatever dy holds, and its row of d_rows is left alone."""
    T = 5
    g = _gen(k * N)
    pos = torch.randperm(T * k, generator=g).to(torch.int32)
    here = pos.clone()
    for t, j, p in ((0, 0, -1), (2, k - 1, T * k), (3, k // 2, -(1 << 31)), (4, 0, (1 << 31) - 1)):
        here[t * k + j] = p
    w, rows = torch.randn(T, k, generator=g), torch.randn(T * k, N, generator=g).to(dtype)
    for dy_type in (BF16, F32):
        dy = torch.randn(T, N, generator=g).to(dy_type)
        dy[:4, N // 3], dy[2, N - 1] = bad, -bad
        d_rows = torch.full((T * k, N), 3.0, dtype=dtype, device="cuda")
        _, d_w = nv.moe_combine_backward(dy.cuda(), rows.cuda(), w.cuda(), here.cuda(), d_rows=d_rows)
        gone = ((here < 0) | (here >= T * k)).view(T, k)
        got = d_w.cpu()
        assert not got[gone].any() and not got[gone].isnan().any()
        assert not got[:4][~gone[:4]].isfinite().any() and got[4][~gone[4]].isfinite().all()
        left = torch.ones(T * k, dtype=torch.bool)
        left[here[~gone.view(-1)].long()] = False
        assert left.sum() == gone.sum() and (d_rows.cpu()[left] == 3).all()
