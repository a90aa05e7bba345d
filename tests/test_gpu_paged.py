"""GPU: the paged 4-bit cache (append, read back) and its attention against the plain 64-bit forms."""
import numpy as np
import pytest

import serving_ref as ref
from gpu_util import to_dev, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fg():
    import torch
    assert torch.cuda.is_available()
    import bit_group_quantized_fg_b200 as m
    m.lib()
    return m


def i32(x):
    return to_dev(np.asarray(x, np.int32))


def make_table(r, held, page, spare=2, extra_cols=1):
    """Pages in no order for sequences that hold so many positions; -1 where there is none."""
    need = [-(-n // page) for n in held]
    cols = max(need) + extra_cols
    order = r.permutation(sum(need) + spare)
    table, at = np.full((len(held), cols), -1, np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, len(order)


def rows(r, n, h, scale=1.0):
    return (r.standard_normal((n, h)) * scale).astype(np.float16)


def pair(fg, r, held, nkv, hd, group, page, **kw):
    table, n_pages = make_table(r, held, page, **kw)
    dev = fg.DevicePagedKVCache(i32(table), nkv, hd, n_pages, page, group)
    return dev, ref.Paged(table, nkv, hd, n_pages, page, group)


def same_cache(dev, cpu):
    for i, (c, p) in enumerate(((dev.k_codes, dev.k_params), (dev.v_codes, dev.v_params))):
        assert np.array_equal(to_np(c), cpu.codes[i])
        assert np.array_equal(to_np(p).view(np.uint16), cpu.params[i].view(np.uint16))


@pytest.mark.parametrize("hd,group,page,nkv,new,prefix", [
    (64, 64, 16, 12, [0, 33, 1, 20], [3, 7, 0, 15]),     # an empty sequence, pages that end inside the rows
    (128, 64, 64, 4, [1, 1, 1], [63, 64, 0]),            # one token each, at page borders
    (128, 32, 16, 1, [5], [0]),
    (128, 128, 128, 3, [130, 0, 0, 2], [1, 200, 0, 127]),
    (64, 32, 1024, 5, [40, 8, 9, 10, 1, 1, 1, 70, 2], [0, 1, 2, 3, 4, 5, 6, 7, 8]),
])
def test_append_and_read_are_exact(fg, hd, group, page, nkv, new, prefix):
    import torch
    r = np.random.default_rng(hd + page + nkv)
    dev, cpu = pair(fg, r, [a + b for a, b in zip(new, prefix)], nkv, hd, group, page)
    h = nkv * hd
    start = np.concatenate([[0], np.cumsum(new)])
    n = int(start[-1]) + 2                              # two rows of padding behind the last sequence
    k, v = rows(r, n, 3 * h), rows(r, n, 3 * h, 0.1)
    k[0, :group] = 1.5                                  # a constant group
    k[-2:] = np.nan                                     # never read as a value
    kd, vd = to_dev(k), to_dev(v)
    fg.fg_paged_append(dev, kd[:, h:], vd[:, h:], 3 * h, n, i32(prefix), row_start=i32(start))
    cpu.append(k[:, h:2 * h], v[:, h:2 * h], start, prefix)
    same_cache(dev, cpu)
    ko, vo = torch.full((2, n, h), 7.0, dtype=torch.float16, device="cuda")
    fg.fg_paged_read(dev, n, i32(start), pos0=i32(prefix), k=ko, v=vo)
    want = np.full((2, n, h), 7.0)
    for b in range(len(new)):
        for i in range(new[b]):
            want[:, start[b] + i] = cpu.values(b, prefix[b] + i).reshape(2, h)
    for got, w in zip((ko, vo), want):                  # one rounding of mn + code * s; padding left as it was
        assert np.all(np.abs(to_np(got).astype(np.float64) - w) <= 2.0 ** -11 * np.abs(w) + 2.0 ** -25)
        assert np.all(to_np(got)[n - 2:] == 7.0)


def test_append_matches_the_dense_cache(fg):
    """The same codes and parameters as fg_kv_append, bit for bit."""
    r = np.random.default_rng(1)
    B, nkv, hd, g, T = 3, 4, 128, 64, 21
    h = nkv * hd
    k, v = to_dev(rows(r, B * T, h, 3.0)), to_dev(rows(r, B * T, h))
    dense = fg.DeviceKVCache(B, nkv, hd, T, g)
    fg.fg_kv_append(dense, k, v, h, T)
    dev, _ = pair(fg, r, [T] * B, nkv, hd, g, 16)
    fg.fg_paged_append(dev, k, v, h, B * T, i32([0] * B), row_start=i32(np.arange(B + 1) * T))
    table = to_np(dev.page_table)
    for b in range(B):
        for t in range(T):
            p, s = table[b, t // 16], t % 16
            assert np.array_equal(to_np(dev.k_codes[p, :, s]), to_np(dense.k_codes[b, :, t]))
            assert np.array_equal(to_np(dev.v_params[p, :, s]), to_np(dense.v_params[b, :, t]))


def test_append_without_row_start(fg):
    """One row per sequence (a decode step); fewer rows than sequences is allowed."""
    r = np.random.default_rng(2)
    dev, cpu = pair(fg, r, [10, 20, 30], 2, 64, 32, 16)
    k, v = rows(r, 2, 128), rows(r, 2, 128)
    fg.fg_paged_append(dev, to_dev(k), to_dev(v), 128, 2, i32([9, 16, 0]))
    cpu.append(k, v, [0, 1, 2, 2], [9, 16, 0])
    same_cache(dev, cpu)


def test_indices_out_of_range(fg):
    """Bad pages, positions and rows are skipped by append, zeros in read, invisible to attention."""
    import torch
    r = np.random.default_rng(3)
    nkv, hd, g, page = 2, 128, 64, 16
    table = np.array([[0, -1, 3, 99], [-7, 2, 1, 4], [5, 6, 1 << 30, -(1 << 31)]], np.int32)
    dev = fg.DevicePagedKVCache(i32(table), nkv, hd, 7, page, g)
    cpu = ref.Paged(table, nkv, hd, 7, page, g)
    start, pos0 = [2, 66, 130, 197], [0, -3, 0]
    k, v = rows(r, 200, nkv * hd), rows(r, 200, nkv * hd)
    fg.fg_paged_append(dev, to_dev(k), to_dev(v), nkv * hd, 200, i32(pos0), row_start=i32(start))
    cpu.append(k, v, start, pos0)
    same_cache(dev, cpu)
    ko, vo = torch.full((2, 200, nkv * hd), 7.0, dtype=torch.float16, device="cuda")
    fg.fg_paged_read(dev, 200, i32(start), pos0=i32(pos0), k=ko, v=vo)
    got = to_np(ko)
    assert np.all(got[:2] == 7) and np.all(got[197:] == 7)
    for b in range(3):
        for i in range(start[b], start[b + 1]):
            w = cpu.values(b, pos0[b] + i - start[b])
            w = np.zeros(nkv * hd) if w is None else w[0].reshape(-1)
            assert np.all(np.abs(got[i] - w) <= 2.0 ** -11 * np.abs(w) + 2.0 ** -25)
    q = rows(r, 3, 4 * hd)
    for lens in ([64, 64, 64], [1000, 20, 33], [-5, 0, 1 << 30], [17, 17, 17]):
        out = fg.fg_paged_attention(to_dev(q), 4 * hd, dev, i32(lens), 4)
        check(to_np(out), q, cpu, lens, 4)
    # an unsorted row_start: no row may land outside the pages, nothing else is promised
    fg.fg_paged_append(dev, to_dev(k), to_dev(v), nkv * hd, 200, i32(pos0), row_start=i32([50, -4, 300, 7]))
    torch.cuda.synchronize()


def check(out, q, cpu, lens, nh, window=0, n_sink=0, heads=None):
    hd, rep = cpu.hd, nh // cpu.nkv
    worst = 0.0
    for b in range(len(lens)):
        k, v, rise, there = cpu.gather(b, lens[b])
        n = k.shape[1]
        see = ref.visible(n - 1, n, window, n_sink) & there
        for j in range(nh) if heads is None else heads:
            want, budget = ref.attend(q[b, j * hd:(j + 1) * hd].astype(np.float64), k[j // rep], v[j // rep], see,
                                      rise[j // rep])
            got = out[b, j * hd:(j + 1) * hd].astype(np.float64)
            tol = ref.attend_tol(want, budget)
            assert np.all(np.isfinite(got)), (b, j)
            worst = max(worst, float(np.max(np.abs(got - want) / tol)))
            assert worst <= 1.0, (b, j, worst)
    return worst


def filled(fg, seed, held, nkv, hd, group, page, scale=1.0, vscale=1.0):
    r = np.random.default_rng(seed)
    dev, cpu = pair(fg, r, held, nkv, hd, group, page)
    start = np.concatenate([[0], np.cumsum(held)])
    n = int(start[-1])
    k, v = rows(r, n, nkv * hd, scale), rows(r, n, nkv * hd, vscale)
    if n:
        fg.fg_paged_append(dev, to_dev(k), to_dev(v), nkv * hd, n, i32([0] * len(held)), row_start=i32(start))
    cpu.codes = [to_np(dev.k_codes), to_np(dev.v_codes)]     # append is checked above
    cpu.params = [to_np(dev.k_params), to_np(dev.v_params)]
    return r, dev, cpu


@pytest.mark.parametrize("hd,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("nkv,rep", [(3, 1), (2, 2), (1, 5), (2, 8), (1, 13), (1, 24)])
def test_paged_attention(fg, hd, group, nkv, rep):
    """Every head layout and group: lengths 0, 1, around the tiles' and pages' ends, a long one."""
    lens = [0, 1, 15, 16, 17, 31, 33, 64, 65, 200, 777]
    nh = nkv * rep
    r, dev, cpu = filled(fg, hd + group + rep, lens, nkv, hd, group, 16 if rep % 2 else 64)
    q = rows(r, len(lens), nh * hd + 8)
    out = fg.fg_paged_attention(to_dev(q), nh * hd + 8, dev, i32(lens), nh)
    assert np.all(to_np(out)[0] == 0)
    print("worst / tolerance", check(to_np(out), q, cpu, lens, nh))


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (7, 0), (16, 4), (33, 5), (100, 70), (64, 0), (250, 1), (4096, 4),
                                           (2 ** 31 - 1, 2 ** 31 - 1), (-3, 9)])
@pytest.mark.parametrize("page", [16, 32, 256])
def test_paged_attention_window_and_sinks(fg, window, n_sink, page):
    lens = [0, 1, 3, 17, 64, 65, 130, 401]
    nkv, rep, hd, group = 2, 4, 128, 64
    r, dev, cpu = filled(fg, window % 97 + page, lens, nkv, hd, group, page)
    q = rows(r, len(lens), nkv * rep * hd)
    out = fg.fg_paged_attention(to_dev(q), nkv * rep * hd, dev, i32(lens), nkv * rep, window=window, n_sink=n_sink)
    check(to_np(out), q, cpu, lens, nkv * rep, window if window > 0 else 0, n_sink)


@pytest.mark.parametrize("lens,nkv,rep,hd,group", [
    ([20000], 1, 1, 128, 64),            # one long context over every warp
    ([9000, 5], 2, 8, 64, 32),
    ([3000, 0, 12000, 1, 700], 1, 4, 128, 128),
])
def test_paged_attention_long(fg, lens, nkv, rep, hd, group):
    r, dev, cpu = filled(fg, len(lens) + nkv, lens, nkv, hd, group, 64)
    q = rows(r, len(lens), nkv * rep * hd)
    out = fg.fg_paged_attention(to_dev(q), nkv * rep * hd, dev, i32(lens), nkv * rep)
    print("worst / tolerance", check(to_np(out), q, cpu, lens, nkv * rep))
    out = fg.fg_paged_attention(to_dev(q), nkv * rep * hd, dev, i32(lens), nkv * rep, window=2500, n_sink=3)
    check(to_np(out), q, cpu, lens, nkv * rep, 2500, 3)


@pytest.mark.parametrize("scale,vscale,qscale", [(1.0, 1e-3, 1.0), (0.01, 1.0, 1e-3), (4.0, 300.0, 4.0), (1.0, 1.0, 100.0)])
def test_paged_attention_ranges(fg, scale, vscale, qscale):
    """Small and large keys, values and queries: flat and one-key softmaxes, value scales far from 1."""
    lens = [300, 50]
    r, dev, cpu = filled(fg, 11, lens, 2, 128, 64, 32, scale, vscale)
    q = rows(r, 2, 4 * 128, qscale)
    out = fg.fg_paged_attention(to_dev(q), 512, dev, i32(lens), 4)
    print("worst / tolerance", check(to_np(out), q, cpu, lens, 4))


def test_paged_attention_value_scales_grow(fg):
    """Value groups whose scales grow by five orders of magnitude along the context, and scores that do too."""
    r, dev, cpu = filled(fg, 13, [400], 1, 128, 64, 16)
    for grow in (dev.v_params, dev.k_params):
        pages = to_np(dev.page_table)[0]
        for i in range(25):
            grow[int(pages[i])] *= 2.0 ** (i * 0.7 - 12) if grow is dev.v_params else 2.0 ** (i * 0.2 - 4)
    cpu.params = [to_np(dev.k_params), to_np(dev.v_params)]
    q = rows(r, 1, 2 * 128)
    out = fg.fg_paged_attention(to_dev(q), 256, dev, i32([400]), 2)
    print("worst / tolerance", check(to_np(out), q, cpu, [400], 2))


def test_paged_attention_what_is_not_visible_does_not_matter(fg):
    """NaN and infinite parameters behind the length, before the window and in unused pages."""
    import torch
    lens = [100, 37]
    r, dev, cpu = filled(fg, 17, [130, 64], 2, 128, 64, 16)
    q = to_dev(rows(r, 2, 4 * 128))
    clean = {w: fg.fg_paged_attention(q, 512, dev, i32(lens), 4, window=w, n_sink=3) for w in (0, 20)}
    table = to_np(dev.page_table)
    used = {(int(table[b, t // 16]), t % 16) for b in range(2) for t in range(lens[b])}
    seen = {(int(table[b, t // 16]), t % 16) for b in range(2) for t in range(lens[b]) if t >= lens[b] - 20 or t < 3}
    for w, see in ((0, used), (20, seen)):
        for p in range(dev.c.n_pages):
            for s in range(16):
                if (p, s) not in see:
                    dev.k_params[p, :, s] = float("nan") if (p + s) % 2 else float("inf")
                    dev.v_params[p, :, s] = float("-inf") if (p + s) % 3 else float("nan")
        got = fg.fg_paged_attention(q, 512, dev, i32(lens), 4, window=w, n_sink=3)
        assert torch.equal(got, clean[w])
    # a NaN that is visible does reach its head's output, and only that
    p, s = int(table[1, 2]), 3
    dev.v_params[p, 1, s] = float("nan")
    got = to_np(fg.fg_paged_attention(q, 512, dev, i32(lens), 4, window=20, n_sink=3))
    assert np.isnan(got[1, 256:]).all() and np.isfinite(got[1, :256]).all() and np.isfinite(got[0]).all()


def test_paged_attention_repeats_streams_and_graphs(fg):
    """The same bits on every run, on another stream, two calls at once with their own workspaces, and
    from a captured graph replayed with new lengths, queries and pages."""
    import torch
    held = [600, 1, 333, 90]
    r, dev, cpu = filled(fg, 19, held, 2, 128, 64, 64)
    nh = 8
    q = to_dev(rows(r, 4, nh * 128))
    lens = i32(held)
    first = fg.fg_paged_attention(q, nh * 128, dev, lens, nh)
    for _ in range(3):
        assert torch.equal(fg.fg_paged_attention(q, nh * 128, dev, lens, nh), first)
    torch.cuda.synchronize()
    n = fg.fg_paged_attention_workspace_bytes(nh, 2, 128)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.zeros_like(first) for _ in streams]
    wss = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, o, ws in zip(streams, outs, wss):
            fg.fg_paged_attention(q, nh * 128, dev, lens, nh, out=o, workspace=ws, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    # capture
    out, g = torch.zeros_like(first), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fg.fg_paged_attention(q, nh * 128, dev, lens, nh, window=100, n_sink=2, out=out, workspace=wss[0])
    for new in ([600, 1, 333, 90], [5, 0, 300, 64], [599, 1, 1, 1]):
        lens.copy_(i32(new))
        q.copy_(to_dev(rows(r, 4, nh * 128)))
        g.replay()
        torch.cuda.synchronize()
        check(to_np(out), to_np(q), cpu, new, nh, 100, 2)


def test_paged_attention_many_sequences(fg):
    """More sequences than a block has threads, most of them short or empty; a shared prefix page."""
    r = np.random.default_rng(23)
    lens = r.integers(0, 40, 700)
    lens[[3, 699]] = [2000, 500]
    r2, dev, cpu = filled(fg, 29, list(lens), 1, 64, 64, 16)
    table = cpu.table.copy()
    table[lens >= 16, 0] = table[3, 0]
    dev.page_table.copy_(i32(table))
    cpu.table = table
    q = rows(r, 700, 2 * 64)
    out = fg.fg_paged_attention(to_dev(q), 128, dev, i32(lens), 2)
    print("worst / tolerance", check(to_np(out), q, cpu, lens, 2))


def test_paged_cache_past_2_31_bytes(fg):
    """Slots whose byte offsets pass 2^32: the last pages of a 5 GB cache."""
    import torch
    n_pages, nkv, hd, g, page = 20500, 32, 128, 64, 64
    table = i32([[n_pages - 1, 3, n_pages - 2, 0]])
    dev = fg.DevicePagedKVCache(table, nkv, hd, n_pages, page, g)
    r = np.random.default_rng(31)
    n, h = 200, nkv * hd
    k, v = rows(r, n, h), rows(r, n, h)
    fg.fg_paged_append(dev, to_dev(k), to_dev(v), h, n, i32([0]), row_start=i32([0, n]))
    small = ref.Paged(np.array([[0, 1, 2, 3]]), nkv, hd, 4, page, g)
    small.append(k, v, [0, n], [0])
    ids = [n_pages - 1, 3, n_pages - 2, 0]
    assert np.array_equal(to_np(dev.k_codes[ids]), small.codes[0])
    assert np.array_equal(to_np(dev.v_codes[ids]), small.codes[1])
    ko, vo = fg.fg_paged_read(dev, n, i32([0, n]))
    w = np.stack([small.values(0, t)[1].reshape(-1) for t in range(n)])
    assert np.all(np.abs(to_np(vo) - w) <= 2.0 ** -11 * np.abs(w) + 2.0 ** -25)
    q = rows(r, 1, h)
    out = fg.fg_paged_attention(to_dev(q), h, dev, i32([n]), nkv)
    check(to_np(out), q, small, [n], nkv, heads=[0, 17, 31])
    del dev, ko, vo
    torch.cuda.empty_cache()


@pytest.mark.parametrize("window,n_sink", [(0, 0), (40, 0), (100, 3)])
@pytest.mark.parametrize("below", [20.0, 500.0])
def test_paged_attention_scores_far_below_zero(fg, window, n_sink, below):
    lens, nkv, rep, hd = [70, 1, 333], 2, 2, 64
    r = np.random.default_rng(int(below))
    dev, cpu = pair(fg, r, lens, nkv, hd, 64, 16)
    start = np.concatenate([[0], np.cumsum(lens)])
    a, n = np.sqrt(below / np.sqrt(hd)), int(start[-1])        # q . k / sqrt(hd) = -below + noise
    k = (-a + r.standard_normal((n, nkv * hd)) * 0.1).astype(np.float16)
    v = rows(r, n, nkv * hd)
    fg.fg_paged_append(dev, to_dev(k), to_dev(v), nkv * hd, n, i32([0] * 3), row_start=i32(start))
    cpu.codes = [to_np(dev.k_codes), to_np(dev.v_codes)]
    cpu.params = [to_np(dev.k_params), to_np(dev.v_params)]
    q = (a + r.standard_normal((3, nkv * rep * hd)) * 0.1).astype(np.float16)
    out = fg.fg_paged_attention(to_dev(q), nkv * rep * hd, dev, i32(lens), nkv * rep, window=window, n_sink=n_sink)
    check(to_np(out), q, cpu, lens, nkv * rep, window, n_sink)


@pytest.mark.parametrize("scale", [1e-7, 5e-7, 3e-6, 1e-4, 2e-3, 1e4])
def test_append_of_small_and_large_ranges_is_exact(fg, scale):
    """Scales that are 0, subnormal (codes that pass 15 are held there), just normal, and near the largest."""
    r = np.random.default_rng(21)
    nkv, hd, group, n = 3, 64, 32, 40
    dev, cpu = pair(fg, r, [n], nkv, hd, group, 16)
    k, v = rows(r, n, nkv * hd, scale), (r.random((n, nkv * hd)) * scale).astype(np.float16)
    k, v = np.clip(k, -30000, 30000), v + np.float16(0 if scale > 1 else 0.25)
    fg.fg_paged_append(dev, to_dev(k), to_dev(v), nkv * hd, n, i32([0]), row_start=i32([0, n]))
    cpu.append(k, v, np.array([0, n]), [0])
    same_cache(dev, cpu)


@pytest.mark.parametrize("vscale", [1e-4, 1e-5])
@pytest.mark.parametrize("rep", [1, 2, 4, 8, 16])
def test_paged_attention_small_values_wherever_the_window_starts(fg, rep, vscale):
    """The fp16 weights are relative to the value scales that are seen, also where the first positions of the first tile are
    not: before the window, in a page that is not there, or with values that are all equal (scale 0)."""
    nkv, hd, group, page = 2, 64, 32, 16
    lens = [30, 17, 64, 100, 127, 128, 50]
    r, dev, cpu = filled(fg, rep, lens, nkv, hd, group, page, vscale=vscale)
    nh = nkv * rep
    q = rows(r, len(lens), nh * hd)
    for window in (1, 2, 9, 14, 33, 47, 60):
        out = fg.fg_paged_attention(to_dev(q), nh * hd, dev, i32(lens), nh, window=window)
        check(to_np(out), q, cpu, lens, nh, window)
    table = cpu.table.copy()
    for i in range(4):                      # the first pages of a sequence are not there
        table[3 + i % 3, i] = -1
    dev.page_table.copy_(i32(table))
    cpu.table = table
    out = fg.fg_paged_attention(to_dev(q), nh * hd, dev, i32(lens), nh)
    check(to_np(out), q, cpu, lens, nh)
    for b in range(len(lens)):              # a page of equal values, then the others
        p = next((int(p) for p in table[b] if p >= 0), None)
        dev.v_params[p, :, :, :, 1] = 0
    cpu.params = [to_np(dev.k_params), to_np(dev.v_params)]
    out = fg.fg_paged_attention(to_dev(q), nh * hd, dev, i32(lens), nh)
    check(to_np(out), q, cpu, lens, nh)


def test_paged_attention_heads_past_2_32_bytes_of_a_page(fg):
    """More key/value heads than 4 GiB of a page's codes hold: the last ones are read from where append put them."""
    import torch
    nkv, hd, g, page, n = (1 << 16) + 4, 128, 128, 1024, 3
    h = nkv * hd
    dev = fg.DevicePagedKVCache(i32([[0]]), nkv, hd, 1, page, g)
    r = np.random.default_rng(41)
    k, v, q = rows(r, n, h), rows(r, n, h), rows(r, 1, h)
    fg.fg_paged_append(dev, to_dev(k), to_dev(v), h, n, i32([0]), row_start=i32([0, n]))
    heads = [0, 1, 3, nkv - 5, nkv - 4, nkv - 1]
    pick = lambda x: x.reshape(len(x), nkv, hd)[:, heads].reshape(len(x), -1)   # noqa: E731
    small = ref.Paged(np.array([[0]]), len(heads), hd, 1, page, g)
    small.append(pick(k), pick(v), [0, n], [0])
    for i, codes in enumerate((dev.k_codes, dev.v_codes)):
        assert np.array_equal(to_np(codes[0, heads, :n]), small.codes[i][0, :, :n])
    out = fg.fg_paged_attention(to_dev(q), h, dev, i32([n]), nkv)
    check(pick(to_np(out)), pick(q), small, [n], len(heads))
    del dev
    torch.cuda.empty_cache()


def middle_tol(cpu, b, n, j, q):
    """Budget of head j's output when what a weight's rounding took off is given back with the mean code: the rounding
    2^-11 p s is multiplied by c - 7.5 in place of c (the other terms as in attend_tol)."""
    k, v, rise, there = cpu.gather(b, n)
    pages, t = cpu.table[b, np.arange(n) // cpu.page], np.arange(n) % cpu.page
    s = np.repeat(cpu.params[1][pages, j, t, :, 1].astype(np.float64), cpu.group, axis=-1)
    out, (mass, size, _, vmax) = ref.attend(q, k[j], v[j], there, rise[j])
    e = np.exp(k[j] @ q / np.sqrt(cpu.hd) - (k[j] @ q / np.sqrt(cpu.hd)).max())
    off = (e / e.sum()) @ np.abs(rise[j] - 7.5 * s)
    fp32 = 2 * (16 * 2.0 ** -23 * size + 2.0 ** -22) + 128 * 2.0 ** -23
    return out, 2.0 ** -11 * np.abs(out) + 2.0 ** -25 + 2.0 ** -11 * off + fp32 * mass + n * 2.0 ** -25 * vmax


@pytest.mark.parametrize("hd,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("rep", [1, 2, 4, 8, 13])
def test_paged_attention_gives_back_what_the_weights_lost(fg, hd, group, rep):
    """Values whose codes are 7 and 8 but for the two ends of a group, and whose outputs are small: their error is that of
    half a code, not of seven and a half."""
    nkv, page, lens = 3, 16, [2, 3, 5, 8, 13, 40]
    r = np.random.default_rng(hd + group + rep)
    dev, cpu = pair(fg, r, lens, nkv, hd, group, page)
    start, n = np.concatenate([[0], np.cumsum(lens)]), int(sum(lens))
    v = r.choice([-0.5, 0.5], (n, nkv * hd // group, group)) * r.uniform(0.2, 1.0, (n, nkv * hd // group, 1))
    v[:, :, 0], v[:, :, 1] = -7.5 * np.abs(v[:, :, 2]) * 2, 7.5 * np.abs(v[:, :, 2]) * 2
    k, v = rows(r, n, nkv * hd), v.reshape(n, -1).astype(np.float16)
    fg.fg_paged_append(dev, to_dev(k), to_dev(v), nkv * hd, n, i32([0] * len(lens)), row_start=i32(start))
    cpu.codes, cpu.params = [to_np(dev.k_codes), to_np(dev.v_codes)], [to_np(dev.k_params), to_np(dev.v_params)]
    q = rows(r, len(lens), nkv * rep * hd)
    out = to_np(fg.fg_paged_attention(to_dev(q), nkv * rep * hd, dev, i32(lens), nkv * rep)).astype(np.float64)
    worst = 0.0
    for b, m in enumerate(lens):
        for j in range(nkv * rep):
            x = q[b, j * hd:(j + 1) * hd].astype(np.float64)
            want, tol = middle_tol(cpu, b, m, j // rep, x)
            worst = max(worst, float(np.max(np.abs(out[b, j * hd:(j + 1) * hd] - want) / tol)))
    print("worst / tolerance", worst)
    assert worst <= 1.0
