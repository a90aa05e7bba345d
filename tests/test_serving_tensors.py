"""The binding's checks of the tensors given to the serving calls: what is accepted lies where the kernels
read and write it, everything else is refused (on host tensors here, by the calls themselves on the GPU)."""
import pytest

import serving_ref as ref


@pytest.fixture(scope="module")
def fg():
    import torch

    import bit_group_quantized_fg_b200 as m
    m._torch = torch
    return m


H, N = 16, 6


def wide():
    """[N, 3 H] rows."""
    import torch
    return torch.zeros((N, 3 * H), dtype=torch.float16)


def accepted(fg, t, n, cols, stride, **kw):
    return fg._rows(t, n, cols, stride, -1, "t", **kw) == t.data_ptr()


def test_rows_whose_stride_the_call_knows(fg):
    """x, E, out, and the rows of packed attention: the tensor's rows are the call's rows."""
    import torch
    x = wide()
    whole = torch.zeros((N, H), dtype=torch.float16)
    for t in (whole, whole.view(-1), whole.view(N, 4, 4), whole.view(2 * N, H // 2), torch.zeros((N + 2, H), dtype=torch.float16),
              whole[1:]):
        assert accepted(fg, t, N if t.numel() >= whole.numel() else N - 1, H, H)
    assert accepted(fg, x[:, H:2 * H], N, H, 3 * H) and accepted(fg, x, N, 3 * H, 3 * H)
    assert accepted(fg, x.view(N, 3, 4, 4)[:, 1], N, H, 3 * H)          # [N, heads, hd] inside wider rows
    assert accepted(fg, x[2:3, H:2 * H], 1, H, H)                       # one row: its stride says nothing
    assert accepted(fg, x[:0], 0, H, H)
    hidden = torch.zeros((N, 4, H), dtype=torch.float16)
    for t in (x[:, :H], x[:, H:2 * H], x, hidden[:, -1], hidden, whole[:1].expand(N, H), whole.t().contiguous().t(),
              whole[::2], whole[:N - 1], whole.view(-1)[8:], whole.view(N, 4, 4).transpose(1, 2),
              whole.view(4, N, 4).transpose(0, 1)):
        with pytest.raises(ValueError):
            fg._rows(t, N, H, H, -1, "t")
    with pytest.raises(ValueError):
        fg._rows(x.view(N, 3, 4, 4)[:, 1].transpose(1, 2), N, H, 3 * H, -1, "t")     # heads and dims swapped
    with pytest.raises(ValueError):
        fg._rows(whole.float(), N, H, H, -1, "t")
    with pytest.raises(ValueError):
        fg._rows(whole, N, H, H, 0, "t")                                # not on that device


def test_rows_whose_stride_the_caller_states(fg):
    """k, v of append and q of paged attention: a flat buffer or a start is taken at its word, a tensor whose own rows
    lie elsewhere is not."""
    import torch
    x = wide()
    flat = x.view(-1)
    for t, n, stride in ((x[:, H:], N, 3 * H), (flat[H:], N, 3 * H), (x[0, H:2 * H], N, 3 * H), (x[:1, H:2 * H], N, 3 * H),
                         (x, N // 2, 6 * H), (x.view(2, 3, 3 * H), N, 3 * H), (x.view(2, 3, 3 * H), 3 * N, H)):
        assert accepted(fg, t, n, H, stride, stated=True)
    for t, n, stride in ((x[:, :H], N, H), (x[::2], N // 2, 3 * H), (x[:, ::3], N, 3 * H), (flat[H:], N + 1, 3 * H),
                         (x[:, 2 * H:], N, 3 * H + 8), (x.view(N, 3, 4, 4)[:, 1].transpose(1, 2), N, 3 * H)):
        with pytest.raises(ValueError):
            fg._rows(t, n, H, stride, -1, "t", stated=True)


def test_index_arrays_and_workspaces(fg):
    import torch
    n = torch.zeros(5, dtype=torch.int32)
    assert fg._index(n, 5, torch.int32, -1, "n") == n.data_ptr() and fg._index(None, 5, torch.int32, -1, "n") is None
    for t, count, dev in ((n.long(), 5, -1), (n, 6, -1), (torch.zeros(10, dtype=torch.int32)[::2], 5, -1), (n, 5, 0)):
        with pytest.raises(ValueError):
            fg._index(t, count, torch.int32, dev, "n")
    w = torch.zeros(64, dtype=torch.float32)
    assert fg._bytes(w, -1, "w") == (w.data_ptr(), 256) and fg._bytes(None, -1, "w") == (None, 0)
    for t, dev in ((w[::2], -1), (w, 0)):
        with pytest.raises(ValueError):
            fg._bytes(t, dev, "w")


# ------------------------------------------------------------------------- the calls themselves
def on_gpu():
    import numpy as np
    from gpu_util import to_dev
    import bit_group_quantized_fg_b200 as m
    m.lib()
    return m, np.random.default_rng(3), to_dev


@pytest.mark.gpu
def test_lm_head_sample_of_strided_rows():
    """The last position's hidden states of a batch, uncopied: refused; their copy gives the tokens of those rows."""
    import numpy as np
    import torch
    fg, r, to_dev = on_gpu()
    B, T, h, V = 5, 3, 128, 1000
    hidden = to_dev(r.standard_normal((B, T, h)).astype(np.float16))
    E = to_dev((r.standard_normal((V, 2 * h)) * 0.2).astype(np.float16))
    u = r.random(B).astype(np.float32)
    with pytest.raises(ValueError):
        fg.fg_lm_head_sample(hidden[:, -1], E[:, :h].contiguous(), to_dev(u))
    with pytest.raises(ValueError):
        fg.fg_lm_head_sample(hidden[:, -1].contiguous(), E[:, :h], to_dev(u))
    logits = torch.empty((B, V), device="cuda")
    tok = fg.fg_lm_head_sample(hidden[:, -1].contiguous(), E[:, :h].contiguous(), to_dev(u), logits=logits)
    x, e = hidden[:, -1].double(), E[:, :h].double()
    assert torch.all((logits - x @ e.T).abs() <= 2.0 ** -20 * (x.abs() @ e.abs().T))   # 16 fp32 roundings of the sums
    lg = logits.cpu().numpy()
    assert [int(t) for t in tok] == [ref.sample_row(lg[b], u[b])[0] for b in range(B)]
    for kw in (dict(logits=torch.empty((B, V + 8), device="cuda")[:, :V]), dict(tokens=torch.zeros(B, dtype=torch.int64, device="cuda")),
               dict(workspace=torch.zeros(8, dtype=torch.uint8)), dict(top_p=torch.full((B,), 0.5))):
        with pytest.raises(ValueError):
            fg.fg_lm_head_sample(hidden[:, -1].contiguous(), E[:, :h].contiguous(), to_dev(u), **kw)
    with pytest.raises(ValueError):
        fg.fg_sample(logits.t(), to_dev(u))
    with pytest.raises(ValueError):
        fg.fg_sample(logits.half(), to_dev(u))
    with pytest.raises(ValueError):
        fg.fg_sample(logits, None)


@pytest.mark.gpu
def test_attention_into_and_out_of_strided_tensors():
    """A column slice as the output and permuted heads are refused and touch nothing; three-dimensional rows are not."""
    import numpy as np
    import torch
    fg, r, to_dev = on_gpu()
    i32 = lambda x: to_dev(np.asarray(x, np.int32))   # noqa: E731
    B, nh, nkv, hd, n = 3, 4, 2, 64, 40
    h, hk = nh * hd, nkv * hd
    cache = fg.DevicePagedKVCache(i32([[0, 1], [2, 3], [4, 5]]), nkv, hd, 6, 32, 64)
    start = i32([0, 10, 30, n])
    x = to_dev(r.standard_normal((n, h + 2 * hk)).astype(np.float16))
    q, k, v = x[:, :h], x[:, h:h + hk], x[:, h + hk:]
    fg.fg_paged_append(cache, k, v, h + 2 * hk, n, i32([0] * B), row_start=start)
    with pytest.raises(ValueError):      # rows h + 2 hk apart, not hk
        fg.fg_paged_append(cache, k, v, hk, n, i32([0] * B), row_start=start)
    lens = i32([10, 20, 10])
    want = fg.fg_paged_attention(q, h + 2 * hk, cache, lens, nh)
    out = torch.zeros((B, 2 * h), dtype=torch.float16, device="cuda")
    for o in (out[:, :h], out[:, h:], out):
        with pytest.raises(ValueError):
            fg.fg_paged_attention(q, h + 2 * hk, cache, lens, nh, out=o)
    assert not out.any()
    got = torch.zeros((B, nh, hd), dtype=torch.float16, device="cuda")
    assert torch.equal(fg.fg_paged_attention(q[:B], h + 2 * hk, cache, lens, nh, out=got).view(B, h), want)
    with pytest.raises(ValueError):
        fg.fg_paged_attention(q, h, cache, lens, nh)
    with pytest.raises(ValueError):
        fg.fg_paged_attention(q, h + 2 * hk, cache, lens[:2], nh)
    with pytest.raises(ValueError):
        fg.fg_paged_attention(q, h + 2 * hk, cache, lens, nh, workspace=torch.zeros(1 << 20, dtype=torch.uint8))

    want = fg.fg_varlen_attention(q, k, v, start, start, 20, nh, nkv, hd)
    out = torch.zeros((n, 2 * h), dtype=torch.float16, device="cuda")
    for o in (out[:, :h], out[:, h:], out):
        with pytest.raises(ValueError):
            fg.fg_varlen_attention(q, k, v, start, start, 20, nh, nkv, hd, out=o)
    assert not out.any()
    three = lambda t, heads: t.unflatten(1, (heads, hd))   # noqa: E731
    got = torch.zeros((n, nh, hd), dtype=torch.float16, device="cuda")
    fg.fg_varlen_attention(three(q, nh), three(k, nkv), three(v, nkv), start, start, 20, nh, nkv, hd, out=got)
    assert torch.equal(got.view(n, h), want)
    swapped = three(q, nh).contiguous().transpose(0, 1).contiguous().transpose(0, 1)     # [n, heads, hd], heads outermost
    with pytest.raises(ValueError):
        fg.fg_varlen_attention(swapped, k, v, start, start, 20, nh, nkv, hd)
    with pytest.raises(ValueError):
        fg.fg_varlen_attention(q, k, v[:, ::2], start, start, 20, nh, nkv, hd)
    with pytest.raises(ValueError):
        fg.fg_varlen_attention(q, k, v, start, start.long(), 20, nh, nkv, hd)
    ko = torch.zeros((n, 2 * hk), dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):      # one stride for both
        fg.fg_paged_read(cache, n, start, k=ko[:, :hk], v=torch.zeros((n, hk), dtype=torch.float16, device="cuda"))
    a, b = fg.fg_paged_read(cache, n, start, k=ko[:, :hk], v=ko[:, hk:])
    c, d = fg.fg_paged_read(cache, n, start)
    assert torch.equal(a, c) and torch.equal(b, d)
