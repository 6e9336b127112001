"""The binding's own checks of tensor layouts, on CPU tensors (device number -1): what the
library would read with other strides than the tensor has is refused."""
import pytest
import torch

import weight_sequence_layers_amd as W

CPU = -1


def table(got, shape):
    t = torch.zeros(got, dtype=torch.int32)
    return W._table(t, "table", torch.int32, shape, CPU), t.data_ptr()


@pytest.mark.parametrize("got,shape", [
    ((4, 7), (4, 7)), ((28,), (4, 7)), ((30,), (4, 7)), ((6, 7), (4, 7)), ((1, 28), (4, 7)), ((1, 4, 7), (4, 7)),
    ((1, 9), (1, 7)), ((9, 1), (1, 7)), ((2, 5), (1, 7)), ((3, 2, 7), (3, 14)), ((5, 1), (5, 1)),
    ((2, 3, 5), (2, 3, 5)), ((6, 5), (2, 3, 5)), ((30,), (2, 3, 5)), ((7, 3, 5), (2, 3, 5)), ((2, 1, 5), (2, 1, 5)),
    ((2, 5), (2, 1, 5)), ((4, 9), (0, 7)), ((4, 9), (4, 0)),
])
def test_tables_read_as_they_lie(got, shape):
    p, want = table(got, shape)
    assert p == want


@pytest.mark.parametrize("got,shape", [
    ((4, 8), (4, 7)),           # a page table wider than max_pages
    ((7, 4), (4, 7)), ((2, 9), (2, 7)), ((3, 9), (3, 7)),     # positions behind the last token
    ((5, 2), (2, 5)), ((2, 5, 3), (2, 3, 5)), ((3, 2, 5), (2, 3, 5)), ((2, 4, 5), (2, 3, 5)), ((6, 8), (2, 3, 5)),
    ((5, 6), (2, 3, 5)), ((4, 6, 5), (4, 3, 5)),
])
def test_tables_of_another_layout_are_refused(got, shape):
    with pytest.raises(W.TTTError) as e:
        table(got, shape)
    assert e.value.status == 2 and str(list(got)) in str(e.value) and str(list(shape)) in str(e.value)


def test_tables_too_small_or_of_another_type_are_refused():
    for t, code in ((torch.zeros(27, dtype=torch.int32), 2), (torch.zeros(4, 7), 3),
                    (torch.zeros(4, 14, dtype=torch.int32)[:, ::2], 2)):
        with pytest.raises(W.TTTError) as e:
            W._table(t, "table", torch.int32, (4, 7), CPU)
        assert e.value.status == code
    assert W._table(None, "table", torch.int32, (4, 7), CPU) is None


def rows(t, n, width, ld):
    return W._rows(t, "x", t.dtype, n, width, ld, CPU)


def test_rows_read_as_they_lie():
    x = torch.zeros(5, 48)
    for t, n, width, ld in (
            (x, 5, 48, 48), (x, 5, 16, 48), (x[:, 16:], 5, 16, 48), (x[:, 32:], 5, 16, 48), (x[1:3, :16], 2, 16, 48),
            (x.view(5, 3, 16), 5, 48, 48), (x.view(5, 3, 16)[:, 1], 5, 16, 48), (x.view(5, 3, 16)[:, 1:], 5, 32, 48),
            (x.view(15, 16), 15, 16, 16), (x.view(5, 3, 16), 15, 16, 16), (x.flatten(), 5, 16, 48),
            (x.flatten(), 3, 40, 60), (x.view(1, 5, 48)[..., 16:], 5, 32, 48), (x[:1], 1, 16, 1000), (x[2:3, 8:24], 1, 16, 48),
            (torch.zeros(2, 5, 48)[..., 16:], 10, 32, 48), (torch.zeros(2, 5, 3, 16)[:, :, 1], 10, 16, 48),
            (torch.zeros(2, 1, 48)[..., 16:], 2, 32, 48), (torch.zeros(5, 16, 1)[:, :, 0], 5, 16, 16), (x, 0, 48, 64)):
        assert rows(t, n, width, ld) == t.data_ptr()
    assert W._rows(None, "x", torch.float32, 5, 48, 48, CPU) is None


def test_rows_of_another_layout_are_refused():
    for t, n, width, ld in (
            (torch.zeros(7, 6, 16).transpose(0, 1), 6, 112, 112),    # [heads, tokens, dim] as [tokens, heads, dim]
            (torch.zeros(96, 6).t(), 6, 96, 96),            # columns for rows
            (torch.zeros(6, 192)[:, ::2], 6, 96, 96), (torch.zeros(6, 192)[:, ::2], 6, 96, 192),
            (torch.zeros(12, 96)[::2], 6, 96, 96),          # every second row
            (torch.zeros(6, 192), 6, 96, 96),               # wider rows than said
            (torch.zeros(4, 5, 96)[:, :3], 12, 96, 96),     # sequences further apart than their rows
            (torch.zeros(1000, 96)[:1].expand(6, 96), 6, 96, 96), (torch.zeros(6, 96, 2)[..., 0], 6, 96, 96)):
        with pytest.raises(W.TTTError) as e:
            rows(t, n, width, ld)
        assert e.value.status == 2 and str(ld) in str(e.value)


BIG = (1 << 32) + 4    # 4, once it has been cut to 32 bits


@pytest.mark.parametrize("field", ["q_heads", "k_heads", "head_dim", "rot_dim", "axes"])
@pytest.mark.parametrize("value", [1 << 31, BIG, (1 << 32) + 64])
def test_config_numbers_past_32_bits_are_refused(field, value):
    with pytest.raises(W.TTTError) as e:
        W.make_rope_config(**{**dict(q_heads=4, k_heads=2, head_dim=64), field: value})
    assert e.value.status == 2
    assert W.make_rope_config(q_heads=-1, k_heads=2, head_dim=64).q_heads == -1    # the library's to refuse


@pytest.mark.parametrize("at", range(4))
def test_cache_sizes_past_32_bits_are_refused(at):
    shape = [1, 1, 1, 16]
    shape[at] = BIG
    k = torch.empty(shape, dtype=torch.bfloat16, device="meta")
    with pytest.raises(W.TTTError) as e:
        W.make_kv_cache(k, k)
    assert e.value.status == 2


@pytest.mark.parametrize("at", range(4))
def test_call_numbers_past_32_bits_are_refused(at):
    x = [1, 4, 1, 2]
    x[at] = BIG
    paged = x[0], x[1], x[2], x[3]
    calls = [lambda: W.ttt_paged_attention_work(W.ttt_kv_cache(), *paged),
             lambda: W.ttt_paged_attention(None, 512, W.ttt_kv_cache(), None, None, None, 512, None, *paged, 0.0, None)]
    if at != 2:    # seq_len is a 64-bit number
        calls += [lambda: W.ttt_window_attention_lse(None, None, None, 512, None, 512, None, x[0], x[1], 1, x[3]),
                  lambda: W.ttt_window_attention_backward(*[None] * 3, 512, None, 512, None, None, 512, *[None] * 3, 512,
                                                          None, x[0], x[1], 1, x[3])]
    for call in calls:
        with pytest.raises(W.TTTError) as e:
            call()
        assert e.value.status == 2 and "2^31" in str(e.value)


@pytest.mark.parametrize("scale", [1e-50, 2.0 ** -150, -1e-300])
def test_a_scale_that_32_bits_make_zero_is_refused(scale):
    with pytest.raises(W.TTTError) as e:
        W.ttt_paged_attention(None, 512, W.ttt_kv_cache(), None, None, None, 512, None, 1, 4, 1, 0, scale, None)
    assert e.value.status == 4


def test_heads_given_as_rows_of_their_own_are_the_same_memory():
    x = torch.zeros(20, 16)
    y = torch.zeros(4, 5, 96)[:, :3]                # the first of several sequences
    assert rows(y, 3, 96, 96) == y.data_ptr()
    assert rows(x, 5, 64, 64) == x.data_ptr()       # [tokens * heads, dim]
    with pytest.raises(W.TTTError):
        rows(x, 4, 64, 80)                          # with a gap that it does not have


def test_rows_outside_the_view_are_refused():
    """A view's rows end where the view does, however large the memory behind it is; one row has to
    be dense."""
    x = torch.zeros(8, 128)
    for t, n, width, ld in ((x[:2, :96], 3, 48, 128), (x[:4, :16], 2, 32, 128), (x.view(8, 2, 64)[:2, 0], 3, 32, 128),
                            (x[:, 0], 1, 8, 128), (x[:, ::2], 1, 64, 128), (x.t(), 1, 8, 8), (x[:2, :32], 1, 48, 128)):
        with pytest.raises(W.TTTError) as e:
            rows(t, n, width, ld)
        assert e.value.status == 2


def test_rows_whose_heads_are_named_before_their_tokens_are_the_same_memory():
    B, T, H, D = 2, 5, 3, 16
    x = torch.zeros(B, T, 3, H, D)
    for i in range(3):
        for t in (x[:, :, i], x[:, :, i].transpose(1, 2), x.permute(2, 0, 3, 1, 4)[i]):     # [B, H, T, D]
            assert rows(t, B * T, H * D, 3 * H * D) == t.data_ptr()
    y = torch.zeros(T, H, D)
    assert rows(y.transpose(0, 1), T, H * D, H * D) == y.data_ptr()
    for t, ld in ((torch.zeros(B, H, T, D), H * D), (torch.zeros(B, H, T, D).transpose(1, 2), H * D)):
        with pytest.raises(W.TTTError):
            rows(t, B * T, H * D, ld)           # heads outermost in the memory itself
