"""What the Python calls of the rotated appends and the 16-bit attention refuse
before they hand addresses over, on the host: the library's functions are
stood in for by one that counts its calls."""
import pytest
import torch

import compressed_space_decode_b200 as native

BF = torch.bfloat16


class Library:
    """Every function succeeds and is noted."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


class Ctx:
    handle, num_kv_heads, bits, device = None, 2, 3, -1  # the device index of host tensors



@pytest.fixture
def library(monkeypatch):
    stand_in = Library()
    monkeypatch.setattr(native, "lib", lambda: stand_in)
    return stand_in


def packed(pages=2, heads=2, words=13, ps=64, **other):
    shape = {"codes": (pages, 2, heads, words, ps), "norms": (pages, 2, heads, ps)}
    shape.update(other)
    return native.PagedCache(torch.zeros(shape["codes"], dtype=torch.int32),
                             torch.zeros(shape["norms"], dtype=torch.float16), ps)


def append(cache, ctx=Ctx(), **changed):
    k, q = torch.zeros(5, ctx.num_kv_heads, 128, dtype=BF), torch.zeros(5, 8, 128, dtype=BF)
    pos = torch.zeros(5, dtype=torch.int64)
    args = dict(k=k, v=k, slot_mapping=pos, k_pos=pos, q=q, q_pos=pos, rope=native.Rope(torch.zeros(9, 128)),
                q_rot=torch.zeros(5, 8, 128))
    args.update(changed)
    native.isoquant_decode_prep_rope(ctx, cache, stream=0, **args)


def test_packed_cache_has_to_fit_the_context(library):
    append(packed())
    assert [name for name, _ in library.calls] == ["isoquant_decode_prep_rope"]
    wide = packed()
    wide.codes = torch.zeros((2, 2, 2, 13, 128), dtype=torch.int32)[..., ::2]
    late = packed()
    late.page_size = 128
    short = packed()
    short.num_pages = 3
    for cache in (packed(heads=1), packed(heads=3), packed(words=8), packed(words=16),
                  packed(codes=(2, 2, 2, 13, 32)), packed(norms=(2, 2, 1, 64)),
                  packed(norms=(1, 2, 2, 64)), packed(norms=(2, 2, 2, 32)), wide, late, short):
        with pytest.raises(AssertionError):
            append(cache)
    four = Ctx()
    four.bits = 4
    with pytest.raises(AssertionError):
        append(packed(), four)
    append(packed(words=16), four)
    assert len(library.calls) == 2


def dense(pages=2, ps=64, dtype=BF):
    return native.DenseCache(torch.zeros((pages, 2, 2, ps, 128), dtype=dtype), ps)


def dense_append(**changed):
    k, q = torch.zeros(5, 2, 128, dtype=BF), torch.zeros(5, 8, 128, dtype=BF)
    pos = torch.zeros(5, dtype=torch.int64)
    args = dict(ctx=Ctx(), cache=dense(), k=k, v=k, slot_mapping=pos, k_pos=pos, q=q, q_pos=pos,
                rope=native.Rope(torch.zeros(9, 128)), q_out=q)
    args.update(changed)
    native.isoquant_dense_prep(stream=0, **args)


def test_missing_tensors(library):
    for missing in ("slot_mapping", "k_pos", "q_pos"):
        with pytest.raises(AssertionError):
            append(packed(), **{missing: None})
    for missing in ("v", "slot_mapping", "k_pos", "q_pos"):
        with pytest.raises(AssertionError):
            dense_append(**{missing: None})
    assert library.calls == []
    # what a call without rotation, or without a cache, does not look at
    dense_append(rope=None, k_pos=None, q_pos=None)
    dense_append(cache=None, v=None, slot_mapping=None, k_out=torch.zeros(5, 2, 128, dtype=BF))
    assert len(library.calls) == 2


def address(library, field):
    """`field` of the structure that the last call was given."""
    return next(getattr(a, field) for a in library.calls[-1][1] if hasattr(a, field))


def test_replaced_storage_is_used(library):
    """A cache's or table's tensor replaced, as a whole or in place, is the one
    that later calls use; one of another form is refused."""
    cache, rope = dense(), native.Rope(torch.zeros(9, 128))
    dense_append(cache=cache, rope=rope)
    assert address(library, "data") == cache.data.data_ptr()
    assert address(library, "cos_sin") == rope.cos_sin.data_ptr()
    cache.data, rope.cos_sin = torch.ones((4, 2, 2, 64, 128), dtype=BF), torch.ones(7, 128)
    dense_append(cache=cache, rope=rope)
    assert address(library, "data") == cache.data.data_ptr() and address(library, "num_pages") == 4 == cache.num_pages
    assert address(library, "cos_sin") == rope.cos_sin.data_ptr() and address(library, "num_positions") == 7
    cache.data.data, rope.cos_sin.data = torch.zeros((4, 2, 2, 64, 128), dtype=BF), torch.zeros(7, 128)
    dense_append(cache=cache, rope=rope)
    assert address(library, "data") == cache.data.data_ptr()
    assert address(library, "cos_sin") == rope.cos_sin.data_ptr()
    for bad in (cache.data.float(), cache.data[:, :1], cache.data[..., :64], cache.data[:, :, :, ::2], cache.data[0]):
        with pytest.raises(AssertionError):
            cache.data = bad
    for bad in (rope.cos_sin.double(), rope.cos_sin[:, :64], rope.cos_sin[0], rope.cos_sin[:, ::2]):
        with pytest.raises(AssertionError):
            rope.cos_sin = bad
    assert cache.data.shape == (4, 2, 2, 64, 128) and rope.cos_sin.shape == (7, 128)


class OnGpu(torch.Tensor):
    """Host memory that says it lies on device 0."""

    def get_device(self):
        return 0


def here(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


def test_tensors_of_another_device(library):
    """Addresses of host memory, or of another device than the context's, reach
    no kernel: each tensor in turn lies elsewhere."""
    ctx = Ctx()
    ctx.device = 0
    k, q, pos = here(5, 2, 128), here(5, 8, 128), here(5, dtype=torch.int64)
    rows, ints = here(5, 1, 8, 128), here(5, dtype=torch.int32)

    def cache(codes=here(2, 2, 2, 13, 64, dtype=torch.int32), norms=here(2, 2, 2, 64, dtype=torch.float16)):
        return native.PagedCache(codes, norms, 64)

    table, data = here(9, 128, dtype=torch.float32), here(2, 2, 2, 64, 128)
    rope, pages = native.Rope(table), native.DenseCache(data, 64)
    step = dict(k=k, v=k, slot_mapping=pos, k_pos=pos, q=q, q_pos=pos, rope=rope)
    calls = (
        (native.isoquant_decode_prep_rope, dict(step, cache=cache(), q_rot=here(5, 8, 128, dtype=torch.float32))),
        (native.isoquant_dense_prep, dict(step, cache=pages, q_out=q, k_out=k)),
        (native.isoquant_dense_attend, dict(cache=pages, q=rows, page_table=here(5, 3, dtype=torch.int32),
                                            seq_lens=ints, workspace=ints, out=rows)),
        (native.isoquant_prompt_attend, dict(q=q, k=k, v=k, cu_seqlens=ints, out=q)),
    )
    elsewhere = {id(rope): [native.Rope(table.as_subclass(torch.Tensor))],
                 id(pages): [native.DenseCache(data.as_subclass(torch.Tensor), 64)]}
    for call, args in calls:
        call(ctx, stream=0, **args)
        count = len(library.calls)
        for name, value in args.items():
            others = elsewhere.get(id(value))
            if isinstance(value, torch.Tensor):
                others = [value.as_subclass(torch.Tensor)]
            elif others is None:
                others = [cache(codes=value.codes.as_subclass(torch.Tensor)),
                          cache(norms=value.norms.as_subclass(torch.Tensor))]
            for other in others:
                with pytest.raises(AssertionError):
                    call(ctx, stream=0, **dict(args, **{name: other}))
        assert len(library.calls) == count
        second = Ctx()
        second.device = 1
        with pytest.raises(AssertionError):
            call(second, stream=0, **args)


def test_current_stream(monkeypatch):
    """The current device's current stream, with torch's short way to it and without."""
    class Stream:
        cuda_stream = 4321

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    monkeypatch.setattr(native, "_raw_stream", lambda device: 1000 + device)
    assert native._stream(None).value == 1003
    monkeypatch.setattr(native, "_raw_stream", None)
    assert native._stream(None).value == 4321
    assert native._stream(77).value == 77
