"""The Python binding of cross attention, the tree of drafted tokens and the cache commit, without a GPU."""
import types

import pytest
import torch

import periodic_sparse_attention_b200 as pia


def on(index):
    """Stands in for a CUDA tensor (or stream) of device `index`."""
    return types.SimpleNamespace(is_cuda=True, device=torch.device("cuda", index), get_device=lambda: index)


def test_a_stream_of_another_device_is_refused():
    """Its work would be ordered by a stream that the caller did not name."""
    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
        pia._elsewhere(on(0), on(1))
    x, s = on(0), on(1)
    x.shape = (1, 2, 3, 64)
    for call in (lambda: pia.pi_attn_cross_fwd(x, x, x, stream=s), lambda: pia.pi_attn_cross_bwd(x, x, x, x, x, x, stream=s),
                 lambda: pia.pi_attn_decode_tree(x, x, x, x, x, x, x, x, x, 4, 4, 2, stream=s),
                 lambda: pia.pi_attn_cache_commit(x, x, x, x, x, x, x, stream=s)):
        with pytest.raises(ValueError, match="cuda:1"):
            call()


def test_first_call_leaves_nothing_half_set():
    """A thread that finds the binding's torch set finds what goes with it set too."""
    import dis

    names = [i.argval for i in dis.get_instructions(pia._elsewhere) if i.opname == "STORE_GLOBAL"]
    assert sorted(names) == ["_current_device", "_raw_stream", "_torch"] and names[-1] == "_torch"


def test_verification_and_commit_take_the_same_cache_by_default():
    """With the choice left alone in both, a full plain cache is an overflow, not a ring that wraps."""
    import inspect

    ring = [inspect.signature(f).parameters["ring"].default for f in (pia.pi_attn_decode_tree, pia.pi_attn_cache_commit)]
    assert ring == [False, False]


def test_size_tables_stay_bounded():
    """A program whose source lengths are ever new (generation over growing contexts) keeps a bounded table."""
    calls = []

    class Library:
        def pi_attn_cross_fwd_workspace_bytes(self, *sizes):
            calls.append(sizes)
            return 0

        def pi_attn_cross_fwd(self, *args):
            return 0

    class Tensor(types.SimpleNamespace):
        def __init__(self, shape, dtype=torch.float32):
            super().__init__(shape=shape, dtype=dtype, device=torch.device("cuda", 0), is_cuda=True, get_device=lambda: 0,
                             is_contiguous=lambda: True, data_ptr=lambda: 0, new_empty=lambda shape, dtype: Tensor(shape, dtype))

    saved = {n: getattr(pia, n) for n in ("_lib", "_current_device", "_raw_stream")}
    kept = dict(pia._cross_plans)
    with pytest.raises(ValueError):
        pia._elsewhere(torch.zeros(1), None)  # (the binding's torch is set from here on)
    try:
        pia._lib, pia._current_device, pia._raw_stream = Library(), lambda: 0, lambda dev: 0
        q = Tensor((1, 2, 1, 64))
        for n in range(1, 20001):
            k = Tensor((1, 2, n, 64))
            pia.pi_attn_cross_fwd(q, k, k, out=q, want_lse=False)
        assert len(calls) == 20000 and len(pia._cross_plans) <= 4096
        pia.pi_attn_cross_fwd(q, k, k, out=q, want_lse=False)
        assert len(calls) == 20000  # a size that is at hand is not asked for again
    finally:
        for n, v in saved.items():
            setattr(pia, n, v)
        pia._cross_plans.clear()
        pia._cross_plans.update(kept)
