"""Arguments of the four-bit cache's binding that must not reach the library as something else (no GPU: the library is
stood in for)."""

from types import SimpleNamespace

import pytest
import torch

from rejection_sampling_verify_10_amd import kvq
from test_kvq_commit_host import gpu, make


def stand_in(monkeypatch):
    machine, cache, ints = make(monkeypatch, 0)
    cache._needs, cache._ref = {}, 0
    called = []

    def call(*args):
        called.append(args)
        return 0

    library = SimpleNamespace(spec_kvq_score=call, spec_kvq_evict=call, spec_kvq_score_workspace_bytes=lambda *a: 0,
                              spec_kvq_evict_workspace_bytes=lambda *a: 0, spec_kv_commit=call)
    monkeypatch.setattr(kvq, "lib", lambda: library)
    return cache, ints, called


@pytest.mark.parametrize("width", [0, 1, 4])
def test_a_path_of_no_nodes_is_not_a_missing_path(monkeypatch, width):
    cache, ints, called = stand_in(monkeypatch)
    q = gpu(torch.zeros(2, 4, 6, 64))
    args = (q, gpu(torch.zeros(2, 4, 6)), cache, ints(2), ints(2), gpu(torch.zeros(2, 3, 8)), ints(2, 3, 8), ints(2))
    calls = (lambda: kvq.kvq_score(*args, path=ints(2, width)), lambda: kvq.kvq_commit(cache, ints(2), ints(2, width), ints(2), 4))
    for call in calls:
        if width:
            call()
        else:
            with pytest.raises(ValueError, match="path"):
                call()
    assert bool(called) == bool(width)


@pytest.mark.parametrize("name", ["sink", "recent"])
@pytest.mark.parametrize("value", [0, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, -1])
def test_counts_past_31_bits_do_not_wrap(monkeypatch, name, value):
    cache, ints, called = stand_in(monkeypatch)
    call = lambda: kvq.kvq_evict(cache, gpu(torch.zeros(2, 3, 8)), ints(2, 3, 8), ints(2), ints(2), 4, **{name: value})  # noqa: E731
    if 0 <= value < 2 ** 31:
        call()
        assert called[0][6 if name == "sink" else 7] == value
    else:
        with pytest.raises(ValueError, match=name):
            call()
        assert not called


@pytest.mark.parametrize("scale", [2.5e38, 3.4e38])
def test_scales_whose_base_two_form_is_infinite(scale):
    """scale * log2(e) is what the kernels multiply by: an infinite one would make NaN of a score of zero."""
    import test_kvq_host as host
    import rejection_sampling_verify_10_amd as R
    c = host.cache(R)
    assert host.attend(R, c, scale=scale) == host.EINVAL
    assert host.score(R, c, scale=scale) == host.EINVAL
