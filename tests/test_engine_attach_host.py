"""What SpecVerifyEngine makes of a state and a paged cache attached to it, on the CPU with recorded calls."""

import pytest

torch = pytest.importorskip("torch")

import mtp_speculative_decoding_spec_gb300 as spec  # noqa: E402
from mtp_speculative_decoding_spec_gb300 import engine as eng_mod  # noqa: E402
from test_engine_host import B, K_MAX, R, _engine, _names, calls, d  # noqa: E402,F401


def pair(kv_layers, state_len, cache_len):
    st, c = spec.spec_state_desc(), spec.spec_paged_cache()
    st.kv_layers, st.kv_len, c.kv_len = kv_layers, state_len, cache_len
    return st, c


@pytest.mark.parametrize("state_first", [True, False])
def test_one_kv_len_of_two_caches_is_refused(calls, state_first):  # noqa: F811
    """Both commits would move it."""
    st, c = pair(2, 4096, 4096)
    e = _engine()
    both = [lambda: e.attach_state(st, spec.SPEC_COMMIT_SNAPSHOT), lambda: e.attach_paged(c)]
    first, second = both if state_first else both[::-1]
    first()
    with pytest.raises(ValueError, match="kv_len"):
        second()
    assert (e.state, e.paged) == ((st, None) if state_first else (None, c))


@pytest.mark.parametrize("kv_layers,state_len", [(0, 4096), (0, None), (2, 8192)])
@pytest.mark.parametrize("state_first", [True, False])
def test_a_state_without_kv_layers_or_with_lengths_of_its_own_is_taken(calls, monkeypatch, kv_layers,  # noqa: F811
                                                                       state_len, state_first):
    monkeypatch.setattr(eng_mod, "spec_paged_commit", lambda *a: calls.append(("spec_paged_commit", a)))
    st, c = pair(kv_layers, state_len, 4096)
    e = _engine()
    both = [lambda: e.attach_state(st, spec.SPEC_COMMIT_SNAPSHOT), lambda: e.attach_paged(c)]
    for attach in both if state_first else both[::-1]:
        attach()
    e.verify_cycle(torch.zeros((B * R, d)))
    assert _names(calls)[-2:] == ["spec_commit_rollback", "spec_paged_commit"]


def test_what_is_attached_after_a_width_graph_is_committed_too(calls, monkeypatch):  # noqa: F811
    """The graph's bodies hold the commits: it is captured anew."""
    monkeypatch.setattr(eng_mod, "spec_paged_commit", lambda *a: calls.append(("spec_paged_commit", a)))
    st, c = pair(0, None, 4096)
    e = _engine(b=1, adaptive_cost=[1.0, 1.5, 2.0, 2.5])
    H, Hd = torch.ones((K_MAX + 1, d)), torch.ones((K_MAX, 1, d))
    e.cycle(H, Hd, K_MAX)
    assert e.graph_exec is not None and "spec_paged_commit" not in _names(calls)
    for attach, name in ((lambda: e.attach_paged(c), "spec_paged_commit"),
                         (lambda: e.attach_state(st, spec.SPEC_COMMIT_SNAPSHOT), "spec_commit_rollback")):
        calls.clear()
        attach()
        e.cycle(H, Hd, K_MAX)
        names = _names(calls)
        assert names[:2] == ["spec_graph_destroy", "spec_width_graph_create"]
        assert names.count(name) == K_MAX + 1 and names[-1] == "spec_graph_launch"
        calls.clear()
        e.cycle(H, Hd, K_MAX)
        assert _names(calls) == ["spec_graph_launch"]
