"""Trees of drafted tokens without a GPU: arguments that share memory, and the order
of TreeDecode's calls."""

import ctypes as C

import pytest
import torch

import mla_chunked_context_gb300 as M
from mla_chunked_context_gb300 import _lib

from test_abi_cpu import built_library  # noqa: F401  (builds the library when it is stale)
from test_decode_cpu import INVALID, UNSUPPORTED, dims


def commit(new, R=3, path=1 << 20, path_ld=4, kept=2 << 20, qsl=3 << 20, lens=4 << 20, table=5 << 20, stride=2):
    arr = (C.c_void_p * 1)(8 << 20)
    p = C.c_void_p
    return _lib.lib().mla_commit_tree(C.byref(dims()), R, 3, p(path), path_ld, p(kept), p(qsl), p(lens), arr, 1, 4,
                                      p(table), stride, p(new), None, None)


@pytest.mark.parametrize("at,size,code", [(4 << 20, 3, INVALID), (2 << 20, 3, UNSUPPORTED), (3 << 20, 4, UNSUPPORTED),
                                          (1 << 20, 12, UNSUPPORTED), (5 << 20, 6, UNSUPPORTED)])
def test_commit_refuses_new_lengths_over_its_inputs(at, size, code):
    """Three new lengths over `size` integers: the same, the first or the last one in
    common; right beside them is no overlap."""
    for shift in (0, -2, size - 1):
        assert commit(at + 4 * shift) == code, shift
    if not torch.cuda.is_available():                # (would launch on these addresses)
        for shift in (-3, size):
            assert commit(at + 4 * shift) not in (INVALID, UNSUPPORTED), shift


def planned(monkeypatch, capturing, max_tokens=4):
    """A TreeDecode on the CPU whose calls only note that they were made, and the
    notes."""
    made = []
    for name in ("mla_tree_layout", "mla_verify_tree", "mla_commit_tree"):
        monkeypatch.setattr(M, name, lambda *a, name=name: made.append(name))
    monkeypatch.setattr(M, "_capturing", lambda stream: capturing)
    d = M.Dims(2, 64, 16, 32, 32, 16, 0.1, torch.float32)
    return M.TreeDecode(d, max_tokens, 2, device="cpu"), made


def plan(dec):
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    dec.plan(z(3), z(3), z(2))


def test_commit_wants_a_verification_of_the_planned_trees(monkeypatch):
    """Else it would commit the path of the step before."""
    dec, made = planned(monkeypatch, False)
    for _ in range(2):
        plan(dec)
        with pytest.raises(ValueError, match="verify comes before commit"):
            dec.commit([], None)
        dec.verify(None, None)
        dec.commit([], None)
        dec.commit([], None)                         # other layers' caches
    assert made == ["mla_tree_layout", "mla_verify_tree", "mla_commit_tree", "mla_commit_tree"] * 2


def test_a_captured_verification_may_be_replayed_between_plan_and_commit(monkeypatch):
    dec, made = planned(monkeypatch, True)
    plan(dec)
    dec.verify(None, None)
    plan(dec)
    dec.commit([], None)
    assert made[-1] == "mla_commit_tree"


@pytest.mark.parametrize("tokens,words", [(1, 1), (64, 1), (65, 2), (200, 4), (1024, 16), (5000, 16)])
def test_masks_have_room_for_any_tree_that_is_verified(tokens, words):
    d = M.Dims(1, 16, 0, 8, 8, 16, 0.1, torch.float32)
    assert M.TreeDecode(d, tokens, 2, device="cpu").tree_mask.shape == (tokens, words)
    assert M.TreeDecode(d, tokens, 2, mask_words=3, device="cpu").tree_mask.shape == (tokens, 3)
